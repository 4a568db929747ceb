// Host side of the C ABI declared in include/kda_linear.h and
// include/kda_norm.h: argument validation, workspace carving and kernel
// launches on the caller's stream. No host synchronisation, no allocation, no
// host read of device memory.
#include <math.h>

#include <algorithm>

#include "../../include/kda_linear.h"
#include "../../include/kda_norm.h"
#include "linear_launch.h"

namespace {

constexpr int kMaxHeads = 4096;  // as in kda.h: one chunk's rows stay below 2^31 bytes
constexpr int kMaxNormWidth = 16384;
constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned256(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
bool width_ok(int d) { return d >= 8 && d <= 256 && d % 8 == 0; }
int qk_heads(const kda_linear_args *a) { return a->Hk > 0 ? a->Hk : a->H; }
float resolve_scale(const kda_linear_args *a) { return a->scale > 0.f ? a->scale : 1.0f / sqrtf((float)a->K); }

// Sizes only (also for the workspace queries).
kda_status check_sizes(const kda_linear_args *a) {
  if (!a) return KDA_ERR_NULL;
  if (a->B < 1 || a->T < 0 || a->H < 1 || a->H > kMaxHeads || a->N < 0) return KDA_ERR_SHAPE;
  if (a->Hk < 0 || (a->Hk > 0 && a->H % a->Hk != 0)) return KDA_ERR_SHAPE;
  if (a->K < 1 || a->V < 1) return KDA_ERR_SHAPE;
  if (a->dtype != KDA_BF16 && a->dtype != KDA_F32) return KDA_ERR_DTYPE;
  if (a->decay != KDA_DECAY_TOKEN && a->decay != KDA_DECAY_HEAD) return KDA_ERR_GATE;
  if (!width_ok(a->K) || !width_ok(a->V)) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

kda_status check_common(const kda_linear_args *a, const void *q, const void *k, const void *v, const float *g,
                        const float *h0, const int32_t *cu, const void *o, const float *ht) {
  const kda_status s = check_sizes(a);
  if (s != KDA_OK && s != KDA_ERR_UNSUPPORTED) return s;
  if (cu ? a->B != 1 : a->N != a->B) return KDA_ERR_SHAPE;
  if (a->T > 0 && (!q || !k || !v || !o || !g)) return KDA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(h0) || !aligned16(o) ||
      !aligned16(ht))
    return KDA_ERR_ALIGN;
  return s;
}

// What one walk keeps in the workspace: the segments' boundary states and
// decays, and copies of the initial states (for an in-place final state).
struct SegPlan {
  int seg = 0;
  size_t state = 0, decay = 0, first = 0;
  size_t total() const { return align_up(state) + align_up(decay) + align_up(first); }
};

SegPlan seg_plan(const kda_linear_args *a, bool packed, int P, int Q, bool dots) {
  SegPlan s;
  s.seg = kda::linear_segment(a->T, a->N, a->H, P, Q, a->dtype == KDA_BF16, packed, dots);
  if (!s.seg) return s;
  const size_t elems = (size_t)a->H * a->K * a->V;
  const size_t bounds = (size_t)((int64_t)a->B * a->T / s.seg + 1);
  s.state = 4 * bounds * elems;
  s.decay = 8 * bounds * a->H;
  s.first = 4 * (size_t)a->N * elems;
  return s;
}

void set_segments(kda::LinearWalk &w, const SegPlan &s, char *ws, bool in_place) {
  w.seg = s.seg;
  if (!s.seg) return;
  w.seg_state = reinterpret_cast<float *>(ws);
  w.seg_decay = reinterpret_cast<double *>(ws + align_up(s.state));
  w.seg_first = in_place ? reinterpret_cast<float *>(ws + align_up(s.state) + align_up(s.decay)) : nullptr;
}

kda::LinearWalk walk_base(const kda_linear_args *a, const float *g, const int32_t *cu) {
  kda::LinearWalk w{};
  w.g = g;
  w.g_head = a->decay == KDA_DECAY_HEAD;
  w.cu = cu;
  w.B = a->B;
  w.T = a->T;
  w.H = a->H;
  w.N = a->N;
  w.Hk = qk_heads(a);
  w.scale = resolve_scale(a);
  w.is_bf16 = a->dtype == KDA_BF16;
  return w;
}

bool walk_fits(const kda_linear_args *a, int P, int Q, int seg) {
  kda::LinearWalk w = walk_base(a, nullptr, nullptr);
  w.P = P;
  w.Q = Q;
  w.seg = seg;
  return kda::linear_walk_fits(w);
}

// The backward's workspace.
struct BwdPlan {
  SegPlan seg;  // of all three walks: dk's starts from the boundary states of dv's
  size_t segs, ckpt, dots, adot, ends, heads, part;
  int ncb;
  int64_t anchors, items;
  size_t total() const {
    return align_up(segs) + align_up(ckpt) + 4 * align_up(dots) + align_up(adot) + 2 * align_up(ends) +
           align_up(heads) + align_up(part);
  }
};

BwdPlan bwd_plan(const kda_linear_args *a, bool packed) {
  BwdPlan b;
  b.seg = seg_plan(a, packed, a->V, a->K, true);
  b.segs = b.seg.total();
  const int qt = kda::linear_cols(a->V, a->K, a->dtype == KDA_BF16, (int64_t)a->N * a->H, &b.ncb);
  const int64_t rows = (int64_t)a->B * a->T;
  b.anchors = rows / kda::kLinearAnchor + 1;
  b.ckpt = 4 * (size_t)b.anchors * a->H * b.ncb * kda::linear_tile(a->V) * qt;
  b.dots = 4 * (size_t)b.ncb * a->H * rows;
  b.adot = 4 * (size_t)b.anchors * a->H * b.ncb;
  b.ends = 4 * (size_t)a->N * a->H * b.ncb;
  b.heads = qk_heads(a) != a->H ? 4 * (size_t)rows * a->H * a->K : 0;
  b.items = kda::linear_dg_items(a->B, a->T, a->N);
  b.part = a->decay == KDA_DECAY_HEAD ? 8 * (size_t)b.items * a->H : 0;
  return b;
}

// Whether these sizes describe a dense batch, and whether a packed one (a
// workspace query sees no cu_seqlens; N == B == 1 can be either).
bool maybe_dense(const kda_linear_args *a) { return a->N == a->B; }
bool maybe_packed(const kda_linear_args *a) { return a->B == 1; }

}  // namespace

extern "C" size_t kda_linear_chunk_workspace_bytes(const kda_linear_args *a) {
  if (check_sizes(a) != KDA_OK) return 0;
  size_t n = 0;
  if (maybe_dense(a)) n = std::max(n, seg_plan(a, false, a->K, a->V, false).total());
  if (maybe_packed(a)) n = std::max(n, seg_plan(a, true, a->K, a->V, false).total());
  return n;
}

extern "C" kda_status kda_linear_chunk_fwd(const kda_linear_args *a, const void *q, const void *k, const void *v,
                                           const float *g, const float *h0, const int32_t *cu, void *o, float *ht,
                                           void *workspace, size_t ws_bytes, void *stream) {
  const kda_status s = check_common(a, q, k, v, g, h0, cu, o, ht);
  if (s != KDA_OK) return s;
  const SegPlan plan = seg_plan(a, cu != nullptr, a->K, a->V, false);
  if (!walk_fits(a, a->K, a->V, plan.seg)) return KDA_ERR_UNSUPPORTED;
  if (plan.total() > 0 && (!workspace || ws_bytes < plan.total())) return KDA_ERR_WORKSPACE;
  if (plan.total() > 0 && !aligned256(workspace)) return KDA_ERR_ALIGN;
  kda::LinearWalk w = walk_base(a, g, cu);
  w.x = q;
  w.z = k;
  w.w = v;
  w.y = o;
  w.Hx = qk_heads(a);
  w.Hw = w.Hu = a->H;
  w.P = a->K;
  w.Q = a->V;
  w.s0 = h0;
  w.sT = ht;
  w.sp = a->V;
  w.sq = 1;
  set_segments(w, plan, static_cast<char *>(workspace), h0 && ht == h0);
  return kda::report_hip(kda::launch_linear_walk(w, (hipStream_t)stream));
}

extern "C" size_t kda_linear_chunk_bwd_workspace_bytes(const kda_linear_args *a) {
  if (check_sizes(a) != KDA_OK) return 0;
  size_t n = 0;
  if (maybe_dense(a)) n = std::max(n, bwd_plan(a, false).total());
  if (maybe_packed(a)) n = std::max(n, bwd_plan(a, true).total());
  return n;
}

extern "C" kda_status kda_linear_chunk_bwd(const kda_linear_args *a, const void *q, const void *k, const void *v,
                                           const float *g, const float *h0, const int32_t *cu, const void *d_o,
                                           const float *dht, void *dq, void *dk, void *dv, float *dg, float *dh0,
                                           void *workspace, size_t ws_bytes, void *stream) {
  const kda_status s = check_common(a, q, k, v, g, h0, cu, d_o, dht);
  if (s != KDA_OK && s != KDA_ERR_UNSUPPORTED) return s;
  if (!dg && (a->T > 0 || a->decay == KDA_DECAY_HEAD)) return KDA_ERR_NULL;
  if (a->T > 0 && (!dq || !dk || !dv)) return KDA_ERR_NULL;
  if (!aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(dg) || !aligned16(dh0)) return KDA_ERR_ALIGN;
  if (s != KDA_OK) return s;
  const BwdPlan b = bwd_plan(a, cu != nullptr);
  if (!walk_fits(a, a->V, a->K, b.seg.seg) || !walk_fits(a, a->K, a->V, b.seg.seg) ||
      (b.heads > 0 && !kda::linear_group_sum_fits((int64_t)a->B * a->T, qk_heads(a), a->K)) ||
      !kda::linear_dg_fits(b.items, a->H))
    return KDA_ERR_UNSUPPORTED;
  if (!workspace || ws_bytes < b.total()) return KDA_ERR_WORKSPACE;
  if (!aligned256(workspace)) return KDA_ERR_ALIGN;
  char *at = static_cast<char *>(workspace);
  auto take = [&](size_t bytes) {
    char *r = at;
    at += align_up(bytes);
    return r;
  };
  char *segs = take(b.segs);
  float *ckpt = reinterpret_cast<float *>(take(b.ckpt));
  float *dot_q = reinterpret_cast<float *>(take(b.dots)), *dot_k = reinterpret_cast<float *>(take(b.dots));
  float *far_q = reinterpret_cast<float *>(take(b.dots)), *far_k = reinterpret_cast<float *>(take(b.dots));
  float *adot = reinterpret_cast<float *>(take(b.adot));
  float *sdot = reinterpret_cast<float *>(take(b.ends)), *edot = reinterpret_cast<float *>(take(b.ends));
  float *heads = reinterpret_cast<float *>(take(b.heads));
  double *part = reinterpret_cast<double *>(take(b.part));
  const int Hk = qk_heads(a);
  const bool shared = Hk != a->H;
  const int64_t rows = (int64_t)a->B * a->T;
  const hipStream_t st = (hipStream_t)stream;

  // dq: a walk with the state transposed, h^T; it leaves q.dq and the states that anchor dg
  kda::LinearWalk w = walk_base(a, g, cu);
  w.x = d_o;
  w.z = v;
  w.w = k;
  w.u = q;
  w.y = shared ? static_cast<void *>(heads) : dq;
  w.y_f32 = shared;
  w.dot = dot_q;
  w.dot_far = far_q;
  w.Hx = a->H;
  w.Hw = w.Hu = Hk;
  w.P = a->V;
  w.Q = a->K;
  w.s0 = h0;
  w.sp = 1;
  w.sq = a->V;
  w.s_dot = dht;
  w.end_dot = dht ? edot : nullptr;
  w.ckpt = ckpt;
  set_segments(w, b.seg, segs, false);
  hipError_t e = kda::launch_linear_walk(w, st);
  if (e == hipSuccess && shared)
    e = kda::launch_linear_group_sum(heads, dq, w.is_bf16, cu, a->N, rows, a->H, Hk, a->K, st);
  if (e != hipSuccess) return kda::report_hip(e);

  // dv: the reverse walk of dh, which ends in dh0
  kda::LinearWalk r = walk_base(a, g, cu);
  r.reverse = true;
  r.x = k;
  r.z = q;
  r.w = d_o;
  r.y = dv;
  r.Hx = Hk;
  r.Hw = r.Hu = a->H;
  r.P = a->K;
  r.Q = a->V;
  r.s0 = dht;
  r.sT = dh0;
  r.sp = a->V;
  r.sq = 1;
  set_segments(r, b.seg, segs, false);
  e = kda::launch_linear_walk(r, st);
  if (e != hipSuccess) return kda::report_hip(e);

  // dk: the reverse walk of dh^T, with <h, dh> at the anchors and at its end
  w.reverse = true;
  w.x = v;
  w.z = d_o;
  w.w = q;
  w.u = k;
  w.y = shared ? static_cast<void *>(heads) : dk;
  w.dot = dot_k;
  w.dot_far = far_k;
  w.s0 = dht;
  w.s_dot = h0;
  w.end_dot = h0 ? sdot : nullptr;
  w.anchor_dot = adot;
  set_segments(w, b.seg, segs, false);
  w.seg_ready = true;  // dv's boundary states, read across
  e = kda::launch_linear_walk(w, st);
  if (e == hipSuccess && shared)
    e = kda::launch_linear_group_sum(heads, dk, w.is_bf16, cu, a->N, rows, a->H, Hk, a->K, st);
  if (e != hipSuccess) return kda::report_hip(e);

  kda::LinearDg d{};
  d.a = dot_q;
  d.b = dot_k;
  d.a_far = far_q;
  d.b_far = far_k;
  d.chunk = kda::linear_chunk_rows(a->V, a->dtype == KDA_BF16);
  d.anchor_dot = adot;
  d.start_dot = h0 ? sdot : nullptr;
  d.end_dot = dht ? edot : nullptr;
  d.cu = cu;
  d.dg = dg;
  d.part = part;
  d.g_head = a->decay == KDA_DECAY_HEAD;
  d.B = a->B;
  d.T = a->T;
  d.H = a->H;
  d.N = a->N;
  d.ncb = b.ncb;
  return kda::report_hip(kda::launch_linear_dg(d, st));
}

extern "C" kda_status kda_linear_recurrent_fwd(const kda_linear_args *a, const void *q, const void *k, const void *v,
                                               const float *g, const float *h0, const int32_t *cu, void *o, float *ht,
                                               void *stream) {
  const kda_status s = check_common(a, q, k, v, g, h0, cu, o, ht);
  if (s != KDA_OK) return s;
  kda::LinearRecurrent p{};
  p.q = q;
  p.k = k;
  p.v = v;
  p.g = g;
  p.h0 = h0;
  p.cu = cu;
  p.o = o;
  p.ht = ht;
  p.scale = resolve_scale(a);
  p.g_head = a->decay == KDA_DECAY_HEAD;
  p.is_bf16 = a->dtype == KDA_BF16;
  p.B = a->B;
  p.T = a->T;
  p.H = a->H;
  p.K = a->K;
  p.V = a->V;
  p.N = a->N;
  p.Hk = qk_heads(a);
  if (!kda::linear_recurrent_fits(p)) return KDA_ERR_UNSUPPORTED;
  return kda::report_hip(kda::launch_linear_recurrent(p, (hipStream_t)stream));
}

// ---------------------------------------------------------------------------------------------
// block norm
// ---------------------------------------------------------------------------------------------
namespace {

kda_status check_norm(const kda_norm_args *a) {
  if (!a) return KDA_ERR_NULL;
  if (a->rows < 0 || a->D < 1 || !(a->eps >= 0.f) || a->rows > (int64_t)1 << 40) return KDA_ERR_SHAPE;
  if ((a->dtype != KDA_BF16 && a->dtype != KDA_F32) || (a->res_dtype != a->dtype && a->res_dtype != KDA_F32))
    return KDA_ERR_DTYPE;
  if ((a->norm != KDA_NORM_RMS && a->norm != KDA_NORM_L2) ||
      (a->gate_act != KDA_ACT_SIGMOID && a->gate_act != KDA_ACT_SILU))
    return KDA_ERR_GATE;
  if (a->D % 8 != 0 || a->D > kMaxNormWidth) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

kda::BlockNorm norm_base(const kda_norm_args *a, const void *x, const float *weight, const void *gate,
                         const void *residual, const float *scale_vec, const float *next_weight) {
  kda::BlockNorm p{};
  p.x = x;
  p.weight = weight;
  p.gate = gate;
  p.residual = residual;
  p.scale_vec = scale_vec;
  p.next_weight = next_weight;
  p.rows = a->rows;
  p.D = a->D;
  p.is_bf16 = a->dtype == KDA_BF16;
  p.res_f32 = a->res_dtype == KDA_F32;
  p.l2 = a->norm == KDA_NORM_L2;
  p.silu = a->gate_act == KDA_ACT_SILU;
  p.scale = a->scale;
  p.eps = a->eps;
  return p;
}

}  // namespace

extern "C" kda_status kda_block_norm_fwd(const kda_norm_args *a, const void *x, const float *weight, const void *gate,
                                         const void *residual, const float *scale_vec, const float *next_weight,
                                         void *y, void *z, void *stream) {
  const kda_status s = check_norm(a);
  if (s != KDA_OK) return s;
  if (a->rows > 0 && !residual && a->res_dtype != a->dtype) return KDA_ERR_DTYPE;  // no rows: no address
  if (a->rows > 0 && (!x || !y)) return KDA_ERR_NULL;
  if (!aligned16(x) || !aligned16(weight) || !aligned16(gate) || !aligned16(residual) || !aligned16(scale_vec) ||
      !aligned16(next_weight) || !aligned16(y) || !aligned16(z))
    return KDA_ERR_ALIGN;
  kda::BlockNorm p = norm_base(a, x, weight, gate, residual, scale_vec, next_weight);
  p.y = y;
  p.z = z;
  return kda::report_hip(kda::launch_block_norm_fwd(p, (hipStream_t)stream));
}

extern "C" size_t kda_block_norm_bwd_workspace_bytes(const kda_norm_args *a) {
  return check_norm(a) == KDA_OK ? kda::block_norm_bwd_part_bytes(a->rows, a->D) : 0;
}

extern "C" kda_status kda_block_norm_bwd(const kda_norm_args *a, const void *x, const float *weight, const void *gate,
                                         const void *residual, const float *scale_vec, const float *next_weight,
                                         const void *dy, const void *dz, void *dx, void *dgate, void *dresidual,
                                         float *dweight, float *dscale_vec, float *dnext_weight, void *workspace,
                                         size_t ws_bytes, void *stream) {
  const kda_status s = check_norm(a);
  if (s != KDA_OK) return s;
  if (a->rows > 0 && !residual && a->res_dtype != a->dtype) return KDA_ERR_DTYPE;  // no rows: no address
  if (a->rows > 0 && (!x || !dx || (!dy && !dz) || (gate && !dgate) || (dnext_weight && !dz)))
    return KDA_ERR_NULL;
  if (!aligned16(x) || !aligned16(weight) || !aligned16(gate) || !aligned16(residual) || !aligned16(scale_vec) ||
      !aligned16(next_weight) || !aligned16(dy) || !aligned16(dz) || !aligned16(dx) || !aligned16(dgate) ||
      !aligned16(dresidual) || !aligned16(dweight) || !aligned16(dscale_vec) || !aligned16(dnext_weight))
    return KDA_ERR_ALIGN;
  if (dweight || dscale_vec || dnext_weight) {
    if (!workspace || ws_bytes < kda_block_norm_bwd_workspace_bytes(a)) return KDA_ERR_WORKSPACE;
    if (!aligned256(workspace)) return KDA_ERR_ALIGN;
  }
  kda::BlockNorm p = norm_base(a, x, weight, gate, residual, scale_vec, next_weight);
  p.dy = dy;
  p.dz = dz;
  p.dx = dx;
  p.dgate = gate ? dgate : nullptr;
  p.dresidual = dresidual;
  p.dweight = dweight;
  p.dscale_vec = dscale_vec;
  p.dnext_weight = dnext_weight;
  p.part = static_cast<float *>(workspace);
  return kda::report_hip(kda::launch_block_norm_bwd(p, (hipStream_t)stream));
}
