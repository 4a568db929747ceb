// Host side of the C ABI declared in include/kda_delta.h: argument validation,
// workspace carving and kernel launches on the caller's stream. No host
// synchronisation, no allocation, no host read of device memory.
#include <math.h>

#include <algorithm>

#include "../../include/kda_delta.h"
#include "delta_launch.h"

namespace {

constexpr int kMaxHeads = 4096;  // as in kda.h: one chunk's rows stay below 2^31 bytes
constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned256(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
bool width_ok(int d) { return d >= 8 && d <= 256 && d % 8 == 0; }
int qk_heads(const kda_delta_args *a) { return a->Hk > 0 ? a->Hk : a->H; }

// Sizes only (also for the workspace queries).
kda_status check_sizes(const kda_delta_args *a) {
  if (!a) return KDA_ERR_NULL;
  if (a->B < 1 || a->T < 0 || a->H < 1 || a->H > kMaxHeads || a->N < 0) return KDA_ERR_SHAPE;
  if (a->Hk < 0 || (a->Hk > 0 && a->H % a->Hk != 0)) return KDA_ERR_SHAPE;
  if (a->K < 1 || a->V < 1) return KDA_ERR_SHAPE;
  if (a->dtype != KDA_BF16 && a->dtype != KDA_F32) return KDA_ERR_DTYPE;
  if (!width_ok(a->K) || !width_ok(a->V)) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

kda_status check_common(const kda_delta_args *a, const void *q, const void *k, const void *v, const float *g,
                        const float *beta, const float *h0, const int32_t *cu, const void *o, const float *ht) {
  const kda_status s = check_sizes(a);
  if (s != KDA_OK && s != KDA_ERR_UNSUPPORTED) return s;
  if (cu ? a->B != 1 : a->N != a->B) return KDA_ERR_SHAPE;
  if (a->T > 0 && (!q || !k || !v || !beta || !o)) return KDA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(beta) || !aligned16(h0) ||
      !aligned16(o) || !aligned16(ht))
    return KDA_ERR_ALIGN;
  return s;
}

int chunk_of(const kda_delta_args *a) { return kda::delta_chunk(kda::linear_tile(a->K), a->dtype == KDA_BF16); }
int64_t rows_of(const kda_delta_args *a) { return (int64_t)a->B * a->T; }
int64_t slots_of(const kda_delta_args *a) { return a->T > 0 ? kda::delta_slots(rows_of(a), a->N, chunk_of(a)) : 0; }
size_t inverse_bytes(const kda_delta_args *a) {
  return align_up((size_t)slots_of(a) * a->H * kda::delta_inverse_bytes(chunk_of(a)));
}

kda::DeltaPrep prep_base(const kda_delta_args *a, const void *k, const float *g, const float *beta, const int32_t *cu) {
  kda::DeltaPrep p{};
  p.k = k;
  p.g = g;
  p.beta = beta;
  p.cu = cu;
  p.B = a->B;
  p.T = a->T;
  p.H = a->H;
  p.K = a->K;
  p.N = a->N;
  p.Hk = qk_heads(a);
  p.is_bf16 = a->dtype == KDA_BF16;
  return p;
}

kda::DeltaWalk walk_base(const kda_delta_args *a, const void *q, const void *k, const float *g, const float *beta,
                         const int32_t *cu) {
  kda::DeltaWalk w{};
  w.q = q;
  w.k = k;
  w.g = g;
  w.beta = beta;
  w.cu = cu;
  w.B = a->B;
  w.T = a->T;
  w.H = a->H;
  w.K = a->K;
  w.V = a->V;
  w.N = a->N;
  w.Hk = qk_heads(a);
  w.scale = a->scale > 0.f ? a->scale : 1.0f / sqrtf((float)a->K);
  w.is_bf16 = a->dtype == KDA_BF16;
  return w;
}

// What the segments of a walk keep in the workspace.
struct SegPlan {
  int seg = 0;
  size_t state = 0, map = 0, first = 0, bound = 0, zero = 0;
  size_t total() const { return align_up(state) + align_up(map) + align_up(first) + align_up(bound) + align_up(zero); }
};
SegPlan seg_plan(const kda_delta_args *a, bool packed, bool gated) {
  SegPlan s;
  kda::DeltaWalk w = walk_base(a, nullptr, nullptr, nullptr, nullptr, nullptr);
  s.seg = kda::delta_segment(w, packed, gated);
  if (!s.seg) return s;
  const size_t bounds = (size_t)(rows_of(a) / s.seg + 1) * a->H;
  s.state = 4 * bounds * a->K * a->V;
  s.map = 4 * bounds * a->K * a->K;
  s.first = 4 * (size_t)a->N * a->H * a->K * a->V;
  s.bound = 4 * (size_t)slots_of(a) * a->H;
  s.zero = 4 * bounds;
  return s;
}
// Whether these sizes describe a dense batch, and whether a packed one (a workspace query
// sees no cu_seqlens; N == B == 1 can be either).
bool maybe_dense(const kda_delta_args *a) { return a->N == a->B; }
bool maybe_packed(const kda_delta_args *a) { return a->B == 1; }
// What segments may need for these sizes, with g or without.
size_t most_segments(const kda_delta_args *a) {
  size_t n = 0;
  for (int gated = 0; gated < 2; ++gated) {
    if (maybe_dense(a)) n = std::max(n, seg_plan(a, false, gated).total());
    if (maybe_packed(a)) n = std::max(n, seg_plan(a, true, gated).total());
  }
  return n;
}

// The backward's workspace.
struct BwdPlan {
  size_t inv, row, state, heads;
  size_t total() const { return inv + 2 * align_up(row) + 2 * align_up(state) + 2 * align_up(heads); }
};
BwdPlan bwd_plan(const kda_delta_args *a) {
  BwdPlan b;
  b.inv = inverse_bytes(a);
  b.row = 4 * (size_t)rows_of(a) * a->H * a->V;                   // u, du
  b.state = 4 * (size_t)slots_of(a) * a->H * a->K * a->V;         // states and their gradients
  b.heads = qk_heads(a) != a->H ? 4 * (size_t)rows_of(a) * a->H * a->K : 0;  // dq, dk of each value head
  return b;
}

}  // namespace

extern "C" size_t kda_delta_chunk_workspace_bytes(const kda_delta_args *a) {
  if (check_sizes(a) != KDA_OK || a->T == 0) return 0;
  return most_segments(a) + inverse_bytes(a);
}

extern "C" kda_status kda_delta_chunk_fwd(const kda_delta_args *a, const void *q, const void *k, const void *v,
                                          const float *g, const float *beta, const float *h0, const int32_t *cu,
                                          void *o, float *ht, void *workspace, size_t ws_bytes, void *stream) {
  const kda_status s = check_common(a, q, k, v, g, beta, h0, cu, o, ht);
  if (s != KDA_OK) return s;
  kda::DeltaPrep p = prep_base(a, k, g, beta, cu);
  kda::DeltaWalk w = walk_base(a, q, k, g, beta, cu);
  const SegPlan plan = a->T > 0 ? seg_plan(a, cu != nullptr, g != nullptr) : SegPlan{};
  w.seg = plan.seg;
  if (!kda::delta_prep_fits(p) || !kda::delta_walk_fits(w)) return KDA_ERR_UNSUPPORTED;
  const size_t need = inverse_bytes(a) + plan.total();
  if (need > 0 && (!workspace || ws_bytes < need)) return KDA_ERR_WORKSPACE;
  if (need > 0 && !aligned256(workspace)) return KDA_ERR_ALIGN;
  const hipStream_t st = (hipStream_t)stream;
  char *at = static_cast<char *>(workspace) + inverse_bytes(a);
  if (plan.seg) {
    w.seg_state = reinterpret_cast<float *>(at);
    at += align_up(plan.state);
    w.seg_map = reinterpret_cast<float *>(at);
    at += align_up(plan.map);
    w.seg_first = h0 && ht == h0 ? reinterpret_cast<float *>(at) : nullptr;
    at += align_up(plan.first);
    p.bound = reinterpret_cast<float *>(at);
    w.bound = p.bound;
    w.seg_zero = reinterpret_cast<int *>(at + align_up(plan.bound));
  }
  if (a->T > 0) {
    p.inv = static_cast<char *>(workspace);
    p.fold = true;
    const hipError_t e = kda::launch_delta_prep(p, st);
    if (e != hipSuccess) return kda::report_hip(e);
  }
  w.v = v;
  w.inv = static_cast<const char *>(workspace);
  w.s0 = h0;
  w.sT = ht;
  w.o = o;
  return kda::report_hip(kda::launch_delta_walk(w, st));
}

extern "C" kda_status kda_delta_recurrent_fwd(const kda_delta_args *a, const void *q, const void *k, const void *v,
                                              const float *g, const float *beta, const float *h0, const int32_t *cu,
                                              void *o, float *ht, void *stream) {
  const kda_status s = check_common(a, q, k, v, g, beta, h0, cu, o, ht);
  if (s != KDA_OK) return s;
  kda::DeltaRecurrent p{};
  p.q = q;
  p.k = k;
  p.v = v;
  p.g = g;
  p.beta = beta;
  p.h0 = h0;
  p.cu = cu;
  p.o = o;
  p.ht = ht;
  p.scale = a->scale > 0.f ? a->scale : 1.0f / sqrtf((float)a->K);
  p.is_bf16 = a->dtype == KDA_BF16;
  p.B = a->B;
  p.T = a->T;
  p.H = a->H;
  p.K = a->K;
  p.V = a->V;
  p.N = a->N;
  p.Hk = qk_heads(a);
  if (!kda::delta_recurrent_fits(p)) return KDA_ERR_UNSUPPORTED;
  return kda::report_hip(kda::launch_delta_recurrent(p, (hipStream_t)stream));
}

extern "C" size_t kda_delta_chunk_bwd_workspace_bytes(const kda_delta_args *a) {
  return check_sizes(a) == KDA_OK ? bwd_plan(a).total() : 0;
}

extern "C" kda_status kda_delta_chunk_bwd(const kda_delta_args *a, const void *q, const void *k, const void *v,
                                          const float *g, const float *beta, const float *h0, const int32_t *cu,
                                          const void *d_o, const float *dht, void *dq, void *dk, void *dv, float *dg,
                                          float *dbeta, float *dh0, void *workspace, size_t ws_bytes, void *stream) {
  const kda_status s = check_common(a, q, k, v, g, beta, h0, cu, d_o, dht);
  if (s != KDA_OK && s != KDA_ERR_UNSUPPORTED) return s;
  if (a->T > 0 && (!dq || !dk || !dv || (g && !dg) || !dbeta)) return KDA_ERR_NULL;
  if (!aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(dg) || !aligned16(dbeta) || !aligned16(dh0))
    return KDA_ERR_ALIGN;
  if (s != KDA_OK) return s;
  const int Hk = qk_heads(a);
  const bool shared = Hk != a->H;
  kda::DeltaPrep p = prep_base(a, k, g, beta, cu);
  kda::DeltaWalk f = walk_base(a, q, k, g, beta, cu), r = f;
  kda::DeltaGrad d{};
  d.q = q;
  d.k = k;
  d.v = v;
  d.d_o = d_o;
  d.g = g;
  d.beta = beta;
  d.cu = cu;
  d.B = a->B;
  d.T = a->T;
  d.H = a->H;
  d.K = a->K;
  d.V = a->V;
  d.N = a->N;
  d.Hk = Hk;
  d.scale = f.scale;
  d.is_bf16 = f.is_bf16;
  if (!kda::delta_prep_fits(p) || !kda::delta_walk_fits(f) || !kda::delta_grad_fits(d) ||
      (shared && !kda::linear_group_sum_fits(rows_of(a), Hk, a->K)))
    return KDA_ERR_UNSUPPORTED;
  const BwdPlan b = bwd_plan(a);
  if (b.total() > 0 && (!workspace || ws_bytes < b.total())) return KDA_ERR_WORKSPACE;
  if (b.total() > 0 && !aligned256(workspace)) return KDA_ERR_ALIGN;
  const hipStream_t st = (hipStream_t)stream;
  char *at = static_cast<char *>(workspace);
  auto take = [&](size_t bytes) {
    char *x = at;
    at += align_up(bytes);
    return x;
  };
  r.v = d_o;
  r.s0 = dht;
  r.sT = dh0;
  if (a->T == 0) return kda::report_hip(dh0 ? kda::launch_delta_walk_rev(r, st) : hipSuccess);
  p.inv = take(b.inv);
  f.rows_out = reinterpret_cast<float *>(take(b.row));
  r.rows_out = reinterpret_cast<float *>(take(b.row));
  f.states = reinterpret_cast<float *>(take(b.state));
  r.states = reinterpret_cast<float *>(take(b.state));
  float *hq = reinterpret_cast<float *>(take(b.heads)), *hd = reinterpret_cast<float *>(take(b.heads));
  f.v = v;
  f.s0 = h0;
  f.inv = p.inv;
  r.inv = p.inv;
  d.u = f.rows_out;
  d.du = r.rows_out;
  d.h = f.states;
  d.dh = r.states;
  d.qk_f32 = shared;
  d.dq = shared ? static_cast<void *>(hq) : dq;
  d.dk = shared ? static_cast<void *>(hd) : dk;
  d.dv = dv;
  d.dg = dg;
  d.dbeta = dbeta;
  d.from_zero = !h0;
  hipError_t e = kda::launch_delta_prep(p, st);
  if (e == hipSuccess) e = kda::launch_delta_walk(f, st);
  if (e == hipSuccess) e = kda::launch_delta_walk_rev(r, st);
  if (e == hipSuccess) e = kda::launch_delta_grad(d, st);
  if (e == hipSuccess && shared) {
    e = kda::launch_linear_group_sum(hq, dq, d.is_bf16, cu, a->N, rows_of(a), a->H, Hk, a->K, st);
    if (e == hipSuccess) e = kda::launch_linear_group_sum(hd, dk, d.is_bf16, cu, a->N, rows_of(a), a->H, Hk, a->K, st);
  }
  return kda::report_hip(e);
}
