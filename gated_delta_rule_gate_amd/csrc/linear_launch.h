// Kernel parameter blocks and launcher declarations of the linear attention
// and block norm operators, shared by their host API (linear_api.hip) and
// their kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/kda.h"

namespace kda {

// kda_status of a HIP result; a failure's text becomes kda_last_error() (kda_api.hip)
kda_status report_hip(hipError_t e);

int device_cus();  // compute units of the current device (chunk_fused.hip)

// Workgroups of one launch: its threads are counted in 32 bits.
constexpr int64_t most_blocks(int threads) { return 0xffffffffLL / threads; }

constexpr int kLinearAnchor = 256;  // tokens between the states that anchor dg

// One walk over the chunks of every sequence. With per-chunk cumulative decays
// b and rows r, s of a chunk of L,
//     y_r = scale (a_r S^T x_r + sum over s of D_rs (x_r . z_s) w_s)
//     S'  = 2^{b_L} S + sum over s of c_s z_s w_s^T
// with S in R^{P x Q}. Walking forward, D_rs = 2^{b_r - b_s} for s <= r,
// a_r = 2^{b_r} and c_s = 2^{b_L - b_s}; in reverse D_rs = 2^{b_s - b_r} for
// s >= r, a_r = 2^{b_L - b_r} and c_s = 2^{b_s}; the scale then goes with z,
// since a state's gradient holds it but the one it starts from does not. The
// forward and all three gradients are such walks:
//     o:  x = q,   z = k,   w = v    S = h           dq: x = d_o, z = v,   w = k   S = h^T
//     dv: x = k,   z = q,   w = d_o  S = dh, reverse  dk: x = v,   z = d_o, w = q   S = dh^T, reverse
struct LinearWalk {
  const void *x, *z, *w;  // [rows, Hx, P], [rows, Hx, P], [rows, Hw, Q]
  const void *u;          // [rows, Hu, Q] or null: partner of the row dots
  void *y;                // [rows, H, Q]
  float *dot, *dot_far;   // [ncb][H][rows]: y_r . u_r in fp32, before y is rounded, and the part
                          // of it that comes through the state (with u)
  int Hx, Hw, Hu;
  bool y_f32;             // y is fp32 whatever the type (a head's part, summed over heads later)
  const float *g;
  bool g_head;            // g [H] instead of [rows, H]
  const float *s0;        // state at the start of the walk or null, [N, H, P x Q]
  float *sT;              // state at its end or null
  int64_t sp, sq;         // strides of the state's P and Q axes in s0, sT and s_dot
  const float *s_dot;     // with end_dot (and sp == 1): state-shaped partner of the last state
  float *end_dot;         // [N, H, ncb] or null
  float *ckpt;            // with u: states every kLinearAnchor tokens of a sequence, written by a
  float *anchor_dot;      // forward walk; a reverse walk leaves <ckpt, S> there, [.., H, ncb]
  const int32_t *cu;
  int B, T, H, P, Q, N;
  int Hk;                 // heads that share q/k data are walked next to each other
  float scale;
  bool is_bf16, reverse;
  // Long sequences on few heads: cut into segments of seg tokens (0: whole
  // sequences) that are walked side by side. A first pass leaves each
  // segment's own state change (and decay) at the boundary behind it, a second
  // chains them, and the walk of every segment starts from its boundary.
  int seg;
  bool seg_ready;         // the boundaries hold the states already (of the same walk, or of its transpose)
  float *seg_state;       // [boundary, H, P x Q], strided as s0
  double *seg_decay;      // [boundary, H] log2
  float *seg_first;       // copies of s0 where sT is s0 itself, [N, H, P x Q], or null
};

int linear_tile(int width);              // padded P: 64, 128 or 256
// columns per workgroup (64 or 128) and column blocks, for `pairs` (sequence, head) pairs
int linear_cols(int P, int width, bool is_bf16, int64_t pairs, int *ncb);
// tokens per segment for one walk with Q columns, or 0 for none; dots: a walk with row dots
int linear_segment(int T, int slots, int H, int P, int Q, bool is_bf16, bool packed, bool dots);
// Workgroups of a walk of ncb column blocks: a unit of those that read the same q/k
// rows after another, units dealt to the eight XCDs.
inline int64_t linear_walk_blocks(const LinearWalk &p, int ncb) {
  const int64_t items = p.N + (p.seg ? ((int64_t)p.B * p.T) / p.seg : 0);
  return (items * p.Hk + 7) / 8 * 8 * (p.H / p.Hk) * ncb;
}
// Whether the launches of these sizes are within HIP's limits: asked before the first
// of a call, so that none fails behind others. (A state pass by 64 columns is taken
// for few pairs only.)
bool linear_walk_fits(const LinearWalk &p);
bool linear_group_sum_fits(int64_t rows, int Hk, int D);
hipError_t launch_linear_walk(const LinearWalk &p, hipStream_t st);
hipError_t launch_linear_walk_bf16_fwd(const LinearWalk &p, hipStream_t st);
hipError_t launch_linear_walk_bf16_rev(const LinearWalk &p, hipStream_t st);
hipError_t launch_linear_walk_f32_fwd(const LinearWalk &p, hipStream_t st);
hipError_t launch_linear_walk_f32_rev(const LinearWalk &p, hipStream_t st);
hipError_t launch_linear_chain(const LinearWalk &p, bool rev, hipStream_t st);

// out[rows, Hk, D] = sum over the heads of a group of in[rows, H, D], in order
hipError_t launch_linear_group_sum(const float *in, void *out, bool is_bf16, const int32_t *cu, int N, int64_t rows,
                                   int H, int Hk, int D, hipStream_t st);

// dg from the row dots a = q.dq and b = k.dk. What a decay at token t scales is
// the sum of a - b from t to the end of the sequence. Most of it cancels, and so
// that the cancelled terms' roundings do not add up, that sum runs to the end of
// t's chunk only; there it is <h, dh>, which is carried over chunks by the dots'
// parts through the states alone (a chunk's own pairs sum to zero) from every
// kLinearAnchor-th token, where the states themselves are at hand; or the same
// from the other side, <h, dh> before t less a - b of the tokens up to t.
struct LinearDg {
  const float *a, *b, *a_far, *b_far;  // [ncb][H][rows]
  const float *anchor_dot, *start_dot, *end_dot;  // <h0, dh0> and <ht, dht>, null: zero
  const int32_t *cu;
  float *dg;
  double *part;        // head decays: [items][H] sums
  bool g_head;
  int chunk;           // rows of the walks' chunks
  int B, T, H, N, ncb;
};
int linear_chunk_rows(int P, bool is_bf16);
int64_t linear_dg_items(int B, int T, int N);
bool linear_dg_fits(int64_t items, int H);
hipError_t launch_linear_dg(const LinearDg &p, hipStream_t st);

struct LinearRecurrent {
  const void *q, *k, *v;
  const float *g, *h0;
  const int32_t *cu;
  void *o;
  float *ht;
  float scale;
  bool g_head, is_bf16;
  int B, T, H, K, V, N, Hk;
};
bool linear_recurrent_fits(const LinearRecurrent &p);
hipError_t launch_linear_recurrent(const LinearRecurrent &p, hipStream_t st);

struct BlockNorm {
  const void *x, *gate, *residual;
  const float *weight, *scale_vec, *next_weight;
  void *y, *z;
  // backward
  const void *dy, *dz;
  void *dx, *dgate, *dresidual;
  float *dweight, *dscale_vec, *dnext_weight;
  float *part;  // [blocks][3][D]
  int64_t rows;
  int D;
  bool is_bf16, res_f32, l2, silu;
  float scale, eps;
};
hipError_t launch_block_norm_fwd(const BlockNorm &p, hipStream_t st);
hipError_t launch_block_norm_bwd(const BlockNorm &p, hipStream_t st);
size_t block_norm_bwd_part_bytes(int64_t rows, int D);

}  // namespace kda
