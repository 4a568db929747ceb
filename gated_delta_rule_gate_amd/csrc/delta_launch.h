// Kernel parameter blocks and launcher declarations of the gated delta rule
// with one decay per head, shared by its host API (delta_api.hip) and its
// kernels.
#pragma once

#include "linear_launch.h"

namespace kda {

// Rows of a chunk: 64; 32 where 64 rows do not fit in LDS beside each other
// (fp32 inputs, three bf16 parts each, and 256 channels).
inline __host__ __device__ constexpr int delta_chunk(int tile, bool is_bf16) { return is_bf16 && tile <= 128 ? 64 : 32; }

// A chunk's place in workspaces that hold something for every chunk: a sequence's
// first chunk has the sequence's number, the others follow by the multiple of the
// chunk size at or before their first token (one sequence has at most one chunk
// after its first that starts in such a window, and no two share one).
inline __host__ __device__ int64_t delta_slots(int64_t rows, int N, int chunk) { return N + rows / chunk; }

// (I + beta M)^{-1} of every chunk in memory: its 16 x 16 blocks on and below the
// diagonal, row by row of blocks, fp32; lane l of a block has row l % 16, columns 4 (l /
// 16).. of it. In LDS the walks hold 16 x 32 pieces in bf16 parts.
inline __host__ __device__ constexpr int delta_frags(int chunk) { return chunk == 64 ? 6 : 2; }
inline __host__ __device__ constexpr int64_t delta_inverse_bytes(int chunk) { return (chunk == 64 ? 10 : 3) * 1024; }

struct DeltaPrep {
  const void *k;
  const float *g, *beta;  // g null: no decay
  const int32_t *cu;
  char *inv;
  float *bound;           // [slot, H] or null: log2 of what a chunk's map enlarges a state by, at most
  bool fold;              // inv times beta's diagonal, from the right
  int B, T, H, K, N, Hk;
  bool is_bf16;
};
bool delta_prep_fits(const DeltaPrep &p);
hipError_t launch_delta_prep(const DeltaPrep &p, hipStream_t st);

struct DeltaWalk {
  const void *q, *k, *v;  // v: d_o in the gradient's walk
  const float *g, *beta;
  const int32_t *cu;
  const char *inv;        // of every chunk; with o, and of a segment: times beta's diagonal
  const float *s0;        // [N, H, K, V] or null
  float *sT;              // [N, H, K, V] or null
  void *o;                // forward, or null: nothing but the state (and what is kept)
  float *rows_out;        // u (the gradient's walk: du, before beta) [rows, H, V], or null
  float *states;          // the state before (the gradient's walk: behind) every chunk, [slot, H, K, V], with rows_out
  int B, T, H, K, V, N, Hk;
  float scale;
  bool is_bf16;
  // Long sequences on few heads, with o: cut into segments of seg tokens (0: whole
  // sequences) that are walked side by side. A segment maps the state that enters it
  // affinely, S -> M S + B: a first pass walks it from zeros (B; a sequence's first from
  // its own start) and, with no rows written, from the identity (M), and leaves both at
  // the boundary behind it; a second chains them; then every segment is walked from its
  // boundary.
  int seg;
  const float *bound;     // of every chunk (delta_prep.hip)
  float *seg_state;       // [boundary, H, K, V]
  float *seg_map;         // [boundary, H, K, K]
  int *seg_zero;          // [boundary, H]: whether the map is zero, and not written
  float *seg_first;       // copies of s0 where sT is s0 itself, [N, H, K, V], or null
};
int delta_cols(const DeltaWalk &p, int *ncb);  // columns of a workgroup and column blocks
// tokens per segment of a walk, or 0 for none; gated: with decays (p.g is not looked at)
int delta_segment(const DeltaWalk &p, bool packed, bool gated);
// Workgroups of a walk of ncb column blocks: a unit of those that read the same q/k
// rows after another, units dealt to the eight XCDs.
inline int64_t delta_walk_blocks(const DeltaWalk &p, int ncb) {
  const int64_t items = p.N + (p.seg ? ((int64_t)p.B * p.T) / p.seg : 0);
  return (items * p.Hk + 7) / 8 * 8 * (p.H / p.Hk) * ncb;
}
// The states at the boundaries from the segments' own, in place: S += M S of the boundary before.
hipError_t launch_delta_chain(const DeltaWalk &p, hipStream_t st);
bool delta_walk_fits(const DeltaWalk &p);
hipError_t launch_delta_walk_bf16(const DeltaWalk &p, hipStream_t st);
hipError_t launch_delta_walk_f32(const DeltaWalk &p, hipStream_t st);
hipError_t launch_delta_rev_bf16(const DeltaWalk &p, hipStream_t st);
hipError_t launch_delta_rev_f32(const DeltaWalk &p, hipStream_t st);
inline hipError_t launch_delta_walk(const DeltaWalk &p, hipStream_t st) {
  return p.is_bf16 ? launch_delta_walk_bf16(p, st) : launch_delta_walk_f32(p, st);
}
inline hipError_t launch_delta_walk_rev(const DeltaWalk &p, hipStream_t st) {
  return p.is_bf16 ? launch_delta_rev_bf16(p, st) : launch_delta_rev_f32(p, st);
}

struct DeltaGrad {
  const void *q, *k, *v, *d_o;
  const float *g, *beta;
  const int32_t *cu;
  const float *u, *du;    // [rows, H, V]
  const float *h, *dh;    // [slot, H, K, V]
  void *dq, *dk;          // [rows, Hk, K], or with shared q/k heads fp32 [rows, H, K]
  bool qk_f32;
  void *dv;
  float *dg, *dbeta;
  bool from_zero;         // no h0
  int B, T, H, K, V, N, Hk;
  float scale;
  bool is_bf16;
};
bool delta_grad_fits(const DeltaGrad &p);
hipError_t launch_delta_grad(const DeltaGrad &p, hipStream_t st);

struct DeltaRecurrent {
  const void *q, *k, *v;
  const float *g, *beta, *h0;
  const int32_t *cu;
  void *o;
  float *ht;
  float scale;
  bool is_bf16;
  int B, T, H, K, V, N, Hk;
};
bool delta_recurrent_fits(const DeltaRecurrent &p);
hipError_t launch_delta_recurrent(const DeltaRecurrent &p, hipStream_t st);

}  // namespace kda
