// What the gated delta rule's kernels share: where a chunk lies, and its decays.
#pragma once

#include "delta_launch.h"
#include "linear_walk.h"

namespace kda {

namespace {

// The sequence's chunk that starts at token lo.
__device__ __forceinline__ int64_t delta_slot(int N, int n, int64_t a, int64_t lo, int chunk) {
  return lo == a ? n : (int64_t)N + lo / chunk - 1;
}

// The chunk with workspace place `slot`: its sequence and rows; false: none.
template <typename P>
__device__ __forceinline__ bool locate_chunk(const P &p, int64_t slot, int chunk, SegLoc &s) {
  LinearWalk w{};
  w.cu = p.cu;
  w.B = p.B;
  w.T = p.T;
  w.N = p.N;
  w.seg = chunk;
  return locate_segment(w, slot, false, s) && s.hi > s.lo;
}

// A row's decays within its chunk. b is summed in fp64 and kept as an integer and a
// fraction, so differences of far larger sums stay exact to fp32; a decay below
// 2^-160 counts as 2^-32768: differences across it give zero, those beyond it stay
// exact.
struct RowDecay {
  float hi, lo;  // b = hi + lo, log2
  float from;    // 2^b
  float rest;    // 2^(b_L - b)
  float all;     // 2^b_L
};
__device__ __forceinline__ RowDecay row_decay(float g) {  // of this lane's row; every lane of the wave calls it
  double b = (double)g * 1.4426950408889634073599;
  if (b <= -160.0) b = -32768.0;
  b = wave_scan(b);
  const double bl = last_lane(b), hi = rint(b);
  return RowDecay{(float)hi, (float)(b - hi), fast_exp2((float)b), fast_exp2((float)(bl - b)), fast_exp2((float)bl)};
}

// One fp32 value a row and head (g, beta) of a chunk's rows: lane's row, zero past them.
__device__ __forceinline__ float row_scalar(const float *at, int lane, int L, int H) {
  const auto rs = tile_rsrc(at, (uint32_t)(((L - 1) * H + 1) * 4));
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, lane < L ? lane * H * 4 : (int)kOffNone, 0, 0));
}

// acc[i] += A_i B over the parts of both that matter, part by part: products
// into one accumulator lie NC apart (mma_rows with the operands' sides exchanged).
template <int NC, int NA, int NB_>
__device__ __forceinline__ void mma_cols(const bf16x8_t (&x)[NC][NA], const bf16x8_t (&s)[NB_], f32x4_t (&y)[NC]) {
  constexpr int M = NA > NB_ ? NA : NB_;
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB_ - 1; j >= 0; --j)
      if (i + j < M) {
#pragma unroll
        for (int r = 0; r < NC; ++r) y[r] = Mma<bf16_t>::mma(x[r][i], s[j], y[r]);
      }
}

// Pieces of a chunk's inverse (rows 16 i, columns 32 s): s <= i / 2, transposed s >= i / 2.
template <int C>
__device__ __forceinline__ constexpr int frag_index(int i, int s, bool tr) {
  if (C == 32) return i;
  return tr ? (i < 2 ? 2 * i + s : 2 + i) : (i < 2 ? i : 2 * i - 2 + s);
}

// acc[i] += inverse rows of tile i times x, for the whole chunk: x[s] the parts of rows 32 s..
template <int C, bool TR>
__device__ __forceinline__ void times_inverse(const bf16_t *sT, int lane, const bf16x8_t (&x)[C / 32][3],
                                              f32x4_t (&acc)[C / 16]) {
  constexpr int NC = C / 16, KS = C / 32;
#pragma unroll
  for (int i = 0; i < NC; ++i) acc[i] = zero4();
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    bf16x8_t t[NC][3];
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (TR ? s >= i / 2 : s <= i / 2) {
#pragma unroll
        for (int pl = 0; pl < 3; ++pl)
          t[i][pl] = row_frag(sT + ((frag_index<C>(i, s, TR) * 3 + pl) * 64 + lane) * 8);
      }
#pragma unroll
    for (int a = 2; a >= 0; --a)
#pragma unroll
      for (int b = 2; b >= 0; --b)
        if (a + b < 3) {
#pragma unroll
          for (int i = 0; i < NC; ++i)
            if (TR ? s >= i / 2 : s <= i / 2) acc[i] = Mma<bf16_t>::mma(t[i][a], x[s][b], acc[i]);
        }
  }
}

// A [K, V] state of which this lane holds channels state_channel(t, grp) + e of column
// q: range-checked accesses (rows past K lie past the end, columns past V at an offset
// past it), their offsets formed where they are used.
template <int NT>
__device__ __forceinline__ void load_state(const float *src, int K, int V, int grp, int q, f32x4_t (&S)[NT]) {
  const auto rs = tile_rsrc(src, src ? (uint32_t)(K * V * 4) : 0u);
  const uint32_t off = q < V ? (uint32_t)((state_channel(0, grp) * V + q) * 4) : kOffNone;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      S[t][e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, (int)(off + (state_channel(t, 0) + e) * V * 4), 0, 0));
}
template <int NT>
__device__ __forceinline__ void store_state(float *dst, int K, int V, int grp, int q, const f32x4_t (&S)[NT]) {
  const auto rs = tile_rsrc(dst, (uint32_t)(K * V * 4));
  uint32_t off = q < V ? (uint32_t)((state_channel(0, grp) * V + q) * 4) : kOffNone;
  asm volatile("" : "+v"(off));
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[t][e]), rs, (int)(off + (state_channel(t, 0) + e) * V * 4), 0, 0);
}

template <int NP>
__device__ __forceinline__ void split_pair(const f32x4_t &a, const f32x4_t &b, bf16x8_t (&part)[NP]) {
  const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  split8<NP>(x, part);
}

}  // namespace

}  // namespace kda
