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

// Part `item` of the batch cut into parts of `part` tokens (linear_segments.h); part 0:
// whole sequences.
template <typename P>
__device__ __forceinline__ bool locate_part(const P &p, int64_t item, int part, SegLoc &s) {
  LinearWalk w{};
  w.cu = p.cu;
  w.B = p.B;
  w.T = p.T;
  w.N = p.N;
  w.seg = part;
  return locate_segment(w, item, false, s);
}
// The chunk with workspace place `slot`: its sequence and rows; false: none.
template <typename P>
__device__ __forceinline__ bool locate_chunk(const P &p, int64_t slot, int chunk, SegLoc &s) {
  return locate_part(p, slot, chunk, s) && s.hi > s.lo;
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

// fp32 values as the sum of NP bf16 parts, largest first. What rounding two values to
// bf16 leaves of them is taken by a dot product of their packed parts with (-1, 0) or
// (0, -1), exact in fp32, in place of an unpack and a subtraction: 7 instructions for
// three parts of two values instead of 11. (An infinity or NaN reaches its neighbour
// in the pair.) The constants are held in scalar registers: as an immediate, (-1, 0)
// was taken as (-1, -1).
__device__ __forceinline__ unsigned minus_low() {
  unsigned m = 0x0000bf80u;
  asm("" : "+s"(m));
  return m;
}
__device__ __forceinline__ unsigned minus_high() {
  unsigned m = 0xbf800000u;
  asm("" : "+s"(m));
  return m;
}
__device__ __forceinline__ float dot2_bf16(unsigned a, unsigned b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, a), __builtin_bit_cast(bf16x2_t, b), c, false);
}
template <int NP, int N>
__device__ __forceinline__ void split_values(float (&x)[2 * N], unsigned (&part)[NP][N]) {
  const unsigned ml = minus_low(), mh = minus_high();
#pragma unroll
  for (int pl = 0; pl < NP; ++pl)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      part[pl][i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
      if (pl + 1 < NP) {
        x[2 * i] = dot2_bf16(part[pl][i], ml, x[2 * i]);
        x[2 * i + 1] = dot2_bf16(part[pl][i], mh, x[2 * i + 1]);
      }
    }
}
// Two accumulator tiles (or any eight values) as a matrix operand.
template <int NP>
__device__ __forceinline__ void split_pair(const f32x4_t &a, const f32x4_t &b, bf16x8_t (&part)[NP]) {
  float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  unsigned u[NP][4];
  split_values<NP, 4>(x, u);
#pragma unroll
  for (int pl = 0; pl < NP; ++pl) part[pl] = __builtin_bit_cast(bf16x8_t, u32x4_t{u[pl][0], u[pl][1], u[pl][2], u[pl][3]});
}
// Four values to LDS (or memory), part by part, `plane` elements apart.
template <int NP>
__device__ __forceinline__ void put_parts(const f32x4_t &v, bf16_t *dst, int plane) {
  float x[4] = {v[0], v[1], v[2], v[3]};
  unsigned u[NP][2];
  split_values<NP, 2>(x, u);
#pragma unroll
  for (int pl = 0; pl < NP; ++pl) *reinterpret_cast<u32x2_t *>(dst + pl * plane) = u32x2_t{u[pl][0], u[pl][1]};
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

// Pieces of a chunk's inverse in LDS, 16 x 32 (rows 16 i, columns 32 s): s <= i / 2,
// transposed s >= i / 2; three parts, a lane's eight values together.
template <int C>
__device__ __forceinline__ constexpr int frag_index(int i, int s, bool tr) {
  if (C == 32) return i;
  return tr ? (i < 2 ? 2 * i + s : 2 + i) : (i < 2 ? i : 2 * i - 2 + s);
}

// A chunk's inverse from memory (its blocks on and below the diagonal, delta_prep.hip)
// to LDS as matrix operands. Four helper waves; a wave takes every fourth block.
template <int C>
struct InverseMove {
  static constexpr int NB = (C / 16) * (C / 16 + 1) / 2, IT = (NB + 3) / 4, PIECES = delta_frags(C);
  static constexpr unsigned bytes = PIECES * 3 * 1024u;
  static __device__ __forceinline__ void load(u32x4_t (&buf)[IT], const char *at, int ht) {
    const auto rs = tile_rsrc(at, (uint32_t)delta_inverse_bytes(C));
#pragma unroll
    for (int it = 0; it < IT; ++it) buf[it] = tile_load16(rs, (uint32_t)((it * 256 + ht) * 16));
  }
  template <bool TR>
  static __device__ __forceinline__ void put(const u32x4_t (&buf)[IT], bf16_t *s, int hw, int lane) {
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      const int b = 4 * it + hw;
      if (4 * it + 4 <= NB || b < NB) {
        const int i = b < 1 ? 0 : (b < 3 ? 1 : (b < 6 ? 2 : 3)), j = b - i * (i + 1) / 2;
        const f32x4_t v = __builtin_bit_cast(f32x4_t, buf[it]);  // row l16 of tile i, columns 4 grp + e of tile j
        if constexpr (!TR) {
          const int f = C == 32 ? i : (i < 2 ? i : 2 * i - 2 + (j >> 1));
          put_parts<3>(v, s + (f * 192 + lane) * 8 + 4 * (j & 1), 512);
        } else {
          // row 4 grp + e of tile j, contraction l16 of tile i
          const int f = C == 32 ? j : (j < 2 ? 2 * j + (i >> 1) : 2 + j);
          const int l16 = lane & 15, grp = lane >> 4;
          float x[4] = {v[0], v[1], v[2], v[3]};
          unsigned u[3][2];
          split_values<3, 2>(x, u);
          bf16_t *const dst = s + (f * 192 + 16 * (l16 >> 2) + 4 * grp) * 8 + 4 * (i & 1) + (l16 & 3);
#pragma unroll
          for (int pl = 0; pl < 3; ++pl)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const unsigned short h = (unsigned short)(u[pl][e >> 1] >> (16 * (e & 1)));
              dst[pl * 512 + 8 * e] = __builtin_bit_cast(bf16_t, h);
            }
        }
      }
    }
  }
};

// A chunk's inverse times x (x[s] the parts of rows 32 s..): the pieces of step s, and
// their products.
template <int C, bool TR>
struct InverseTimes {
  static constexpr int NC = C / 16, KS = C / 32;
  bf16x8_t t[NC][3];
  static __device__ __forceinline__ constexpr bool has(int i, int s) { return TR ? s >= i / 2 : s <= i / 2; }
  __device__ __forceinline__ void read(const bf16_t *sT, int lane, int s) {
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (has(i, s)) {
#pragma unroll
        for (int pl = 0; pl < 3; ++pl) t[i][pl] = row_frag(sT + ((frag_index<C>(i, s, TR) * 3 + pl) * 64 + lane) * 8);
      }
  }
  __device__ __forceinline__ void add(const bf16x8_t (&x)[3], f32x4_t (&acc)[NC], int s) const {
#pragma unroll
    for (int a = 2; a >= 0; --a)
#pragma unroll
      for (int b = 2; b >= 0; --b)
        if (a + b < 3) {
#pragma unroll
          for (int i = 0; i < NC; ++i)
            if (has(i, s)) acc[i] = Mma<bf16_t>::mma(t[i][a], x[b], acc[i]);
        }
  }
};

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
// Two tiles of it.
__device__ __forceinline__ void store_tiles(const __amdgpu_buffer_rsrc_t &rs, int K, int V, int grp, int q, int t, const f32x4_t &a, const f32x4_t &b) {
  uint32_t off = q < V ? (uint32_t)((8 * grp * V + q) * 4) : kOffNone;
  asm volatile("" : "+v"(off));
#pragma unroll
  for (int e = 0; e < 8; ++e)
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(e < 4 ? a[e & 3] : b[e & 3]), rs, (int)(off + (16 * t + e) * V * 4), 0, 0);
}

// A chunk's rows of one [rows, heads, V] tensor in the layout of accumulators: of this
// lane's column, rows 16 i + 4 grp + e; rows past the chunk and columns past V are zero.
// Loaded as they lie, so that the loads stay in flight.
template <typename T, int NC>
struct ColumnRows {
  uint32_t w[NC][4];
  __device__ __forceinline__ void load(const __amdgpu_buffer_rsrc_t &rs, uint32_t off, int ld) {  // off: of row 4 grp, bytes
    asm volatile("" : "+v"(off));
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int at = (int)(off + (16 * i + e) * ld * (int)sizeof(T));
        if constexpr (sizeof(T) == 4) w[i][e] = __builtin_amdgcn_raw_buffer_load_b32(rs, at, 0, 0);
        else w[i][e] = __builtin_amdgcn_raw_buffer_load_b16(rs, at, 0, 0);
      }
  }
  __device__ __forceinline__ f32x4_t get(int i) const {
    f32x4_t r;
#pragma unroll
    for (int e = 0; e < 4; ++e) r[e] = __uint_as_float(sizeof(T) == 4 ? w[i][e] : w[i][e] << 16);
    return r;
  }
};

__device__ __forceinline__ void pin() { __builtin_amdgcn_sched_barrier(0); }

}  // namespace

}  // namespace kda
