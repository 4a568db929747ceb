// Gated delta rule: the inverse of every chunk's triangular system,
//
//     T = (I + A)^{-1},   A_rs = beta_r 2^{b_r - b_s} k_r . k_s  for s < r,
//
// which needs no state and so runs over all chunks at once. A wave takes a chunk and
// a head by itself, with no barrier: rows of k come from memory as operands of the
// causal 16 x 16 blocks of k k^T, and the decays and beta make -A of these accumulators
// in place. The diagonal blocks are inverted by forward substitution, and the blocks
// below, level by level, come from T (I + A) = I as
//
//     T_ij^T = -T_jj^T sum over m = j+1..i of A_mj^T T_im^T
//
// in fp32 matrix products whose operands are accumulators as they stand: of A_mj, of
// T_jj, and of T_im^T. A lane of T_ij^T holds four neighbours of a row of T, which
// leave in 16-byte stores. For the forward T takes beta as factors of its columns.
//
// A wave is a long chain of short steps, which only other waves on its SIMD hide: four of
// them by 114 registers. (Value heads that share a q/k head in one wave, k k^T kept for
// them, were fewer waves with 40 registers spilled: packed t15872, two heads each, 70 us
// for 51.) b4 t4096 h64 d128 takes 98 us, its bytes (k read, T written: 436 MB) 80 us.
#include "delta_chunk.h"

namespace kda {

namespace {

template <typename T, int PT>
struct PrepCfg {
  static constexpr bool F32 = sizeof(T) == 4;
  static constexpr int IN = F32 ? 3 : 1, C = delta_chunk(PT, !F32), NC = C / 16, PS = PT / 32, NB = NC * (NC + 1) / 2;
  static constexpr int LDD = 20;                  // rows of a 16 x 16 block in LDS, 16 bytes past 64
  static constexpr int WAVE = NC * 16 * LDD;      // floats a wave: its diagonal blocks
  static constexpr int TAB = 3 * 64;              // hi, lo, beta of every row
};

// x <- column c of (I + A_ii)^{-1} for one 16 x 16 block, lane (g, c) the rows 4g..4g+3,
// -A_ii at its origin A (fp32, row stride lda). Group g's four rows are solved
// among themselves, broadcast, and taken off the later groups' rows.
__device__ __forceinline__ void unit_inverse16(const float *A0, int lda, f32x4_t &x) {
  const int lane = tid_opaque() & 63, g = lane >> 4, c = lane & 15;
  const float *A = A0 + 4 * g * lda;
  f32x4_t a[4][4];  // rows 4g + e, column quads q
#pragma unroll
  for (int e = 0; e < 4; ++e)
#pragma unroll
    for (int q = 0; q < 4; ++q) a[e][q] = *reinterpret_cast<const f32x4_t *>(A + e * lda + 4 * q);
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = (4 * g + e == c) ? 1.f : 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float z[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      z[e] = x[e];
#pragma unroll
      for (int e2 = 0; e2 < e; ++e2) z[e] += a[e][k][e2] * z[e2];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = g == k ? z[e] : x[e];
    if (k == 3) break;
    float y[4];  // group k's finished rows of this column, in every group
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = k == 0 ? row_bcast<0>(x[e]) : (k == 1 ? row_bcast<1>(x[e]) : row_bcast<2>(x[e]));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float acc = x[e];
#pragma unroll
      for (int e2 = 0; e2 < 4; ++e2) acc += a[e][k][e2] * y[e2];
      x[e] = g > k ? acc : x[e];
    }
  }
}

// acc += P Q of 16 x 16 blocks, P^T and Q in accumulator layout.
__device__ __forceinline__ f32x4_t mma_block(const f32x4_t &pt, const f32x4_t &q, f32x4_t acc) {
#pragma unroll
  for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(pt[e], q[e], acc, 0, 0, 0);
  return acc;
}

template <typename T, int PT>
__global__ __launch_bounds__(256, 4) void delta_prep_kernel(DeltaPrep p, int64_t items) {
  using F = PrepCfg<T, PT>;
  constexpr int C = F::C, NC = F::NC, NB = F::NB, IN = F::IN, LDD = F::LDD;
  __shared__ __align__(16) float sAll[4][F::WAVE + F::TAB];
  const int wave = wave_id(), lane = threadIdx.x & 63, grp = lane >> 4, l16 = lane & 15;
  const int64_t item = (int64_t)blockIdx.x * 4 + wave;
  if (item >= items) return;
  const int h = (int)(item % p.H), hk = h / (p.H / p.Hk);
  const int64_t slot = item / p.H;
  SegLoc sg;
  if (!locate_chunk(p, slot, C, sg)) return;
  const int L = (int)(sg.hi - sg.lo);
  float *const sD = sAll[wave], *const tab = sD + F::WAVE;

  const int64_t row0 = sg.lo * p.H + h;
  const float g = p.g ? row_scalar(p.g + row0, lane, L, p.H) : 0.f, beta = row_scalar(p.beta + row0, lane, L, p.H);

  // ---- k k^T: block (i, j), row 4 grp + e of tile i, column l16 of tile j ----
  f32x4_t A[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) A[b] = zero4();
  {
    const int ldk = p.Hk * p.K;
    const T *const base = reinterpret_cast<const T *>(p.k) + (sg.lo * p.Hk + hk) * p.K;
    const auto rs = tile_rsrc(base, (uint32_t)(((L - 1) * ldk + p.K) * (int)sizeof(T)));
    const uint32_t off = (uint32_t)((l16 * ldk + 8 * grp) * (int)sizeof(T));
#pragma unroll
    for (int s = 0; s < F::PS; ++s) {
      const bool in = 32 * s + 8 * grp < p.K;
      bf16x8_t a[NC][IN];
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const uint32_t at = in ? off + (uint32_t)((16 * i * ldk + 32 * s) * (int)sizeof(T)) : kOffNone;
        if constexpr (F::F32) {
          const f32x4_t lo = __builtin_bit_cast(f32x4_t, tile_load16(rs, at)), hi = __builtin_bit_cast(f32x4_t, tile_load16(rs, at + 16));
          split_pair<3>(lo, hi, a[i]);
        } else {
          a[i][0] = __builtin_bit_cast(bf16x8_t, tile_load16(rs, at));
        }
      }
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j <= i; ++j) A[i * (i + 1) / 2 + j] = mma_parts(a[i], a[j], A[i * (i + 1) / 2 + j]);
    }
  }

  float kk[NC];  // |k|^2, on the diagonals
  if (p.bound) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const f32x4_t &x = A[i * (i + 1) / 2 + i];
      kk[i] = (l16 & 2) ? ((l16 & 1) ? x[3] : x[2]) : ((l16 & 1) ? x[1] : x[0]);
    }
  }
  const RowDecay d = row_decay(g);
  tab[lane] = d.hi;
  tab[64 + lane] = d.lo;
  tab[128 + lane] = beta;
  lds_wave_order();
  // -A: the diagonal blocks to LDS, the others in place
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const f32x4_t hr = *reinterpret_cast<const f32x4_t *>(tab + 16 * i + 4 * grp);
    const f32x4_t lr = *reinterpret_cast<const f32x4_t *>(tab + 64 + 16 * i + 4 * grp);
    const f32x4_t be = *reinterpret_cast<const f32x4_t *>(tab + 128 + 16 * i + 4 * grp);
#pragma unroll
    for (int j = 0; j <= i; ++j) {
      const float hs = tab[16 * j + l16], ls = tab[64 + 16 * j + l16];
      f32x4_t &x = A[i * (i + 1) / 2 + j];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float w = fast_exp2((hr[e] - hs) + (lr[e] - ls)) * be[e];
        x[e] = i != j || 4 * grp + e > l16 ? -x[e] * w : 0.f;
        if (i == j) sD[(16 * i + 4 * grp + e) * LDD + l16] = x[e];
      }
    }
  }
  lds_wave_order();
  // T_ii, and transposed
  f32x4_t D[NC], Tt[NB];
#pragma unroll
  for (int i = 0; i < NC; ++i) unit_inverse16(sD + 16 * i * LDD, LDD, D[i]);
  lds_wave_order();
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) sD[(16 * i + 4 * grp + e) * LDD + l16] = D[i][e];
  lds_wave_order();
#pragma unroll
  for (int i = 0; i < NC; ++i)
    Tt[i * (i + 1) / 2 + i] = *reinterpret_cast<const f32x4_t *>(sD + (16 * i + l16) * LDD + 4 * grp);
#pragma unroll
  for (int n = 1; n < NC; ++n)
#pragma unroll
    for (int j = 0; j + n < NC; ++j) {
      const int i = j + n;
      f32x4_t P = zero4();
#pragma unroll
      for (int m = j + 1; m <= i; ++m) P = mma_block(A[m * (m + 1) / 2 + j], Tt[i * (i + 1) / 2 + m], P);
      Tt[i * (i + 1) / 2 + j] = mma_block(D[j], P, zero4());
    }
  if (p.bound) {
    // a step I - beta k k^T enlarges by |1 - beta |k|^2| if that is above one: by nothing
    // for rows of norm one
    float grow = 0.f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const float f = fabsf(1.f - tab[128 + 16 * i + l16] * kk[i]);
      grow += grp == (l16 >> 2) && !(f <= 1.f) ? fast_log2(f) : 0.f;
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) grow += __shfl_xor(grow, off);
    if (lane == 0) p.bound[slot * p.H + h] = tab[63] + tab[127] + grow;
  }
  // out: row l16 of tile i, columns 4 grp + e of tile j
  char *const dst = p.inv + (slot * p.H + h) * delta_inverse_bytes(C) + lane * 16;
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    f32x4_t be{1.f, 1.f, 1.f, 1.f};
    if (p.fold) be = *reinterpret_cast<const f32x4_t *>(tab + 128 + 16 * j + 4 * grp);
#pragma unroll
    for (int i = j; i < NC; ++i)
      *reinterpret_cast<f32x4_t *>(dst + (i * (i + 1) / 2 + j) * 1024) = Tt[i * (i + 1) / 2 + j] * be;
  }
}

int64_t prep_items(const DeltaPrep &p) {
  return delta_slots((int64_t)p.B * p.T, p.N, delta_chunk(linear_tile(p.K), p.is_bf16)) * p.H;
}

template <typename T, int PT>
hipError_t launch_prep(const DeltaPrep &p, hipStream_t st) {
  const int64_t items = prep_items(p), grid = (items + 3) / 4;
  if (grid == 0) return hipSuccess;
  if (grid > most_blocks(256)) return hipErrorInvalidValue;
  hipLaunchKernelGGL((delta_prep_kernel<T, PT>), dim3((unsigned)grid), dim3(256), 0, st, p, items);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_prep_width(const DeltaPrep &p, hipStream_t st) {
  switch (linear_tile(p.K)) {
    case 64: return launch_prep<T, 64>(p, st);
    case 128: return launch_prep<T, 128>(p, st);
    default: return launch_prep<T, 256>(p, st);
  }
}

}  // namespace

bool delta_prep_fits(const DeltaPrep &p) { return (prep_items(p) + 3) / 4 <= most_blocks(256); }

hipError_t launch_delta_prep(const DeltaPrep &p, hipStream_t st) {
  return p.is_bf16 ? launch_prep_width<bf16_t>(p, st) : launch_prep_width<float>(p, st);
}

}  // namespace kda
