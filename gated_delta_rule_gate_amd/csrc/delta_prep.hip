// Gated delta rule: the inverse of every chunk's triangular system,
//
//     T = (I + A)^{-1},   A_rs = beta_r 2^{b_r - b_s} k_r . k_s  for s < r,
//
// which needs no state and so runs over all chunks at once. One workgroup of four
// waves takes a chunk and a q/k head: k's rows go to LDS, the causal 16 x 16 blocks
// of k k^T stay in accumulators for all value heads that share them. Per head the
// decays and beta make A; the 16 x 16 diagonal blocks are inverted by forward
// substitution, a wave each, and the blocks below, level by level, are
// T_ij = -T_ii sum over m of A_im T_mj in fp32 matrix products. T leaves as the
// walks' operands: three bf16 parts (24 bits) of 16 x 32 pieces.
#include "delta_chunk.h"

namespace kda {

namespace {

template <typename T, int PT>
struct PrepCfg {
  static constexpr bool F32 = sizeof(T) == 4;
  static constexpr int IN = F32 ? 3 : 1, C = delta_chunk(PT, !F32), NC = C / 16, PS = PT / 32, NB = NC * (NC + 1) / 2;
  static constexpr int LDX = PT + 16, XPL = C * LDX, LDA = C + 4;
  static constexpr unsigned oA = 2u * IN * XPL, oT = oA + 4u * C * LDA, oTab = oT + 4u * C * LDA, total = oTab + 4u * 3 * 64;
  static_assert(total <= 160 * 1024, "LDS");
};

// x <- column c of (I + A_ii)^{-1} for one 16 x 16 block, lane (g, c) the rows 4g..4g+3,
// -A_ii at its origin A (fp32, row stride lda). Group g's four rows are solved
// among themselves, broadcast, and taken off the later groups' rows.
__device__ __forceinline__ void unit_inverse16(const float *A0, int lda, float (&x)[4]) {
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

template <typename T, int PT>
__global__ __launch_bounds__(256) void delta_prep_kernel(DeltaPrep p) {
  using F = PrepCfg<T, PT>;
  constexpr int C = F::C, NC = F::NC, NB = F::NB, IN = F::IN, LDA = F::LDA, MB = (NB + 3) / 4;
  using MX = RowsMove<T, 256, C, PT>;
  extern __shared__ __align__(16) char smem[];
  const int hk = (int)(blockIdx.x % p.Hk);
  const int64_t slot = blockIdx.x / p.Hk;
  SegLoc sg;
  if (!locate_chunk(p, slot, C, sg)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), grp = lane >> 4, l16 = lane & 15;
  const int L = (int)(sg.hi - sg.lo), G = p.H / p.Hk;
  bf16_t *const sK = reinterpret_cast<bf16_t *>(smem);
  float *const sA = reinterpret_cast<float *>(smem + F::oA), *const sT = reinterpret_cast<float *>(smem + F::oT);
  float *const tab = reinterpret_cast<float *>(smem + F::oTab);  // hi, lo, beta of every row

  const int64_t ldk = (int64_t)p.Hk * p.K;
  {
    u32x4_t buf[MX::IT];
    MX::load(buf, reinterpret_cast<const T *>(p.k) + (sg.lo * p.Hk + hk) * p.K, ldk, L, p.K,
             MX::lane_offset(tid, ldk, p.K), (uint32_t)(MX::RPI * ldk * sizeof(T)));
    MX::put(buf, sK + MX::lds_offset(tid, F::LDX), F::LDX, F::XPL);
  }
  const int64_t row0 = sg.lo * p.H + hk * G;
  float fg = 0.f, fb = 0.f;
  auto fetch = [&](int j) {  // the last wave forms the rows' decays
    if (p.g) fg = row_scalar(p.g + row0 + j, lane, L, p.H);
    fb = row_scalar(p.beta + row0 + j, lane, L, p.H);
  };
  if (wave == 3) fetch(0);
  __syncthreads();

  f32x4_t gram[MB];
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    const int blk = 4 * m + wave;
    gram[m] = zero4();
    if (blk < NB) {
      const int i = blk < 1 ? 0 : (blk < 3 ? 1 : (blk < 6 ? 2 : 3)), j = blk - i * (i + 1) / 2;
      const bf16_t *r = sK + (16 * i + l16) * F::LDX + 8 * grp, *c = sK + (16 * j + l16) * F::LDX + 8 * grp;
#pragma unroll
      for (int s = 0; s < F::PS; ++s) {
        bf16x8_t a[IN], b[IN];
#pragma unroll
        for (int pl = 0; pl < IN; ++pl) {
          a[pl] = row_frag(r + pl * F::XPL + 32 * s);
          b[pl] = row_frag(c + pl * F::XPL + 32 * s);
        }
        gram[m] = mma_parts(a, b, gram[m]);  // row 4 grp + e of block i, column l16 of block j
      }
    }
  }

  for (int jh = 0; jh < G; ++jh) {
    if (wave == 3) {
      const RowDecay d = row_decay(fg);
      tab[lane] = d.hi;
      tab[64 + lane] = d.lo;
      tab[128 + lane] = fb;
      if (jh + 1 < G) fetch(jh + 1);
    }
    __syncthreads();
#pragma unroll
    for (int m = 0; m < MB; ++m) {
      const int blk = 4 * m + wave;
      if (blk < NB) {
        const int i = blk < 1 ? 0 : (blk < 3 ? 1 : (blk < 6 ? 2 : 3)), j = blk - i * (i + 1) / 2;
        const float hs = tab[16 * j + l16], ls = tab[64 + 16 * j + l16];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 16 * i + 4 * grp + e;
          const float d = fast_exp2((tab[r] - hs) + (tab[64 + r] - ls));
          const bool keep = i != j || 4 * grp + e > l16;
          sA[r * LDA + 16 * j + l16] = keep ? -gram[m][e] * (d * tab[128 + r]) : 0.f;
        }
      }
    }
    __syncthreads();
    if (wave < NC) {
      float x[4];
      unit_inverse16(sA + 16 * wave * (LDA + 1), LDA, x);
#pragma unroll
      for (int e = 0; e < 4; ++e) sT[(16 * wave + 4 * grp + e) * LDA + 16 * wave + l16] = x[e];
    }
    __syncthreads();
#pragma unroll
    for (int d = 1; d < NC; ++d) {
      if (wave < NC - d) {
        const int j = wave, i = wave + d;
        f32x4_t P = zero4();
#pragma unroll
        for (int n = 0; n < d; ++n) {
          const int m = j + n;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            P = __builtin_amdgcn_mfma_f32_16x16x4f32(sA[(16 * i + l16) * LDA + 16 * m + 4 * grp + e],
                                                     sT[(16 * m + 4 * grp + e) * LDA + 16 * j + l16], P, 0, 0, 0);
        }
        f32x4_t R = zero4();
#pragma unroll
        for (int e = 0; e < 4; ++e)
          R = __builtin_amdgcn_mfma_f32_16x16x4f32(sT[(16 * i + l16) * LDA + 16 * i + 4 * grp + e], P[e], R, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) sT[(16 * i + 4 * grp + e) * LDA + 16 * j + l16] = R[e];
      }
      __syncthreads();
    }
    const int64_t at = (slot * p.H + hk * G + jh) * delta_inverse_bytes(C) + lane * 16;
    for (int tr = 0; tr < (p.inv_t ? 2 : 1); ++tr) {
      char *dst = (tr ? p.inv_t : p.inv) + at;
      for (int f = wave; f < delta_frags(C); f += 4) {
        // piece f: rows of tile i, columns of tiles 2 s and 2 s + 1
        const int i = C == 32 ? f : (tr ? (f < 4 ? f >> 1 : f - 2) : (f < 2 ? f : 2 + ((f - 2) >> 1)));
        const int s = C == 32 ? 0 : (tr ? (f < 4 ? f & 1 : 1) : (f < 2 ? 0 : f & 1));
        float x[8];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int c = 2 * s + half;
          const bool in = tr ? c >= i : c <= i;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 16 * i + l16, k = 16 * c + 4 * grp + e;
            x[4 * half + e] = in ? (tr ? sT[k * LDA + r] : sT[r * LDA + k]) : 0.f;
          }
        }
        bf16x8_t part[3];
        split8<3>(x, part);
#pragma unroll
        for (int pl = 0; pl < 3; ++pl) *reinterpret_cast<bf16x8_t *>(dst + (f * 3 + pl) * 1024) = part[pl];
      }
    }
  }
}

template <typename T, int PT>
hipError_t launch_prep(const DeltaPrep &p, hipStream_t st) {
  using F = PrepCfg<T, PT>;
  auto kern = delta_prep_kernel<T, PT>;
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kern), hipFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)F::total);
  if (e != hipSuccess) {
    (void)hipGetLastError();
    return e;
  }
  const int64_t grid = delta_slots((int64_t)p.B * p.T, p.N, F::C) * p.Hk;
  if (grid == 0) return hipSuccess;
  if (grid > most_blocks(256)) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(256), F::total, st, p);
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

// Columns of a workgroup: 128, or 64 where V has no more, and for fp32 inputs, whose
// three parts leave no LDS for more.
int delta_cols(const DeltaWalk &p, int *ncb) {
  const int qt = p.V <= 64 || !p.is_bf16 ? 64 : 128;
  *ncb = (p.V + qt - 1) / qt;
  return qt;
}

bool delta_walk_fits(const DeltaWalk &p) {
  int ncb;
  const int qt = delta_cols(p, &ncb);
  return delta_walk_blocks(p, ncb) <= most_blocks(64 * (qt / 16 + 4));
}

bool delta_prep_fits(const DeltaPrep &p) {
  return delta_slots((int64_t)p.B * p.T, p.N, delta_chunk(linear_tile(p.K), p.is_bf16)) * p.Hk <= most_blocks(256);
}

hipError_t launch_delta_prep(const DeltaPrep &p, hipStream_t st) {
  return p.is_bf16 ? launch_prep_width<bf16_t>(p, st) : launch_prep_width<float>(p, st);
}

}  // namespace kda
