// Gated delta rule: the gradients of every chunk's inputs, all chunks at once, from
// what the two walks left: h, the state before the chunk, D, the state's gradient
// behind it, and u and du of its tokens. With a_t = 2^{b_t}, c_t = 2^{b_L - b_t},
// m_ts = scale 2^{b_t - b_s} d_o_t . u_s (s <= t), n_ts = 2^{b_t - b_s} du_t . u_s (s < t):
//
//     dq = scale a (d_o h^T) + m k,   W = a (du h^T) + n k          (S'_t du_t)
//     Y  = c (u D^T) + m^T q - (beta n)^T k                         (dS_t u_t)
//     dk = Y - beta W,   dv = beta du,   dbeta = du . v - k . W
//     dg_t = sum over r >= t of the chunk of (q . dq - k . Y - beta k . W)
//            + 2^{b_L} <h, D> + sum over the chunk of k . c (u D^T)
//
// (a decay at t scales <S'_t, dS'_t>, which the last line carries from the chunk's
// end back to t.)
//
// One workgroup of eight waves takes a chunk and head. The contractions over V run
// in slabs of 32 columns, whose rows of h, D, u, du and d_o go to LDS in bf16
// parts (three an fp32 operand) while the next slab's loads are in flight; a wave
// holds 16 channels of the three products for all rows, and its share of m and n.
// Then m and n go to LDS in the slabs' place and meet q and k. 256 channels are
// taken 128 at a time.
#pragma once

#include "delta_chunk.h"

namespace kda {

namespace {

template <typename T, int PT_>
struct GradCfg {
  static constexpr bool F32 = sizeof(T) == 4;
  static constexpr int PT = PT_, IN = F32 ? 3 : 1, C = delta_chunk(PT, !F32), NC = C / 16, KS = C / 32;
  static constexpr int HW = PT < 128 ? PT : 128, NH = PT / HW;  // channels at a time, and how many times
  static constexpr int WT = HW / 16, RS = 8 / WT, RT = NC / RS;  // waves over channel tiles, over row tiles; row tiles of a wave
  static constexpr int NB = NC * (NC + 1) / 2, MB = (NB + 7) / 8;
  static constexpr int LDX = HW + 16, XPL = C * LDX;  // q, k
  static constexpr int LDS_ = 40;                     // 32 columns of a slab and 16 bytes
  static constexpr int SPL = C * LDS_, HPL = HW * LDS_;
  static constexpr int LDM = C + 8, MPL = C * LDM;    // m, n, -beta n
  static constexpr unsigned nX = 2u * IN * XPL;
  static constexpr unsigned oDo = 2 * nX, oDu = oDo + 2u * IN * SPL, oU = oDu + 6u * SPL, oH = oU + 6u * SPL,
                            oD = oH + 6u * HPL, slabs = oD + 6u * HPL;
  static constexpr unsigned oM = 2 * nX, mats = oM + 9u * 2 * MPL;
  static constexpr unsigned oTab = slabs > mats ? slabs : mats;
  // rows' hi, lo, a, c, beta; <h, D> of every wave; sums of the rows' dots
  static constexpr unsigned oRed = oTab + 4u * 5 * 64, total = oRed + 8 * 8 + 4u * 2 * C;
  static_assert(RT >= 1, "row tiles");
  static_assert(total <= 160 * 1024, "LDS");
  // the dots of every wave lie where m and n were
  static_assert(4u * 4 * 8 * C <= 9u * 2 * MPL, "dots");
};

template <typename T, int PT>
__global__ __launch_bounds__(512) void delta_grad_kernel(DeltaGrad p) {
  using F = GradCfg<T, PT>;
  constexpr int C = F::C, NC = F::NC, KS = F::KS, IN = F::IN, RT = F::RT, NB = F::NB, MB = F::MB;
  constexpr int SZ = sizeof(T);
  extern __shared__ __align__(16) char smem[];
  const int h = (int)(blockIdx.x % p.H);
  const int64_t slot = blockIdx.x / p.H;
  SegLoc sg;
  if (!locate_chunk(p, slot, C, sg)) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), grp = lane >> 4, l16 = lane & 15;
  const int L = (int)(sg.hi - sg.lo), hk = h / (p.H / p.Hk), K = p.K, V = p.V;
  const int wt = wave % F::WT, i0 = (wave / F::WT) * RT;  // this wave's channel tile and first row tile

  bf16_t *const sQ = reinterpret_cast<bf16_t *>(smem), *const sK = sQ + F::nX / 2;
  bf16_t *const sDo = reinterpret_cast<bf16_t *>(smem + F::oDo), *const sDu = reinterpret_cast<bf16_t *>(smem + F::oDu);
  bf16_t *const sU = reinterpret_cast<bf16_t *>(smem + F::oU), *const sH = reinterpret_cast<bf16_t *>(smem + F::oH);
  bf16_t *const sD = reinterpret_cast<bf16_t *>(smem + F::oD), *const sM = reinterpret_cast<bf16_t *>(smem + F::oM);
  float *const tab = reinterpret_cast<float *>(smem + F::oTab);
  double *const sHD = reinterpret_cast<double *>(smem + F::oRed);
  float *const sVec = reinterpret_cast<float *>(smem + F::oRed + 64);  // du . v of every row; k . W

  // ---- a slab: rows of u, du, d_o and v by 8 lanes of four columns, of h and D alike ----
  constexpr int HIT = F::HW / 64;
  const int sr = tid >> 3, sc = 4 * (tid & 7);
  const bool row_in = C == 64 || sr < C;
  const int ldv = p.H * V;
  const int64_t vrow = (sg.lo * p.H + h) * (int64_t)V, state = (slot * p.H + h) * (int64_t)K * V;
  const auto rU = tile_rsrc(p.u + vrow, (uint32_t)(((L - 1) * ldv + V) * 4)), rDu = tile_rsrc(p.du + vrow, (uint32_t)(((L - 1) * ldv + V) * 4));
  const auto rV = tile_rsrc(reinterpret_cast<const T *>(p.v) + vrow, (uint32_t)(((L - 1) * ldv + V) * SZ));
  const auto rDo = tile_rsrc(reinterpret_cast<const T *>(p.d_o) + vrow, (uint32_t)(((L - 1) * ldv + V) * SZ));
  const auto rDv = tile_rsrc(reinterpret_cast<T *>(p.dv) + vrow, (uint32_t)(((L - 1) * ldv + V) * SZ));
  const auto rH = tile_rsrc(p.h + state, (uint32_t)(K * V * 4)), rD = tile_rsrc(p.dh + state, (uint32_t)(K * V * 4));
  f32x4_t fu, fdu, fv, fdo, fh[HIT], fd[HIT];
  auto load_t = [&](const __amdgpu_buffer_rsrc_t &r, uint32_t el) {  // four of T
    if constexpr (SZ == 2) {
      const u32x2_t x = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(r, (int)(el == kOffNone ? kOffNone : el * 2), 0, 0));
      return to_f32x4(__builtin_bit_cast(bf16x4_t, x));
    } else {
      return __builtin_bit_cast(f32x4_t, tile_load16(r, el == kOffNone ? kOffNone : el * 4));
    }
  };
  auto fetch = [&](int v0, int ch0) {
    const bool in = v0 + sc < V;
    const uint32_t el = in && row_in ? (uint32_t)(sr * ldv + v0 + sc) : kOffNone;
    fu = __builtin_bit_cast(f32x4_t, tile_load16(rU, el == kOffNone ? kOffNone : el * 4));
    fdu = __builtin_bit_cast(f32x4_t, tile_load16(rDu, el == kOffNone ? kOffNone : el * 4));
    fdo = load_t(rDo, el);
    if (ch0 == 0) fv = load_t(rV, el);
#pragma unroll
    for (int it = 0; it < HIT; ++it) {
      const uint32_t at = in ? (uint32_t)(((ch0 + sr + 64 * it) * V + v0 + sc) * 4) : kOffNone;
      fh[it] = __builtin_bit_cast(f32x4_t, tile_load16(rH, at));
      fd[it] = __builtin_bit_cast(f32x4_t, tile_load16(rD, at));
    }
  };
  auto put3 = [&](const f32x4_t &x, bf16_t *dst, int plane) { put_parts<3>(x, dst, plane); };

  fetch(0, 0);
  if (wave == 0) {
    const int64_t at = sg.lo * p.H + h;
    const RowDecay d = row_decay(p.g ? row_scalar(p.g + at, lane, L, p.H) : 0.f);
    tab[lane] = d.hi;
    tab[64 + lane] = d.lo;
    tab[128 + lane] = d.from;
    tab[192 + lane] = d.rest;
    tab[256 + lane] = row_scalar(p.beta + at, lane, L, p.H);
  }
  __syncthreads();

  double hd = 0.0;       // <h, D>
  float duv = 0.f;       // du . v, this lane's columns of row sr
  f32x4_t M[MB], Nn[MB];  // this wave's blocks of d_o u^T and du u^T: row l16 of tile i, four s of tile j
#pragma unroll
  for (int b = 0; b < MB; ++b) M[b] = Nn[b] = zero4();
  float dot_a[RT], dot_f[RT], dot_w[RT];  // of this wave's channels: the decay's, those through D, k . W
#pragma unroll
  for (int i = 0; i < RT; ++i) dot_a[i] = dot_f[i] = dot_w[i] = 0.f;

  for (int half = 0; half < F::NH; ++half) {
    const int ch0 = half * F::HW;
    {  // q and k rows of these channels
      using MX = RowsMove<T, 512, C, F::HW>;
      const int64_t ldk = (int64_t)p.Hk * K, at = (sg.lo * p.Hk + hk) * K + ch0;
      const int ncol = min(F::HW, K - ch0);
      const uint32_t off = MX::lane_offset(tid, ldk, ncol);
      u32x4_t bq[MX::IT], bk[MX::IT];
      MX::load(bq, reinterpret_cast<const T *>(p.q) + at, ldk, L, ncol, off, (uint32_t)(MX::RPI * ldk * SZ));
      MX::load(bk, reinterpret_cast<const T *>(p.k) + at, ldk, L, ncol, off, (uint32_t)(MX::RPI * ldk * SZ));
      MX::put(bq, sQ + MX::lds_offset(tid, F::LDX), F::LDX, F::XPL);
      MX::put(bk, sK + MX::lds_offset(tid, F::LDX), F::LDX, F::XPL);
    }
    f32x4_t X[RT], W[RT], Y[RT];  // channels 4 grp + e of this wave's tile, row l16 of tile i0 + i
#pragma unroll
    for (int i = 0; i < RT; ++i) X[i] = W[i] = Y[i] = zero4();
    for (int v0 = 0; v0 < V; v0 += 32) {
      // ---- this slab to LDS, the next on its way ----
      if (row_in) {
        bf16_t *const d = sDo + sr * F::LDS_ + sc;
        if constexpr (SZ == 2) *reinterpret_cast<bf16x4_t *>(d) = to_bf16x4(fdo);
        else put3(fdo, d, F::SPL);
        put3(fdu, sDu + sr * F::LDS_ + sc, F::SPL);
        put3(fu, sU + sr * F::LDS_ + sc, F::SPL);
        if (half == 0) {
          duv += (fdu[0] * fv[0] + fdu[1] * fv[1]) + (fdu[2] * fv[2] + fdu[3] * fv[3]);
          const f32x4_t dv = fdu * tab[256 + sr];
          const uint32_t el = v0 + sc < V ? (uint32_t)((sr * ldv + v0 + sc) * SZ) : kOffNone;
          if constexpr (SZ == 2)
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2_t, to_bf16x4(dv)), rDv, (int)el, 0, 0);
          else
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, dv), rDv, (int)el, 0, 0);
        }
      }
      float s = 0.f;
#pragma unroll
      for (int it = 0; it < HIT; ++it) {
        put3(fh[it], sH + (sr + 64 * it) * F::LDS_ + sc, F::HPL);
        put3(fd[it], sD + (sr + 64 * it) * F::LDS_ + sc, F::HPL);
        s += (fh[it][0] * fd[it][0] + fh[it][1] * fd[it][1]) + (fh[it][2] * fd[it][2] + fh[it][3] * fd[it][3]);
      }
      hd += (double)s;
      if (v0 + 32 < V) fetch(v0 + 32, ch0);
      else if (half + 1 < F::NH) fetch(0, ch0 + F::HW);
      __syncthreads();
      // ---- its products ----
      bf16x8_t fH[3], fD[3];
#pragma unroll
      for (int pl = 0; pl < 3; ++pl) {
        fH[pl] = row_frag(sH + pl * F::HPL + (16 * wt + l16) * F::LDS_ + 8 * grp);
        fD[pl] = row_frag(sD + pl * F::HPL + (16 * wt + l16) * F::LDS_ + 8 * grp);
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int at = (16 * (i0 + i) + l16) * F::LDS_ + 8 * grp;
        bf16x8_t a[IN], b[3], c[3];
#pragma unroll
        for (int pl = 0; pl < IN; ++pl) a[pl] = row_frag(sDo + pl * F::SPL + at);
#pragma unroll
        for (int pl = 0; pl < 3; ++pl) {
          b[pl] = row_frag(sDu + pl * F::SPL + at);
          c[pl] = row_frag(sU + pl * F::SPL + at);
        }
        X[i] = mma_parts(fH, a, X[i]);
        W[i] = mma_parts(fH, b, W[i]);
        Y[i] = mma_parts(fD, c, Y[i]);
      }
      if (half == 0) {
#pragma unroll
        for (int b = 0; b < MB; ++b) {
          const int blk = 8 * b + wave;
          if (blk < NB) {
            const int i = blk < 1 ? 0 : (blk < 3 ? 1 : (blk < 6 ? 2 : 3)), j = blk - i * (i + 1) / 2;
            const int at = (16 * i + l16) * F::LDS_ + 8 * grp, us = (16 * j + l16) * F::LDS_ + 8 * grp;
            bf16x8_t x[IN], y[3], u[3];
#pragma unroll
            for (int pl = 0; pl < IN; ++pl) x[pl] = row_frag(sDo + pl * F::SPL + at);
#pragma unroll
            for (int pl = 0; pl < 3; ++pl) {
              y[pl] = row_frag(sDu + pl * F::SPL + at);
              u[pl] = row_frag(sU + pl * F::SPL + us);
            }
            M[b] = mma_parts(u, x, M[b]);
            Nn[b] = mma_parts(u, y, Nn[b]);
          }
        }
      }
      __syncthreads();
    }

    // ---- m, n and -beta n in the slabs' place, zero above the diagonal ----
    for (int i = tid; i < (int)(9 * F::MPL / 2); i += 512) reinterpret_cast<unsigned *>(sM)[i] = 0u;
    __syncthreads();
#pragma unroll
    for (int b = 0; b < MB; ++b) {
      const int blk = 8 * b + wave;
      if (blk < NB) {
        const int i = blk < 1 ? 0 : (blk < 3 ? 1 : (blk < 6 ? 2 : 3)), j = blk - i * (i + 1) / 2;
        const float hr = tab[16 * i + l16], lr = tab[64 + 16 * i + l16], be = tab[256 + 16 * i + l16];
        f32x4_t m, n;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float d = fast_exp2((hr - tab[16 * j + 4 * grp + e]) + (lr - tab[64 + 16 * j + 4 * grp + e]));
          m[e] = i != j || 4 * grp + e <= l16 ? M[b][e] * (d * p.scale) : 0.f;
          n[e] = i != j || 4 * grp + e < l16 ? Nn[b][e] * d : 0.f;
        }
        bf16_t *const dst = sM + (16 * i + l16) * F::LDM + 16 * j + 4 * grp;
        put3(m, dst, F::MPL);
        put3(n, dst + 3 * F::MPL, F::MPL);
        put3(-(n * be), dst + 6 * F::MPL, F::MPL);
      }
    }
    __syncthreads();

    // ---- what goes through the states, scaled; then the chunk's own pairs ----
    const int cw = cfrag_lane_off(F::LDX) + 16 * wt, cm = cfrag_lane_off(F::LDM);
    f32x4_t kv[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int r = 16 * (i0 + i) + l16;
      X[i] *= tab[128 + r] * p.scale;
      W[i] *= tab[128 + r];
      Y[i] *= tab[192 + r];
      kv[i] = zero4();
#pragma unroll
      for (int pl = IN - 1; pl >= 0; --pl)
        kv[i] += to_f32x4(*reinterpret_cast<const bf16x4_t *>(sK + pl * F::XPL + r * F::LDX + 16 * wt + 4 * grp));
      dot_f[i] += rows4_sum((kv[i][0] * Y[i][0] + kv[i][1] * Y[i][1]) + (kv[i][2] * Y[i][2] + kv[i][3] * Y[i][3]));
    }
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      bf16x8_t kf[IN], qf[IN];  // channels by 32 rows
#pragma unroll
      for (int pl = 0; pl < IN; ++pl) {
        kf[pl] = load_frag32_at(sK + pl * F::XPL + 32 * s * F::LDX, F::LDX, cw);
        qf[pl] = load_frag32_at(sQ + pl * F::XPL + 32 * s * F::LDX, F::LDX, cw);
      }
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        const int it = i0 + i;
        if (s <= it / 2) {  // row it takes rows 32 s.. before it
          const bf16_t *const r = sM + (16 * it + l16) * F::LDM + 32 * s + 4 * grp;
          bf16x8_t m[3], n[3];
#pragma unroll
          for (int pl = 0; pl < 3; ++pl) {
            m[pl] = join8(*reinterpret_cast<const bf16x4_t *>(r + pl * F::MPL), *reinterpret_cast<const bf16x4_t *>(r + pl * F::MPL + 16));
            n[pl] = join8(*reinterpret_cast<const bf16x4_t *>(r + (3 + pl) * F::MPL), *reinterpret_cast<const bf16x4_t *>(r + (3 + pl) * F::MPL + 16));
          }
          X[i] = mma_parts(kf, m, X[i]);
          W[i] = mma_parts(kf, n, W[i]);
        }
        if (s >= it / 2) {  // and rows 32 s.. behind it
          const bf16_t *const c = sM + 32 * s * F::LDM + 16 * it;
          bf16x8_t m[3], n[3];
#pragma unroll
          for (int pl = 0; pl < 3; ++pl) {
            m[pl] = load_frag32_at(c + pl * F::MPL, F::LDM, cm);
            n[pl] = load_frag32_at(c + (6 + pl) * F::MPL, F::LDM, cm);
          }
          Y[i] = mma_parts(qf, m, Y[i]);
          Y[i] = mma_parts(kf, n, Y[i]);
        }
      }
    }
    // ---- dots and outputs ----
    const int ch = ch0 + 16 * wt + 4 * grp;
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int r = 16 * (i0 + i) + l16;
      const float be = tab[256 + r];
      f32x4_t qv = zero4();
#pragma unroll
      for (int pl = IN - 1; pl >= 0; --pl)
        qv += to_f32x4(*reinterpret_cast<const bf16x4_t *>(sQ + pl * F::XPL + r * F::LDX + 16 * wt + 4 * grp));
      float a = 0.f, w = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        w += kv[i][e] * W[i][e];
        a += qv[e] * X[i][e] - kv[i][e] * Y[i][e];
      }
      a -= be * w;
      dot_a[i] += rows4_sum(a);
      dot_w[i] += rows4_sum(w);
      const f32x4_t dk = Y[i] - W[i] * be;
      if (r < L && ch < K) {
        if (p.qk_f32) {
          const int64_t at = ((sg.lo + r) * p.H + h) * K + ch;
          *reinterpret_cast<f32x4_t *>(reinterpret_cast<float *>(p.dq) + at) = X[i];
          *reinterpret_cast<f32x4_t *>(reinterpret_cast<float *>(p.dk) + at) = dk;
        } else {
          const int64_t at = ((sg.lo + r) * p.Hk + hk) * K + ch;
          if constexpr (SZ == 2) {
            *reinterpret_cast<bf16x4_t *>(reinterpret_cast<bf16_t *>(p.dq) + at) = to_bf16x4(X[i]);
            *reinterpret_cast<bf16x4_t *>(reinterpret_cast<bf16_t *>(p.dk) + at) = to_bf16x4(dk);
          } else {
            *reinterpret_cast<f32x4_t *>(reinterpret_cast<float *>(p.dq) + at) = X[i];
            *reinterpret_cast<f32x4_t *>(reinterpret_cast<float *>(p.dk) + at) = dk;
          }
        }
      }
    }
    __syncthreads();  // q, k, m and n are done with
  }

  // ---- the rows' sums over waves, and dg from the chunk's end back ----
  float *const dots = reinterpret_cast<float *>(sM);  // [3][channel tiles][C]
#pragma unroll
  for (int i = 0; i < RT; ++i)
    if (grp == 0) {
      const int r = 16 * (i0 + i) + l16;
      dots[wt * C + r] = dot_a[i];
      dots[(8 + wt) * C + r] = dot_f[i];
      dots[(16 + wt) * C + r] = dot_w[i];
    }
#pragma unroll
  for (int off = 1; off < 8; off <<= 1) duv += __shfl_xor(duv, off);
  if (row_in && (tid & 7) == 0) sVec[sr] = duv;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) hd += __shfl_xor(hd, off);
  if (lane == 0) sHD[wave] = hd;
  __syncthreads();
  if (wave == 0) {
    double a = 0.0, f = 0.0;
    float w = 0.f;
    if (lane < C) {
      for (int t = 0; t < F::WT; ++t) {
        a += (double)dots[t * C + lane];
        f += (double)dots[(8 + t) * C + lane];
        w += dots[(16 + t) * C + lane];
      }
    }
    const double upto = wave_scan(a), all = last_lane(upto), through = last_lane(wave_scan(f));
    double whole = 0.0;
    for (int i = 0; i < 8; ++i) whole += sHD[i];
    const double end = whole * (double)fast_exp2(tab[C - 1] + tab[64 + C - 1]) + through;
    if (lane < L) {
      const int64_t at = (sg.lo + lane) * p.H + h;
      if (p.dg) p.dg[at] = (float)((all - upto) + a + end);
      p.dbeta[at] = sVec[lane] - w;
    }
  }
}

template <typename T, int PT>
hipError_t launch_grad(const DeltaGrad &p, hipStream_t st) {
  using F = GradCfg<T, PT>;
  auto kern = delta_grad_kernel<T, PT>;
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kern), hipFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)F::total);
  if (e != hipSuccess) {
    (void)hipGetLastError();
    return e;
  }
  const int64_t grid = delta_slots((int64_t)p.B * p.T, p.N, F::C) * p.H;
  if (grid == 0) return hipSuccess;
  if (grid > most_blocks(512)) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(512), F::total, st, p);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_grad_width(const DeltaGrad &p, hipStream_t st) {
  switch (linear_tile(p.K)) {
    case 64: return launch_grad<T, 64>(p, st);
    case 128: return launch_grad<T, 128>(p, st);
    default: return launch_grad<T, 256>(p, st);
  }
}

}  // namespace

}  // namespace kda
