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
// A workgroup of four waves takes one (chunk, head) after another, 64 channels at a
// time, 16 of them a wave. The contractions over V run in slabs of 32 columns: a wave's
// own rows of h and D come from memory as operands, split into three bf16 parts in
// registers; u, du and d_o, which all waves need, go through LDS in parts. The loads of
// the next slab, or of the next item's first, are in flight beside the products of this
// one. Then m and n go to LDS in the slab's place and meet q and k. The steps of an item
// wait on each other, so two workgroups share a compute unit and fill each other's
// pauses: at b4 t2048 h32 d128 389 us, where one workgroup of eight waves and all 128
// channels with two slabs in flight took 473 us, of sixteen 567 us. Bound by bytes first:
// 304 KB a chunk and head, 1.28 GB, and as u, du and d_o are read once for each 64 channels
// 0.34 GB again, together 310 us at the rate of a copy (5.2 TB/s); the matrix cores 85 us.
#pragma once

#include <algorithm>
#include <type_traits>

#include "delta_chunk.h"

namespace kda {

namespace {

template <typename T, int PT_>
struct GradCfg {
  static constexpr bool F32 = sizeof(T) == 4;
  static constexpr int PT = PT_, IN = F32 ? 3 : 1, C = delta_chunk(PT, !F32), NC = C / 16, KS = C / 32;
  static constexpr int HW = 64;  // channels at a time
  static constexpr int NWV = 4, THREADS = 64 * NWV;
  static constexpr int RPT = 8 * C / THREADS;  // rows of a slab of a thread
  static constexpr int NB = NC * (NC + 1) / 2, MB = (NB + NWV - 1) / NWV;
  static constexpr int LDX = HW + 16, XPL = C * LDX;  // q, k
  static constexpr int LDS_ = 48, SPL = C * LDS_;     // 32 columns of a slab and 32 bytes: 16-byte reads of 16 rows hit each bank once
  static constexpr int LDM = C + 8, MPL = C * LDM;    // m, n or -beta n
  static constexpr unsigned nX = 2u * IN * XPL;
  static constexpr unsigned oSlab = 2 * nX, nDo = 2u * IN * SPL, nU = 6u * SPL, slab = nDo + 2 * nU;
  static constexpr unsigned mats = 6u * 2 * MPL;
  static constexpr unsigned oTab = oSlab + (slab > mats ? slab : mats);
  // rows' hi, lo, a, c, beta; <h, D> of every wave; du . v of every row
  static constexpr unsigned oRed = oTab + 4u * 5 * 64, total = oRed + 8 * NWV + 4u * C;
  static_assert(total <= 80 * 1024, "two workgroups a compute unit");
  // the dots of every wave lie where m and n were
  static_assert(4u * 3 * NWV * C <= mats, "dots");
};

template <typename T, int PT>
__global__ __launch_bounds__((GradCfg<T, PT>::THREADS), 2) void delta_grad_kernel(DeltaGrad p, int64_t items) {
  using F = GradCfg<T, PT>;
  constexpr int C = F::C, NC = F::NC, KS = F::KS, IN = F::IN, RPT = F::RPT, NB = F::NB, MB = F::MB, NWV = F::NWV;
  constexpr int SZ = sizeof(T);
  extern __shared__ __align__(16) char smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id(), grp = lane >> 4, l16 = lane & 15;
  const int K = p.K, V = p.V;

  bf16_t *const sQ = reinterpret_cast<bf16_t *>(smem), *const sK = sQ + F::nX / 2;
  bf16_t *const sM = reinterpret_cast<bf16_t *>(smem + F::oSlab);
  float *const tab = reinterpret_cast<float *>(smem + F::oTab);
  double *const sHD = reinterpret_cast<double *>(smem + F::oRed);
  float *const sVec = reinterpret_cast<float *>(smem + F::oRed + 8 * NWV);  // du . v of every row

  // ---- a slab's rows, eight lanes a row, four columns each ----
  const int sr = tid >> 3, sc = 4 * (tid & 7);
  constexpr int RPI = F::THREADS / 8;  // rows apart
  const int ldv = p.H * V;
  // four of T as they lie, so that the loads stay in flight
  typedef typename std::conditional<SZ == 2, bf16x4_t, f32x4_t>::type t4;
  auto load_t = [&](const __amdgpu_buffer_rsrc_t &r, uint32_t el) {
    if constexpr (SZ == 2)
      return __builtin_bit_cast(t4, __builtin_amdgcn_raw_buffer_load_b64(r, (int)(el == kOffNone ? kOffNone : el * 2), 0, 0));
    else
      return __builtin_bit_cast(t4, tile_load16(r, el == kOffNone ? kOffNone : el * 4));
  };
  auto wide = [](const t4 &x) {
    if constexpr (SZ == 2) return to_f32x4(x);
    else return x;
  };
  struct Slab {  // one on its way
    f32x4_t u[RPT], du[RPT], h[2], d[2];
    t4 v[RPT], o[RPT];
  } f;
  struct Item {
    int64_t slot, lo;
    int h, L;
    bool first;  // of its sequence
  };
  auto find = [&](int64_t at, Item &it) {  // the next item at or after `at` (a slot may hold no chunk)
    for (; at < items; at += gridDim.x) {
      SegLoc sg;
      if (!locate_chunk(p, at / p.H, C, sg)) continue;
      it.slot = at / p.H;
      it.h = (int)(at % p.H);
      it.lo = sg.lo;
      it.L = (int)(sg.hi - sg.lo);
      it.first = sg.lo == sg.a;
      break;
    }
    return at;
  };
  auto fetch = [&](const Item &it, int v0, int ch0) {
    const int64_t vrow = (it.lo * p.H + it.h) * (int64_t)V, state = (it.slot * p.H + it.h) * (int64_t)K * V;
    const uint32_t n4 = (uint32_t)(((it.L - 1) * ldv + V) * 4), nt = (uint32_t)(((it.L - 1) * ldv + V) * SZ);
    const auto rU = tile_rsrc(p.u + vrow, n4), rDu = tile_rsrc(p.du + vrow, n4);
    const auto rO = tile_rsrc(reinterpret_cast<const T *>(p.d_o) + vrow, nt), rV = tile_rsrc(reinterpret_cast<const T *>(p.v) + vrow, nt);
#pragma unroll
    for (int x = 0; x < RPT; ++x) {
      const uint32_t el = v0 + sc < V ? (uint32_t)((sr + x * RPI) * ldv + v0 + sc) : kOffNone, el4 = el == kOffNone ? kOffNone : el * 4;
      f.u[x] = __builtin_bit_cast(f32x4_t, tile_load16(rU, el4));
      f.o[x] = load_t(rO, el);
      f.du[x] = __builtin_bit_cast(f32x4_t, tile_load16(rDu, el4));
      if (ch0 == 0) f.v[x] = load_t(rV, el);
    }
    const auto rH = tile_rsrc(p.h + state, (uint32_t)(K * V * 4)), rD = tile_rsrc(p.dh + state, (uint32_t)(K * V * 4));
    const uint32_t at = v0 + 8 * grp < V ? (uint32_t)(((ch0 + 16 * wave + l16) * V + v0 + 8 * grp) * 4) : kOffNone;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      f.h[x] = __builtin_bit_cast(f32x4_t, tile_load16(rH, at + 16 * x));
      f.d[x] = __builtin_bit_cast(f32x4_t, tile_load16(rD, at + 16 * x));
    }
  };
  bf16_t *const sDo = sM, *const sDu = sDo + F::nDo / 2, *const sU = sDu + F::nU / 2;
  auto put3 = [&](const f32x4_t &x, bf16_t *dst, int plane) { put_parts<3>(x, dst, plane); };

  Item it;
  int64_t at = find(blockIdx.x, it);
  if (at < items) {
    fetch(it, 0, 0);
  }
  // g and beta of the next item's rows are on their way beside the work on this one
  auto put_table = [&](float g, float beta) {
    const RowDecay d = row_decay(g);
    tab[lane] = d.hi;
    tab[64 + lane] = d.lo;
    tab[128 + lane] = d.from;
    tab[192 + lane] = d.rest;
    tab[256 + lane] = beta;
  };
  auto scalars = [&](const Item &it, float &g, float &beta) {
    const int64_t g0 = it.lo * p.H + it.h;
    g = p.g ? row_scalar(p.g + g0, lane, it.L, p.H) : 0.f;
    beta = row_scalar(p.beta + g0, lane, it.L, p.H);
  };
  float ng = 0.f, nbeta = 0.f;
  if (wave == 0 && at < items) {
    scalars(it, ng, nbeta);
    put_table(ng, nbeta);
  }
  while (at < items) {
    Item next;
    const int64_t next_at = find(at + gridDim.x, next);
    const int h = it.h, hk = h / (p.H / p.Hk), L = it.L;
    if (wave == 0 && next_at < items) scalars(next, ng, nbeta);
    const auto rDv = tile_rsrc(reinterpret_cast<T *>(p.dv) + (it.lo * p.H + h) * (int64_t)V, (uint32_t)(((L - 1) * ldv + V) * SZ));

    double hd = 0.0;       // <h, D>
    float duv[RPT];        // du . v, this lane's columns of its rows
#pragma unroll
    for (int x = 0; x < RPT; ++x) duv[x] = 0.f;
    f32x4_t M[MB], Nn[MB];  // this wave's blocks of d_o u^T and du u^T: row l16 of tile i, four s of tile j; then of m and n
#pragma unroll
    for (int b = 0; b < MB; ++b) M[b] = Nn[b] = zero4();
    float dot_a[NC], dot_f[NC], dot_w[NC];  // of this wave's channels: the decay's, those through D, k . W
#pragma unroll
    for (int i = 0; i < NC; ++i) dot_a[i] = dot_f[i] = dot_w[i] = 0.f;

    for (int half = 0; half * F::HW < K; ++half) {  // (a part past K would have a negative count of columns)
      const int ch0 = half * F::HW;
      // the lane's offsets are made anew for every item: kept over the loop they would spill
      int own = tid;
      asm volatile("" : "+v"(own));
      const int lane = own & 63, grp = lane >> 4, l16 = lane & 15, sr = own >> 3, sc = 4 * (own & 7);
      {  // q and k rows of these channels
        using MX = RowsMove<T, F::THREADS, C, F::HW>;
        const int64_t ldk = (int64_t)p.Hk * K, k0 = (it.lo * p.Hk + hk) * K + ch0;
        const int ncol = min(F::HW, K - ch0);
        const uint32_t off = MX::lane_offset(tid, ldk, ncol);
        u32x4_t bq[MX::IT], bk[MX::IT];
        MX::load(bq, reinterpret_cast<const T *>(p.q) + k0, ldk, L, ncol, off, (uint32_t)(MX::RPI * ldk * SZ));
        MX::load(bk, reinterpret_cast<const T *>(p.k) + k0, ldk, L, ncol, off, (uint32_t)(MX::RPI * ldk * SZ));
        MX::put(bq, sQ + MX::lds_offset(tid, F::LDX), F::LDX, F::XPL);
        MX::put(bk, sK + MX::lds_offset(tid, F::LDX), F::LDX, F::XPL);
      }
      f32x4_t X[NC], W[NC], Y[NC];  // channels 4 grp + e of this wave's tile, row l16 of tile i
#pragma unroll
      for (int i = 0; i < NC; ++i) X[i] = W[i] = Y[i] = zero4();
      for (int v0 = 0; v0 < V; v0 += 32) {
        __syncthreads();  // the slab before this one is done with; the table is there
        // ---- this slab's shared rows to LDS, the wave's own split ----
#pragma unroll
        for (int x = 0; x < RPT; ++x) {
          const int r = sr + x * RPI;
          if constexpr (SZ == 2) *reinterpret_cast<bf16x4_t *>(sDo + r * F::LDS_ + sc) = f.o[x];
          else put3(f.o[x], sDo + r * F::LDS_ + sc, F::SPL);
          put3(f.u[x], sU + r * F::LDS_ + sc, F::SPL);
          put3(f.du[x], sDu + r * F::LDS_ + sc, F::SPL);
          if (half == 0) {
            const f32x4_t v = wide(f.v[x]), dv = f.du[x] * tab[256 + r];
            duv[x] += (f.du[x][0] * v[0] + f.du[x][1] * v[1]) + (f.du[x][2] * v[2] + f.du[x][3] * v[3]);
            const uint32_t el = v0 + sc < V ? (uint32_t)((r * ldv + v0 + sc) * SZ) : kOffNone;
            if constexpr (SZ == 2)
              __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2_t, to_bf16x4(dv)), rDv, (int)el, 0, 0);
            else
              __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, dv), rDv, (int)el, 0, 0);
          }
        }
        bf16x8_t fH[3], fD[3];
        split_pair<3>(f.h[0], f.h[1], fH);
        split_pair<3>(f.d[0], f.d[1], fD);
        float s = 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x) s += (f.h[x][0] * f.d[x][0] + f.h[x][1] * f.d[x][1]) + (f.h[x][2] * f.d[x][2] + f.h[x][3] * f.d[x][3]);
        hd += (double)s;
        if (v0 + 32 < V) fetch(it, v0 + 32, ch0);
        else if (ch0 + F::HW < K) fetch(it, 0, ch0 + F::HW);
        else if (next_at < items) fetch(next, 0, 0);
        __syncthreads();
        // ---- its products ----
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int r = (16 * i + l16) * F::LDS_ + 8 * grp;
          bf16x8_t a[IN], b[3], c[3];
#pragma unroll
          for (int pl = 0; pl < IN; ++pl) a[pl] = row_frag(sDo + pl * F::SPL + r);
#pragma unroll
          for (int pl = 0; pl < 3; ++pl) {
            b[pl] = row_frag(sDu + pl * F::SPL + r);
            c[pl] = row_frag(sU + pl * F::SPL + r);
          }
          X[i] = mma_parts(fH, a, X[i]);
          W[i] = mma_parts(fH, b, W[i]);
          Y[i] = mma_parts(fD, c, Y[i]);
        }
        if (half == 0) {
#pragma unroll
          for (int b = 0; b < MB; ++b) {
            const int blk = NWV * b + wave;
            if (blk < NB) {
              const int i = blk < 1 ? 0 : (blk < 3 ? 1 : (blk < 6 ? 2 : 3)), j = blk - i * (i + 1) / 2;
              const int r = (16 * i + l16) * F::LDS_ + 8 * grp, us = (16 * j + l16) * F::LDS_ + 8 * grp;
              bf16x8_t x[IN], y[3], u[3];
#pragma unroll
              for (int pl = 0; pl < IN; ++pl) x[pl] = row_frag(sDo + pl * F::SPL + r);
#pragma unroll
              for (int pl = 0; pl < 3; ++pl) {
                y[pl] = row_frag(sDu + pl * F::SPL + r);
                u[pl] = row_frag(sU + pl * F::SPL + us);
              }
              M[b] = mma_parts(u, x, M[b]);
              Nn[b] = mma_parts(u, y, Nn[b]);
            }
          }
        }
      }
      __syncthreads();

      // ---- m and n in the slab's place; of the blocks above the diagonal those that a
      // step of 32 rows takes with a diagonal one are zero ----
      if (wave < KS) {
        bf16_t *const dst = sM + (32 * wave + l16) * F::LDM + 32 * wave + 16 + 4 * grp;
#pragma unroll
        for (int pl = 0; pl < 6; ++pl) *reinterpret_cast<u32x2_t *>(dst + pl * F::MPL) = u32x2_t{0u, 0u};
      }
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        const int blk = NWV * b + wave;
        if (blk < NB) {
          const int i = blk < 1 ? 0 : (blk < 3 ? 1 : (blk < 6 ? 2 : 3)), j = blk - i * (i + 1) / 2;
          if (half == 0) {
            const float hr = tab[16 * i + l16], lr = tab[64 + 16 * i + l16];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float d = fast_exp2((hr - tab[16 * j + 4 * grp + e]) + (lr - tab[64 + 16 * j + 4 * grp + e]));
              M[b][e] = i != j || 4 * grp + e <= l16 ? M[b][e] * (d * p.scale) : 0.f;
              Nn[b][e] = i != j || 4 * grp + e < l16 ? Nn[b][e] * d : 0.f;
            }
          }
          bf16_t *const dst = sM + (16 * i + l16) * F::LDM + 16 * j + 4 * grp;
          put3(M[b], dst, F::MPL);
          put3(Nn[b], dst + 3 * F::MPL, F::MPL);
        }
      }
      __syncthreads();

      // ---- what goes through the states, scaled; then the chunk's own pairs ----
      const int cw = cfrag_lane_off(F::LDX) + 16 * wave, cm = cfrag_lane_off(F::LDM);
      f32x4_t kv[NC];
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int r = 16 * i + l16;
        X[i] *= tab[128 + r] * p.scale;
        W[i] *= tab[128 + r];
        Y[i] *= tab[192 + r];
        kv[i] = zero4();
#pragma unroll
        for (int pl = IN - 1; pl >= 0; --pl)
          kv[i] += to_f32x4(*reinterpret_cast<const bf16x4_t *>(sK + pl * F::XPL + r * F::LDX + 16 * wave + 4 * grp));
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
        for (int i = 0; i < NC; ++i) {
  
          if (s <= i / 2) {  // row tile i takes rows 32 s.. before it
            const bf16_t *const r = sM + (16 * i + l16) * F::LDM + 32 * s + 4 * grp;
            bf16x8_t m[3], n[3];
#pragma unroll
            for (int pl = 0; pl < 3; ++pl) {
              m[pl] = join8(*reinterpret_cast<const bf16x4_t *>(r + pl * F::MPL), *reinterpret_cast<const bf16x4_t *>(r + pl * F::MPL + 16));
              n[pl] = join8(*reinterpret_cast<const bf16x4_t *>(r + (3 + pl) * F::MPL), *reinterpret_cast<const bf16x4_t *>(r + (3 + pl) * F::MPL + 16));
            }
            X[i] = mma_parts(kf, m, X[i]);
            W[i] = mma_parts(kf, n, W[i]);
          }
          if (s >= i / 2) {  // and rows 32 s.. behind it
            const bf16_t *const c = sM + 32 * s * F::LDM + 16 * i;
            bf16x8_t m[3];
#pragma unroll
            for (int pl = 0; pl < 3; ++pl) m[pl] = load_frag32_at(c + pl * F::MPL, F::LDM, cm);
            Y[i] = mma_parts(qf, m, Y[i]);
          }
        }
      }
      __syncthreads();  // m and n are done with: -beta n in m's place
#pragma unroll
      for (int b = 0; b < MB; ++b) {
        const int blk = NWV * b + wave;
        if (blk < NB) {
          const int i = blk < 1 ? 0 : (blk < 3 ? 1 : (blk < 6 ? 2 : 3)), j = blk - i * (i + 1) / 2;
          put3(Nn[b] * -tab[256 + 16 * i + l16], sM + (16 * i + l16) * F::LDM + 16 * j + 4 * grp, F::MPL);
        }
      }
      __syncthreads();
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        bf16x8_t kf[IN];
#pragma unroll
        for (int pl = 0; pl < IN; ++pl) kf[pl] = load_frag32_at(sK + pl * F::XPL + 32 * s * F::LDX, F::LDX, cw);
#pragma unroll
        for (int i = 0; i < NC; ++i)
          if (s >= i / 2) {
            const bf16_t *const c = sM + 32 * s * F::LDM + 16 * i;
            bf16x8_t n[3];
#pragma unroll
            for (int pl = 0; pl < 3; ++pl) n[pl] = load_frag32_at(c + pl * F::MPL, F::LDM, cm);
            Y[i] = mma_parts(kf, n, Y[i]);
          }
      }
      // ---- dots and outputs ----
      const int ch = ch0 + 16 * wave + 4 * grp;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int r = 16 * i + l16;
        const float be = tab[256 + r];
        f32x4_t qv = zero4();
#pragma unroll
        for (int pl = IN - 1; pl >= 0; --pl)
          qv += to_f32x4(*reinterpret_cast<const bf16x4_t *>(sQ + pl * F::XPL + r * F::LDX + 16 * wave + 4 * grp));
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
            const int64_t to = ((it.lo + r) * p.H + h) * K + ch;
            *reinterpret_cast<f32x4_t *>(reinterpret_cast<float *>(p.dq) + to) = X[i];
            *reinterpret_cast<f32x4_t *>(reinterpret_cast<float *>(p.dk) + to) = dk;
          } else {
            const int64_t to = ((it.lo + r) * p.Hk + hk) * K + ch;
            if constexpr (SZ == 2) {
              *reinterpret_cast<bf16x4_t *>(reinterpret_cast<bf16_t *>(p.dq) + to) = to_bf16x4(X[i]);
              *reinterpret_cast<bf16x4_t *>(reinterpret_cast<bf16_t *>(p.dk) + to) = to_bf16x4(dk);
            } else {
              *reinterpret_cast<f32x4_t *>(reinterpret_cast<float *>(p.dq) + to) = X[i];
              *reinterpret_cast<f32x4_t *>(reinterpret_cast<float *>(p.dk) + to) = dk;
            }
          }
        }
      }
      __syncthreads();  // q, k, m and n are done with
    }

    // ---- the rows' sums over waves, and dg from the chunk's end back ----
    float *const dots = reinterpret_cast<float *>(sM);  // [3][waves][C]
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (grp == 0) {
        const int r = 16 * i + l16;
        dots[wave * C + r] = dot_a[i];
        dots[(NWV + wave) * C + r] = dot_f[i];
        dots[(2 * NWV + wave) * C + r] = dot_w[i];
      }
#pragma unroll
    for (int x = 0; x < RPT; ++x) {
#pragma unroll
      for (int off = 1; off < 8; off <<= 1) duv[x] += __shfl_xor(duv[x], off);
      if ((tid & 7) == 0) sVec[sr + x * RPI] = duv[x];
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) hd += __shfl_xor(hd, off);
    if (lane == 0) sHD[wave] = hd;
    __syncthreads();
    if (wave == 0) {
      double a = 0.0, f = 0.0;
      float w = 0.f;
      if (lane < C) {
#pragma unroll
        for (int t = 0; t < NWV; ++t) {
          a += (double)dots[t * C + lane];
          f += (double)dots[(NWV + t) * C + lane];
          w += dots[(2 * NWV + t) * C + lane];
        }
      }
      const double upto = wave_scan(a), all = last_lane(upto), through = last_lane(wave_scan(f));
      double whole = 0.0;
      for (int i = 0; i < NWV; ++i) whole += sHD[i];
      const double end = whole * (double)fast_exp2(tab[C - 1] + tab[64 + C - 1]) + through;
      if (lane < L) {
        const int64_t to = (it.lo + lane) * p.H + h;
        // (the first decay of a sequence that starts from zero scales nothing: no remainder of the sums)
        if (p.dg) p.dg[to] = it.first && p.from_zero && lane == 0 ? 0.f : (float)((all - upto) + a + end);
        p.dbeta[to] = sVec[lane] - w;
      }
      if (next_at < items) put_table(ng, nbeta);
    }
    at = next_at;
    it = next;
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
  const int64_t grid = delta_slots((int64_t)p.B * p.T, p.N, F::C) * p.H;  // items
  if (grid == 0) return hipSuccess;
  // two workgroups a compute unit, by LDS and registers
  hipLaunchKernelGGL(kern, dim3((unsigned)std::min<int64_t>(grid, 2 * device_cus())), dim3(F::THREADS), F::total, st, p, grid);
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
