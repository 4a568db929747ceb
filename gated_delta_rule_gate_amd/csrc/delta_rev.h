// Gated delta rule: the gradient's walk over a sequence's chunks, from the last to
// the first. With D the gradient of the state behind a chunk, T the inverse of the
// chunk's system and b its cumulative log2 decays,
//
//     d0 = 2^{b_L - b} k D + scores^T d_o,   du = T^T d0     (of u, before beta)
//     D' = 2^{b_L} D + (scale 2^b q)^T d_o - (beta 2^b k)^T du.
//
// It leaves du of every token, D behind every chunk and, at the end, dh0. Waves,
// state layout and arithmetic are the forward walk's (delta_walk.h); everything
// here reaches the state, so every fp32 operand takes three parts.
#pragma once

#include "delta_chunk.h"

namespace kda {

namespace {

template <typename T, int PT_, int NW_>
struct DeltaRevCfg {
  static constexpr bool F32 = sizeof(T) == 4;
  static constexpr int PT = PT_, NW = NW_;
  static constexpr int IN = F32 ? 3 : 1, C = delta_chunk(PT, !F32);
  static constexpr int NC = C / 16, KS = C / 32, PS = PT / 32, NT = PT / 16, QT = 16 * NW, NF = delta_frags(C);
  static constexpr int HELPERS = 4, THREADS = 64 * (NW + HELPERS), HT = 64 * HELPERS;
  static constexpr int LDX = PT + 16, LDW = QT + 16, LDP = C + 16;
  static constexpr int XPL = C * LDX, WPL = C * LDW, PPL = C * LDP;
  static constexpr unsigned nX = 2u * IN * XPL, rows = 2 * nX;  // q and k
  static constexpr unsigned nW = 2u * IN * WPL, nT = NF * 3 * 1024u, nP = 2u * 3 * PPL;
  static constexpr unsigned tab = 4u * (6 * 64 + 4);  // hi, lo, a scale, c, beta, beta a; the chunk's decay
  // two chunks' q and k rows where they fit; d_o, the inverse and the scores are used
  // in the first period only and replaced in the second
  static constexpr int NBUF = 2 * rows + nW + nT + nP + 2 * tab <= 160 * 1024 ? 2 : 1;
  static constexpr unsigned oW = NBUF * rows, oT = oW + nW, oP = oT + nT, oTab = oP + nP, total = oTab + 2 * tab;
  static_assert(total <= 160 * 1024, "LDS");
};

template <typename T, int PT, int NW>
__global__ __launch_bounds__(64 * (NW + 4)) __attribute__((amdgpu_waves_per_eu((NW + 4) / 4, (NW + 4) / 4)))
void delta_rev_kernel(DeltaWalk p) {
  using F = DeltaRevCfg<T, PT, NW>;
  constexpr int C = F::C, NC = F::NC, KS = F::KS, IN = F::IN, QT = F::QT, NB = NC * (NC + 1) / 2;
  using MX = RowsMove<T, F::HT, C, PT>;
  using MW = RowsMove<T, F::HT, C, QT>;
  extern __shared__ __align__(16) char smem[];

  // workgroups that read the same q/k rows go to one XCD, next to each other
  const int ncb = (p.V + QT - 1) / QT;
  const int G = p.H / p.Hk, U = G * ncb;
  const int xcd = blockIdx.x & 7, sl = blockIdx.x >> 3;
  const int64_t unit = (int64_t)(sl / U) * 8 + xcd;
  const int member = sl % U;
  const int64_t n64 = unit / p.Hk;
  if (n64 >= p.N) return;
  const int n = (int)n64;
  const int hk = (int)(unit % p.Hk), h = hk * G + member / ncb, cb = member % ncb;
  const SlotRange sr = slot_range(p.cu, n, p.T);

  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int grp = lane >> 4, l16 = lane & 15;
  const int K = p.K, V = p.V, col0 = cb * QT, ncol = min(QT, V - col0);
  const int64_t sbase = ((int64_t)n * p.H + h) * K * V;

  constexpr int SZ = sizeof(T);
  const int nch = (sr.len + C - 1) / C;
  // chunk cc of the walk is chunk nch - 1 - cc of the sequence
  auto start_of = [&](int cc) { return (int64_t)(nch - 1 - cc) * C; };
  auto rows_of = [&](int cc) { return cc == 0 ? sr.len - (nch - 1) * C : C; };
  auto rows_at = [&](int cc) { return reinterpret_cast<bf16_t *>(smem + (F::NBUF == 2 && (cc & 1) ? F::rows : 0u)); };
  auto tab_at = [&](int cc) { return reinterpret_cast<float *>(smem + F::oTab + ((cc & 1) ? F::tab : 0u)); };
  bf16_t *const sW = reinterpret_cast<bf16_t *>(smem + F::oW), *const sT = reinterpret_cast<bf16_t *>(smem + F::oT);
  bf16_t *const sP = reinterpret_cast<bf16_t *>(smem + F::oP);

  if (wave >= NW) {
    // =================================== helper waves ===================================
    __builtin_amdgcn_s_setprio(2);  // what a helper holds up, all state waves wait for
    const int hw = wave - NW, ht = tid - 64 * NW;
    const int ldx = p.Hk * K, ldw = p.H * V;  // row strides, elements
    const uint32_t gx = MX::lane_offset(ht, ldx, K), gw = MW::lane_offset(ht, ldw, ncol);
    const uint32_t rx = (uint32_t)(MX::RPI * ldx * SZ), rw = (uint32_t)(MW::RPI * ldw * SZ);
    const int px = MX::lds_offset(ht, F::LDX), pw = MW::lds_offset(ht, F::LDW);
    const int ax = l16 * F::LDX + 8 * grp;  // a row of q or k as an operand
    const T *const xf = reinterpret_cast<const T *>(p.q) + (sr.t0 * p.Hk + hk) * K;
    const T *const zf = reinterpret_cast<const T *>(p.k) + (sr.t0 * p.Hk + hk) * K;
    const T *const wf = reinterpret_cast<const T *>(p.v) + (sr.t0 * p.H + h) * V + col0;
    using MI = InverseMove<C>;
    u32x4_t fx[MX::IT], fz[MX::IT], fw[MW::IT], ft[MI::IT];
    float fg = 0.f, fb = 0.f;
    constexpr int DW = 3;  // the helper that forms the decays: one with fewer blocks of the scores
    auto fetch_rows = [&](int cc) {
      const int L = rows_of(cc);
      const int64_t t = start_of(cc);
      MX::load(fx, xf + t * ldx, ldx, L, K, gx, rx);
      MX::load(fz, zf + t * ldx, ldx, L, K, gx, rx);
      if (hw == DW) {
        const int64_t at = (sr.t0 + t) * p.H + h;
        if (p.g) fg = row_scalar(p.g + at, lane, L, p.H);
        fb = row_scalar(p.beta + at, lane, L, p.H);
      }
    };
    auto fetch_vt = [&](int cc) {
      const int64_t t = start_of(cc);
      MW::load(fw, wf + t * ldw, ldw, rows_of(cc), ncol, gw, rw);
      const int64_t slot = delta_slot(p.N, n, sr.t0, sr.t0 + t, C);
      MI::load(ft, p.inv + (slot * p.H + h) * delta_inverse_bytes(C), ht);
    };
    auto put_rows = [&](int cc) {
      bf16_t *s = rows_at(cc);
      MX::put(fx, s + px, F::LDX, F::XPL);
      MX::put(fz, s + F::nX / 2 + px, F::LDX, F::XPL);
      if (hw == DW) {
        const RowDecay d = row_decay(fg);
        float *t = tab_at(cc);
        t[lane] = d.hi;
        t[64 + lane] = d.lo;
        t[128 + lane] = d.from * p.scale;
        t[192 + lane] = d.rest;
        t[320 + lane] = fb * d.from;
        if (lane == 0) t[384] = d.all;
      }
    };
    auto put_vt = [&]() {
      MW::put(fw, sW + pw, F::LDW, F::WPL);
      MI::template put<true>(ft, sT, hw, lane);
    };
    // transposed scores: lane has row l16 of k, four later rows of q
    auto scores = [&](int cc) {
      const bf16_t *const sX = rows_at(cc), *const sZ = sX + F::nX / 2;
      const float *const tab = tab_at(cc);
#pragma unroll
      for (int b0 = 0; b0 < NB; b0 += F::HELPERS) {
        const int blk = b0 + hw;
        if (b0 + F::HELPERS <= NB || blk < NB) {
          const int i = blk < 1 ? 0 : (blk < 3 ? 1 : (blk < 6 ? 2 : 3)), j = blk - i * (i + 1) / 2;
          const bf16_t *xs = sX + 16 * i * F::LDX + ax, *zs = sZ + 16 * j * F::LDX + ax;
          f32x4_t acc = zero4();
#pragma unroll
          for (int s = 0; s < F::PS; ++s) {
            bf16x8_t a[IN], bz[IN];
#pragma unroll
            for (int pl = 0; pl < IN; ++pl) {
              a[pl] = row_frag(xs + pl * F::XPL + 32 * s);
              bz[pl] = row_frag(zs + pl * F::XPL + 32 * s);
            }
            acc = mma_parts(a, bz, acc);
          }
          const float hs = tab[16 * j + l16], ls = tab[64 + 16 * j + l16];
          const f32x4_t hr = *reinterpret_cast<const f32x4_t *>(tab + 16 * i + 4 * grp);
          const f32x4_t lr = *reinterpret_cast<const f32x4_t *>(tab + 64 + 16 * i + 4 * grp);
          f32x4_t v;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool keep = i != j || 4 * grp + e >= l16;
            v[e] = keep ? acc[e] * (fast_exp2((hr[e] - hs) + (lr[e] - ls)) * p.scale) : 0.f;
          }
          bf16_t *dst = sP + (16 * j + l16) * F::LDP + 32 * (i >> 1) + 8 * grp + 4 * (i & 1);
          put_parts<3>(v, dst, F::PPL);
        }
      }
    };

    // the blocks of the scores beyond the triangle stay zero
    for (int i = ht; i < (int)(F::nP / 4); i += F::HT) reinterpret_cast<unsigned *>(smem + F::oP)[i] = 0u;
    MI::clear(sT, ht);
    if (nch > 0) {
      fetch_rows(0);
      fetch_vt(0);
      put_rows(0);
    }
    __syncthreads();  // cleared
    if (nch > 0) {
      put_vt();
      if (nch > 1) {
        fetch_rows(1);
        fetch_vt(1);
      }
    }
    __syncthreads();
    if (nch > 0) scores(0);
    __syncthreads();
    for (int cc = 0; cc < nch; ++cc) {  // beside chunk cc of the state waves
      if constexpr (F::NBUF == 2) {
        if (cc + 1 < nch) put_rows(cc + 1);
        if (cc + 2 < nch) fetch_rows(cc + 2);
      }
      __syncthreads();
      if (cc + 1 < nch) put_vt();
      if (cc + 2 < nch) fetch_vt(cc + 2);
      if constexpr (F::NBUF == 1) {
        __syncthreads();
        if (cc + 1 < nch) put_rows(cc + 1);
        if (cc + 2 < nch) fetch_rows(cc + 2);
        __syncthreads();
      }
      if (cc + 1 < nch) scores(cc + 1);
      __syncthreads();
    }
    return;
  }

  // ==================================== state waves ====================================
  const int q = col0 + 16 * wave + l16;  // this lane's state column
  const bool qin = q < V;
  f32x4_t S[F::NT];
  load_state<F::NT>(p.s0 ? p.s0 + sbase : nullptr, K, V, grp, q, S);

  const int ax = l16 * F::LDX + 8 * grp;  // a row of k as an operand
  const int tz = (4 * grp + (l16 >> 2)) * F::LDX + 8 * (l16 & 3), tw = cfrag_lane_off(F::LDW) + 16 * wave;
  const int ap = l16 * F::LDP + 8 * grp;  // a row of the scores
  const int ldy = p.H * V;
  float *const uc = p.rows_out + (sr.t0 * p.H + h) * V + col0;
  const uint32_t gu = qin ? (uint32_t)((4 * grp * ldy + 16 * wave + l16) * 4) : kOffNone;

  __syncthreads();
  __syncthreads();
  __syncthreads();
  for (int cc = 0; cc < nch; ++cc) {
    const int L = rows_of(cc);
    const int64_t t0 = start_of(cc);
    const bf16_t *const sX = rows_at(cc), *const sZ = sX + F::nX / 2;
    const float *const tab = tab_at(cc);
    store_state<F::NT>(p.states + (delta_slot(p.N, n, sr.t0, sr.t0 + t0, C) * p.H + h) * K * V, K, V, grp, q, S);

    // ---- d0 = c (k D) + scores^T d_o ----
    f32x4_t z[NC], u[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) z[i] = zero4();
#pragma unroll
    for (int s = 0; s < F::PS; ++s) {
      bf16x8_t a[NC][IN], sb[3];
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int pl = 0; pl < IN; ++pl) a[i][pl] = row_frag(sZ + pl * F::XPL + 16 * i * F::LDX + ax + 32 * s);
      split_pair<3>(S[2 * s], S[2 * s + 1], sb);
      mma_cols<NC>(a, sb, z);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const f32x4_t c = *reinterpret_cast<const f32x4_t *>(tab + 192 + 16 * i + 4 * grp);
      z[i] *= c;
    }
    bf16x8_t wc[KS][3];  // scale 2^b d_o in parts
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      bf16x8_t w[IN];
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int pl = IN - 1; pl >= 0; --pl) {
        w[pl] = load_frag32_at(sW + pl * F::WPL + 32 * s * F::LDW, F::LDW, tw);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] += static_cast<float>(w[pl][e]);
      }
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if (s >= i / 2) {
          bf16x8_t a[3];
#pragma unroll
          for (int pl = 0; pl < 3; ++pl) a[pl] = row_frag(sP + pl * F::PPL + 16 * i * F::LDP + ap + 32 * s);
          z[i] = mma_parts(a, w, z[i]);
        }
      const f32x4_t a0 = *reinterpret_cast<const f32x4_t *>(tab + 128 + 32 * s + 4 * grp);
      const f32x4_t a1 = *reinterpret_cast<const f32x4_t *>(tab + 128 + 32 * s + 16 + 4 * grp);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] *= a0[e];
        x[e + 4] *= a1[e];
      }
      split_pair<3>(f32x4_t{x[0], x[1], x[2], x[3]}, f32x4_t{x[4], x[5], x[6], x[7]}, wc[s]);
    }
    // ---- du = T^T d0 ----
    bf16x8_t wu[KS][3];
#pragma unroll
    for (int s = 0; s < KS; ++s) split_pair<3>(z[2 * s], z[2 * s + 1], wu[s]);
#pragma unroll
    for (int i = 0; i < NC; ++i) u[i] = zero4();
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      InverseTimes<C, true> ti;
      ti.read(sT, lane, s);
      ti.add(wu[s], u, s);
    }
#pragma unroll
    for (int s = 0; s < KS; ++s) {  // -beta 2^b du in parts
      const f32x4_t b0 = *reinterpret_cast<const f32x4_t *>(tab + 320 + 32 * s + 4 * grp);
      const f32x4_t b1 = *reinterpret_cast<const f32x4_t *>(tab + 320 + 32 * s + 16 + 4 * grp);
      split_pair<3>(-(u[2 * s] * b0), -(u[2 * s + 1] * b1), wu[s]);
    }
    {
      const auto rs = tile_rsrc(uc + t0 * ldy, (uint32_t)(((L - 1) * ldy + ncol) * 4));
      uint32_t off = gu;
      asm volatile("" : "+v"(off));  // formed here, not held in registers over the chunks
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(u[i][e]), rs, (int)(off + (16 * i + e) * ldy * 4), 0, 0);
    }
    __syncthreads();

    // ---- the state's gradient: two tiles at a time, products into one accumulator two apart ----
    const float dec = tab[384];
#pragma unroll
    for (int t = 0; t < F::NT; t += 2) {
      S[t] *= dec;
      S[t + 1] *= dec;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const bf16_t *const src = which ? sZ : sX;
        bf16x8_t a[2][KS][IN];
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int pl = 0; pl < IN; ++pl)
              a[w][s][pl] = load_frag32_at(src + pl * F::XPL + 32 * s * F::LDX + state_channel(t + w, 0), F::LDX, tz);
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int i = IN - 1; i >= 0; --i)
#pragma unroll
            for (int j = 2; j >= 0; --j)
              if (i + j < 3) {
#pragma unroll
                for (int w = 0; w < 2; ++w) S[t + w] = Mma<bf16_t>::mma(a[w][s][i], which ? wu[s][j] : wc[s][j], S[t + w]);
              }
      }
    }
    if constexpr (F::NBUF == 1) {
      __syncthreads();
      __syncthreads();
    }
    __syncthreads();
  }
  if (p.sT && !(nch == 0 && p.sT == p.s0)) store_state<F::NT>(p.sT + sbase, K, V, grp, q, S);
}

template <typename T, int PT, int NW>
hipError_t launch_rev_one(const DeltaWalk &p, hipStream_t st) {
  using F = DeltaRevCfg<T, PT, NW>;
  auto kern = delta_rev_kernel<T, PT, NW>;
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kern), hipFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)F::total);
  if (e != hipSuccess) {
    (void)hipGetLastError();  // do not leave the error for the next launch to report
    return e;
  }
  const int ncb = (p.V + F::QT - 1) / F::QT;
  const int64_t grid = delta_walk_blocks(p, ncb);
  if (grid == 0) return hipSuccess;
  if (grid > most_blocks(F::THREADS)) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(F::THREADS), F::total, st, p);
  return hipGetLastError();
}

template <typename T, int PT>
hipError_t launch_rev_cols(const DeltaWalk &p, hipStream_t st) {
  int ncb;
  const int cols = delta_cols(p, &ncb);
  if constexpr (sizeof(T) == 2) {
    if (cols == 128) return launch_rev_one<T, PT, 8>(p, st);
  }
  return launch_rev_one<T, PT, 4>(p, st);
}

template <typename T>
hipError_t launch_rev_width(const DeltaWalk &p, hipStream_t st) {
  switch (linear_tile(p.K)) {
    case 64: return launch_rev_cols<T, 64>(p, st);
    case 128: return launch_rev_cols<T, 128>(p, st);
    default: return launch_rev_cols<T, 256>(p, st);
  }
}

}  // namespace

}  // namespace kda
