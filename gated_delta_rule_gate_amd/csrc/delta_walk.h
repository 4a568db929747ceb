// Gated delta rule: the forward walk over a sequence's chunks. With the inverse T
// of every chunk's system at hand (delta_prep.hip), S the state at a chunk's start
// and b its cumulative log2 decays,
//
//     r = beta (v - 2^b k S),   u = T r,
//     o = scale (2^b q S + scores u),   S' = 2^{b_L} S + k^T (2^{b_L - b} u).
//
// One workgroup owns a (sequence, head, block of 16 NW columns) and keeps its FP32
// state in matrix accumulators, wave w columns 16w..16w+15 of every 16-row tile
// (linear_walk.h's layout: an accumulator column is, unchanged, an operand of the
// next product). A wave's columns need no other wave's: the whole chain k S, r,
// T r, k^T u runs in its registers, and barriers only hand rows over.
//
// Arithmetic as in linear_walk.h: products on the bf16 matrix cores, an fp32
// operand as a sum of bf16 parts. What reaches the state takes three parts (24
// bits); the scores and what multiplies them in o take OPL.
#pragma once

#include "delta_chunk.h"

namespace kda {

namespace {

enum DeltaMode : int { kDeltaOut = 0, kDeltaKeep = 1 };

template <typename T, int PT_, int NW_, int OPL_, int MODE_>
struct DeltaCfg {
  static constexpr bool F32 = sizeof(T) == 4;
  static constexpr int PT = PT_, NW = NW_, OPL = OPL_, MODE = MODE_;
  static constexpr int IN = F32 ? 3 : 1, C = delta_chunk(PT, !F32);
  static constexpr int NC = C / 16, KS = C / 32, PS = PT / 32, NT = PT / 16, QT = 16 * NW, NF = delta_frags(C);
  static constexpr int HELPERS = 4, THREADS = 64 * (NW + HELPERS), HT = 64 * HELPERS;
  static constexpr int LDX = PT + 16, LDW = QT + 16, LDP = C + 16;
  static constexpr int XPL = C * LDX, WPL = C * LDW, PPL = C * LDP;
  static constexpr bool OUT = MODE == kDeltaOut;
  static constexpr unsigned nX = OUT ? 2u * IN * XPL : 0u, nZ = 2u * IN * XPL, rows = nX + nZ;
  static constexpr unsigned nW = 2u * IN * WPL, nT = NF * 3 * 1024u;
  static constexpr unsigned nP = OUT ? 2u * OPL * PPL : 0u;
  static constexpr unsigned tab = 4u * (6 * 64 + 4);  // hi, lo, a scale, c, beta, beta a; the chunk's decay
  // two chunks' q and k rows and scores where they fit; v and the inverse are used in
  // the first period only and replaced in the second
  static constexpr int NBUF = 2 * rows + nW + nT + 2 * nP + 2 * tab <= 160 * 1024 ? 2 : 1;
  static constexpr int PBUF = NBUF;
  static constexpr bool STAGE = !F32 && OUT && NBUF == 2 && QT <= PT;
  static constexpr unsigned oW = NBUF * rows, oT = oW + nW, oP = oT + nT, oTab = oP + PBUF * nP, total = oTab + 2 * tab;
  static_assert(total <= 160 * 1024, "LDS");
};

template <typename T, int PT, int NW, int OPL, int MODE>
__global__ __launch_bounds__(64 * (NW + 4)) __attribute__((amdgpu_waves_per_eu((NW + 4) / 4, (NW + 4) / 4)))
void delta_walk_kernel(DeltaWalk p) {
  using F = DeltaCfg<T, PT, NW, OPL, MODE>;
  constexpr int C = F::C, NC = F::NC, KS = F::KS, IN = F::IN, QT = F::QT, NB = NC * (NC + 1) / 2;
  constexpr bool OUT = F::OUT;
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
  auto rows_of = [&](int cc) { return min(C, sr.len - cc * C); };
  auto rows_at = [&](int cc) { return reinterpret_cast<bf16_t *>(smem + (F::NBUF == 2 && (cc & 1) ? F::rows : 0u)); };
  auto scores_at = [&](int cc) {
    return reinterpret_cast<bf16_t *>(smem + F::oP + (F::PBUF == 2 && (cc & 1) ? F::nP : 0u));
  };
  auto tab_at = [&](int cc) { return reinterpret_cast<float *>(smem + F::oTab + ((cc & 1) ? F::tab : 0u)); };
  bf16_t *const sV = reinterpret_cast<bf16_t *>(smem + F::oW), *const sT = reinterpret_cast<bf16_t *>(smem + F::oT);

  if (wave >= NW) {
    // =================================== helper waves ===================================
    __builtin_amdgcn_s_setprio(2);  // what a helper holds up, all state waves wait for
    const int hw = wave - NW, ht = tid - 64 * NW;
    const int ldx = p.Hk * K, ldw = p.H * V;  // row strides, elements
    const uint32_t gx = MX::lane_offset(ht, ldx, K), gw = MW::lane_offset(ht, ldw, ncol);
    const uint32_t rx = (uint32_t)(MX::RPI * ldx * SZ), rw = (uint32_t)(MW::RPI * ldw * SZ);
    const int px = MX::lds_offset(ht, F::LDX), pw = MW::lds_offset(ht, F::LDW);
    const int ax = l16 * F::LDX + 8 * grp;  // a row of q or k as an operand
    const T *xf = reinterpret_cast<const T *>(p.q) + (sr.t0 * p.Hk + hk) * K;
    const T *zf = reinterpret_cast<const T *>(p.k) + (sr.t0 * p.Hk + hk) * K;
    const T *wf = reinterpret_cast<const T *>(p.v) + (sr.t0 * p.H + h) * V + col0;
    const float *gf = p.g + sr.t0 * p.H + h, *bf = p.beta + sr.t0 * p.H + h;
    constexpr int TIT = (F::NF * 3 * 64 + F::HT - 1) / F::HT;
    u32x4_t fx[OUT ? MX::IT : 1], fz[MX::IT], fw[MW::IT], ft[TIT];
    float fg = 0.f, fb = 0.f;
    constexpr int DW = 3;  // the helper that forms the decays: one with fewer blocks of the scores
    auto fetch_rows = [&](int cc) {
      const int L = rows_of(cc);
      if constexpr (OUT) MX::load(fx, xf, ldx, L, K, gx, rx);
      MX::load(fz, zf, ldx, L, K, gx, rx);
      if (hw == DW) {
        if (p.g) fg = row_scalar(gf, lane, L, p.H);
        fb = row_scalar(bf, lane, L, p.H);
      }
      xf += (int64_t)C * ldx;
      zf += (int64_t)C * ldx;
      gf += (int64_t)C * p.H;
      bf += (int64_t)C * p.H;
    };
    auto fetch_vt = [&](int cc) {
      MW::load(fw, wf, ldw, rows_of(cc), ncol, gw, rw);
      wf += (int64_t)C * ldw;
      const int64_t slot = delta_slot(p.N, n, sr.t0, sr.t0 + (int64_t)cc * C, C);
      const auto rs = tile_rsrc(p.inv + (slot * p.H + h) * delta_inverse_bytes(C), (uint32_t)delta_inverse_bytes(C));
#pragma unroll
      for (int it = 0; it < TIT; ++it) ft[it] = tile_load16(rs, (uint32_t)((it * F::HT + ht) * 16));
    };
    auto put_rows = [&](int cc) {
      bf16_t *s = rows_at(cc);
      if constexpr (OUT) MX::put(fx, s + px, F::LDX, F::XPL);
      MX::put(fz, s + F::nX / 2 + px, F::LDX, F::XPL);
      if (hw == DW) {
        const RowDecay d = row_decay(fg);
        float *t = tab_at(cc);
        t[lane] = d.hi;
        t[64 + lane] = d.lo;
        t[128 + lane] = d.from * p.scale;
        t[192 + lane] = d.rest;
        t[256 + lane] = fb;
        t[320 + lane] = fb * d.from;
        if (lane == 0) t[384] = d.all;
      }
    };
    auto put_vt = [&]() {
      MW::put(fw, sV + pw, F::LDW, F::WPL);
#pragma unroll
      for (int it = 0; it < TIT; ++it)
        if ((it + 1) * F::HT <= F::NF * 192 || it * F::HT + ht < F::NF * 192)
          *reinterpret_cast<u32x4_t *>(sT + (it * F::HT + ht) * 8) = ft[it];
    };
    // scores of the causal 16 x 16 blocks, decayed and scaled, a wave taking
    // every fourth: lane has row l16 of q, four rows of k
    auto scores = [&](int cc) {
      const bf16_t *const sX = rows_at(cc), *const sZ = sX + F::nX / 2;
      const float *const tab = tab_at(cc);
      bf16_t *const sP = scores_at(cc);
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
            acc = mma_parts(bz, a, acc);
          }
          const float hr = tab[16 * i + l16], lr = tab[64 + 16 * i + l16];
          const f32x4_t hs = *reinterpret_cast<const f32x4_t *>(tab + 16 * j + 4 * grp);
          const f32x4_t ls = *reinterpret_cast<const f32x4_t *>(tab + 64 + 16 * j + 4 * grp);
          f32x4_t v;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool keep = i != j || 4 * grp + e <= l16;
            v[e] = keep ? acc[e] * (fast_exp2((hr - hs[e]) + (lr - ls[e])) * p.scale) : 0.f;
          }
          bf16_t *dst = sP + (16 * i + l16) * F::LDP + 32 * (j >> 1) + 8 * grp + 4 * (j & 1);
#pragma unroll
          for (int pl = 0; pl < OPL; ++pl) {
            const bf16x4_t part = to_bf16x4(v);
            *reinterpret_cast<bf16x4_t *>(dst + pl * F::PPL) = part;
            if (pl + 1 < OPL) v -= to_f32x4(part);
          }
        }
      }
    };
    // o of chunk cc, row by row, from where the state waves left it: a thread
    // reads the places that its own rows of q go to next
    const int ldy = p.H * V;
    const int yr = ht / MX::VPR, yq = (ht % MX::VPR) * MX::EPV;
    char *yc = reinterpret_cast<char *>(p.o) + ((sr.t0 * p.H + h) * V + col0) * 2;
    auto store_rows = [&](int cc) {
      const auto rs = tile_rsrc(yc, (uint32_t)(((rows_of(cc) - 1) * ldy + ncol) * 2));
      yc += (int64_t)C * ldy * 2;
      const bf16_t *s = rows_at(cc) + px;
      u32x4_t v[MX::IT];
#pragma unroll
      for (int it = 0; it < MX::IT; ++it) v[it] = *reinterpret_cast<const u32x4_t *>(s + it * MX::RPI * F::LDX);
#pragma unroll
      for (int it = 0; it < MX::IT; ++it) {
        const int r = yr + it * MX::RPI, c = yq ^ (((r >> 3) & 1) * 8);  // where the state waves put it
        __builtin_amdgcn_raw_buffer_store_b128(v[it], rs, c < ncol && yq < QT ? (r * ldy + c) * 2 : (int)kOffNone, 0, 0);
      }
    };

    if constexpr (OUT) {  // the blocks of the scores beyond the triangle stay zero
      for (int i = ht; i < (int)(F::PBUF * F::nP / 4); i += F::HT) reinterpret_cast<unsigned *>(smem + F::oP)[i] = 0u;
    }
    if (nch > 0) {
      fetch_rows(0);
      fetch_vt(0);
      put_rows(0);
      put_vt();
      if (nch > 1) {
        fetch_rows(1);
        fetch_vt(1);
      }
    }
    __syncthreads();
    if constexpr (OUT) {
      if (nch > 0) scores(0);
      __syncthreads();
    }
    for (int cc = 0; cc < nch; ++cc) {  // beside chunk cc of the state waves
      if (F::STAGE && cc > 0) store_rows(cc - 1);
      if constexpr (F::NBUF == 2) {
        if (cc + 1 < nch) put_rows(cc + 1);
        if (cc + 2 < nch) fetch_rows(cc + 2);
      }
      __syncthreads();
      if (cc + 1 < nch) put_vt();
      if (cc + 2 < nch) fetch_vt(cc + 2);
      if constexpr (F::NBUF == 2) {
        if constexpr (OUT) {
          if (cc + 1 < nch) scores(cc + 1);
        }
      } else {
        __syncthreads();
        if (cc + 1 < nch) put_rows(cc + 1);
        if (cc + 2 < nch) fetch_rows(cc + 2);
        if constexpr (OUT) {
          __syncthreads();
          if (cc + 1 < nch) scores(cc + 1);
        }
      }
      __syncthreads();
    }
    if (F::STAGE && nch > 0) store_rows(nch - 1);
    return;
  }

  // ==================================== state waves ====================================
  const int q = col0 + 16 * wave + l16;  // this lane's state column
  const bool qin = q < V;

  // ---- the state at the start: channels state_channel(t, grp) + e of column q ----
  f32x4_t S[F::NT];
  load_state<F::NT>(p.s0 ? p.s0 + sbase : nullptr, K, V, grp, q, S);

  const int ax = l16 * F::LDX + 8 * grp;  // a row of q or k as an operand
  const int tz = (4 * grp + (l16 >> 2)) * F::LDX + 8 * (l16 & 3), tv = cfrag_lane_off(F::LDW) + 16 * wave;
  const int ap = l16 * F::LDP + 8 * grp;  // a row of the scores
  const int ldy = p.H * V;
  const bool yin = 16 * wave + 4 * grp < ncol;
  const uint32_t gy = yin ? (uint32_t)((l16 * ldy + 16 * wave + 4 * grp) * SZ) : kOffNone;
  char *yc = reinterpret_cast<char *>(p.o) + ((sr.t0 * p.H + h) * V + col0) * SZ;
  float *uc = MODE == kDeltaKeep ? p.rows_out + (sr.t0 * p.H + h) * V + col0 : nullptr;
  const uint32_t gu = qin ? (uint32_t)((4 * grp * ldy + 16 * wave + l16) * 4) : kOffNone;

  __syncthreads();
  if constexpr (OUT) __syncthreads();
  for (int cc = 0; cc < nch; ++cc) {
    const int L = rows_of(cc);
    const bf16_t *const sX = rows_at(cc), *const sZ = sX + F::nX / 2;
    const float *const tab = tab_at(cc);

    if constexpr (MODE == kDeltaKeep) {  // the state at the chunk's start
      const int64_t slot = delta_slot(p.N, n, sr.t0, sr.t0 + (int64_t)cc * C, C);
      store_state<F::NT>(p.states + (slot * p.H + h) * K * V, K, V, grp, q, S);
    }

    // ---- z = k S and y = (q S)^T ----
    f32x4_t y[OUT ? NC : 1], z[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      z[i] = zero4();
      if constexpr (OUT) y[i] = zero4();
    }
#pragma unroll
    for (int s = 0; s < F::PS; ++s) {
      bf16x8_t a[NC][IN], sb[3];
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int pl = 0; pl < IN; ++pl) a[i][pl] = row_frag(sZ + pl * F::XPL + 16 * i * F::LDX + ax + 32 * s);
      split_pair<3>(S[2 * s], S[2 * s + 1], sb);
      mma_cols<NC>(a, sb, z);
      if constexpr (OUT) {
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int pl = 0; pl < IN; ++pl) a[i][pl] = row_frag(sX + pl * F::XPL + 16 * i * F::LDX + ax + 32 * s);
        bf16x8_t so[OPL];
#pragma unroll
        for (int pl = 0; pl < OPL; ++pl) so[pl] = sb[pl];
        mma_rows<NC>(so, a, y);
      }
    }
    // ---- r = beta v - beta a z, u = T r ----
    bf16x8_t rb[KS][3];
    f32x4_t u[NC];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      f32x4_t r[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int i = 2 * s + half;
        f32x4_t v = zero4();
#pragma unroll
        for (int pl = IN - 1; pl >= 0; --pl) v += to_f32x4(load_cfrag_at(sV + pl * F::WPL + 16 * i * F::LDW, tv));
        const f32x4_t be = *reinterpret_cast<const f32x4_t *>(tab + 256 + 16 * i + 4 * grp);
        const f32x4_t ba = *reinterpret_cast<const f32x4_t *>(tab + 320 + 16 * i + 4 * grp);
#pragma unroll
        for (int e = 0; e < 4; ++e) r[half][e] = be[e] * v[e] - ba[e] * z[i][e];
      }
      split_pair<3>(r[0], r[1], rb[s]);
    }
    times_inverse<C, false>(sT, lane, rb, u);
    bf16x8_t ub[KS][OPL], uc3[KS][3];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      if constexpr (OUT) split_pair<OPL>(u[2 * s], u[2 * s + 1], ub[s]);
      const f32x4_t c0 = *reinterpret_cast<const f32x4_t *>(tab + 192 + 32 * s + 4 * grp);
      const f32x4_t c1 = *reinterpret_cast<const f32x4_t *>(tab + 192 + 32 * s + 16 + 4 * grp);
      split_pair<3>(u[2 * s] * c0, u[2 * s + 1] * c1, uc3[s]);
    }
    if constexpr (MODE == kDeltaKeep) {
      const auto rs = tile_rsrc(uc, (uint32_t)(((L - 1) * ldy + ncol) * 4));
      uc += (int64_t)C * ldy;
      uint32_t off = gu;
      asm volatile("" : "+v"(off));  // formed here, not held in registers over the chunks
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(u[i][e]), rs, (int)(off + (16 * i + e) * ldy * 4), 0, 0);
    }
    __syncthreads();

    // ---- y += scores u, out ----
    if constexpr (OUT) {
      const bf16_t *const sP = scores_at(cc);
      const auto rs = tile_rsrc(yc, (uint32_t)(((L - 1) * ldy + ncol) * SZ));
      yc += (int64_t)C * ldy * SZ;
#pragma unroll
      for (int i = 0; i < NC; ++i) y[i] *= tab[128 + 16 * i + l16];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        bf16x8_t a[NC][OPL];
#pragma unroll
        for (int i = 0; i < NC; ++i)
          if (s <= i / 2) {
#pragma unroll
            for (int pl = 0; pl < OPL; ++pl) a[i][pl] = row_frag(sP + pl * F::PPL + 16 * i * F::LDP + ap + 32 * s);
          }
#pragma unroll
        for (int i = 0; i < NC; ++i)
          if (s <= i / 2) y[i] = mma_parts(ub[s], a[i], y[i]);
      }
      if constexpr (F::STAGE) {
        // rows 8..15 of 16 swap 16-byte neighbours: 16 rows then cover all banks
        bf16_t *dst = rows_at(cc) + l16 * F::LDX + ((16 * wave + 4 * grp) ^ (l16 & 8));
#pragma unroll
        for (int i = 0; i < NC; ++i) *reinterpret_cast<bf16x4_t *>(dst + 16 * i * F::LDX) = to_bf16x4(y[i]);
      } else if constexpr (SZ == 4) {
#pragma unroll
        for (int i = 0; i < NC; ++i)
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, y[i]), rs, (int)(gy + 16 * i * ldy * SZ), 0, 0);
      } else {
#pragma unroll
        for (int i = 0; i < NC; ++i)
          __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2_t, to_bf16x4(y[i])), rs,
                                                (int)(gy + 16 * i * ldy * SZ), 0, 0);
      }
    }

    // ---- the state: two tiles at a time, products into one accumulator two apart ----
    const float dec = tab[384];
#pragma unroll
    for (int t = 0; t < F::NT; t += 2) {
      bf16x8_t a[2][KS][IN];
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int pl = 0; pl < IN; ++pl)
            a[w][s][pl] = load_frag32_at(sZ + pl * F::XPL + 32 * s * F::LDX + state_channel(t + w, 0), F::LDX, tz);
      S[t] *= dec;
      S[t + 1] *= dec;
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = IN - 1; i >= 0; --i)
#pragma unroll
          for (int j = 2; j >= 0; --j)
            if (i + j < 3) {
#pragma unroll
              for (int w = 0; w < 2; ++w) S[t + w] = Mma<bf16_t>::mma(a[w][s][i], uc3[s][j], S[t + w]);
            }
    }
    if constexpr (F::NBUF == 1) {
      __syncthreads();
      if constexpr (OUT) __syncthreads();
    }
    __syncthreads();
  }

  if (p.sT && !(nch == 0 && p.sT == p.s0)) store_state<F::NT>(p.sT + sbase, K, V, grp, q, S);
}

template <typename T, int PT, int NW, int OPL, int MODE>
hipError_t launch_delta_one(const DeltaWalk &p, hipStream_t st) {
  using F = DeltaCfg<T, PT, NW, OPL, MODE>;
  auto kern = delta_walk_kernel<T, PT, NW, OPL, MODE>;
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

template <typename T, int PT, int OPL>
hipError_t launch_delta_cols(const DeltaWalk &p, hipStream_t st) {
  int ncb;
  const int cols = delta_cols(p, &ncb);
  if constexpr (sizeof(T) == 2) {
    if (cols == 128)
      return p.o ? launch_delta_one<T, PT, 8, OPL, kDeltaOut>(p, st) : launch_delta_one<T, PT, 8, OPL, kDeltaKeep>(p, st);
  }
  return p.o ? launch_delta_one<T, PT, 4, OPL, kDeltaOut>(p, st) : launch_delta_one<T, PT, 4, OPL, kDeltaKeep>(p, st);
}

template <typename T, int OPL>
hipError_t launch_delta_width(const DeltaWalk &p, hipStream_t st) {
  switch (linear_tile(p.K)) {
    case 64: return launch_delta_cols<T, 64, OPL>(p, st);
    case 128: return launch_delta_cols<T, 128, OPL>(p, st);
    default: return launch_delta_cols<T, 256, OPL>(p, st);
  }
}

}  // namespace

}  // namespace kda
