// Gated delta rule: the gradient's walk over a sequence's chunks, from the last to
// the first. With D the gradient of the state behind a chunk, T the inverse of the
// chunk's system and b its cumulative log2 decays,
//
//     d0 = 2^{b_L - b} k D + scores^T d_o,   du = T^T d0     (of u, before beta)
//     D' = 2^{b_L} D + (scale 2^b q)^T d_o - (beta 2^b k)^T du.
//
// It leaves du of every token, D behind every chunk and, at the end, dh0. Waves,
// state layout and arithmetic are the forward walk's (delta_walk.h); everything
// here reaches the state, so every fp32 operand takes three parts. A chunk's scores are
// needed at its start, so a chunk has two periods: its rows are put to LDS in the first
// of the chunk before, its scores formed in the second.
//
// Bound by the chain of a chunk's steps, as the forward walk: b4 t2048 h32 d128 155 to
// 168 us (600 MB). D leaves tile by tile as it is done: stored whole at a chunk's start it
// takes 173 to 177. With the helpers ahead of the state waves in priority, which the forward
// walk's like, it took 226; with d_o, scores and inverse handed over through single buffers
// in LDS 204; with three chunks of rows and one barrier a chunk, where they fit, packed t4999
// by 64 channels 81 for 83 us and registers spilled at other widths.
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
  static constexpr int LDX = PT + 16, XPL = C * LDX;
  static constexpr unsigned nX = 2u * IN * XPL, rows = 2 * nX;  // q and k
  static constexpr unsigned nT = InverseMove<C>::bytes, nP = NF * 3 * 1024u;  // the inverse and the scores, as pieces
  static constexpr unsigned tab = 4u * (5 * 64 + 4);  // hi, lo, a scale, c, beta a; the chunk's decay
  static constexpr unsigned oB = 2 * (nT + nP + tab);
  // two chunks of everything; one chunk's q and k rows where two do not fit
  static constexpr int NBUF = 2 * rows + oB <= 160 * 1024 ? 2 : 1;
  static constexpr unsigned oT = NBUF * rows, oP = oT + 2 * nT, oTab = oP + 2 * nP, total = oTab + 2 * tab;
  static_assert(total <= 160 * 1024, "LDS");
};

template <typename T, int PT, int NW>
__global__ __launch_bounds__(64 * (NW + 4)) __attribute__((amdgpu_waves_per_eu((NW + 4) / 4, (NW + 4) / 4)))
void delta_rev_kernel(DeltaWalk p) {
  using F = DeltaRevCfg<T, PT, NW>;
  constexpr int C = F::C, NC = F::NC, KS = F::KS, IN = F::IN, QT = F::QT, NB = NC * (NC + 1) / 2;
  using MX = RowsMove<T, F::HT, C, PT>;
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
  auto inverse_at = [&](int cc) { return reinterpret_cast<bf16_t *>(smem + F::oT + ((cc & 1) ? F::nT : 0u)); };
  auto scores_at = [&](int cc) { return reinterpret_cast<bf16_t *>(smem + F::oP + ((cc & 1) ? F::nP : 0u)); };

  if (wave >= NW) {
    // =================================== helper waves ===================================
    const int hw = wave - NW, ht = tid - 64 * NW;
    const int ldx = p.Hk * K;  // row stride, elements
    const uint32_t gx = MX::lane_offset(ht, ldx, K);
    const uint32_t rx = (uint32_t)(MX::RPI * ldx * SZ);
    const int px = MX::lds_offset(ht, F::LDX);
    const int ax = l16 * F::LDX + 8 * grp;  // a row of q or k as an operand
    const T *const xf = reinterpret_cast<const T *>(p.q) + (sr.t0 * p.Hk + hk) * K;
    const T *const zf = reinterpret_cast<const T *>(p.k) + (sr.t0 * p.Hk + hk) * K;
    using MI = InverseMove<C>;
    u32x4_t fx[MX::IT], fz[MX::IT], ft[MI::IT];
    float fg = 0.f, fb = 0.f;
    constexpr int DW = 3;  // the helper that forms the decays: one with fewer blocks of the scores
    auto fetch = [&](int cc) {
      const int L = rows_of(cc);
      const int64_t t = start_of(cc);
      MX::load(fx, xf + t * ldx, ldx, L, K, gx, rx);
      MX::load(fz, zf + t * ldx, ldx, L, K, gx, rx);
      if (hw == DW) {
        const int64_t at = (sr.t0 + t) * p.H + h;
        if (p.g) fg = row_scalar(p.g + at, lane, L, p.H);
        fb = row_scalar(p.beta + at, lane, L, p.H);
      }
      const int64_t slot = delta_slot(p.N, n, sr.t0, sr.t0 + t, C);
      MI::load(ft, p.inv + (slot * p.H + h) * delta_inverse_bytes(C), ht);
    };
    auto put = [&](int cc) {
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
        t[256 + lane] = fb * d.from;
        if (lane == 0) t[320] = d.all;
      }
      MI::template put<true>(ft, inverse_at(cc), hw, lane);
    };
    // transposed scores: lane has row l16 of k, four later rows of q
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
          // frag_index with a tile that is known here only: row tile j, contraction i >> 1
          const int f = C == 32 ? j : (j < 2 ? 2 * j + (i >> 1) : 2 + j);
          put_parts<3>(v, sP + (f * 192 + lane) * 8 + 4 * (i & 1), 512);
        }
      }
    };

    // the halves of pieces beyond the triangles stay zero
    for (int i = ht; i < (int)(2 * (F::nT + F::nP) / 4); i += F::HT) reinterpret_cast<unsigned *>(smem + F::oT)[i] = 0u;
    if (nch > 0) fetch(0);
    __syncthreads();
    if (nch > 0) {
      put(0);
      if (nch > 1) fetch(1);
    }
    __syncthreads();
    if (nch > 0) scores(0);
    __syncthreads();
    for (int cc = 0; cc < nch; ++cc) {  // beside chunk cc of the state waves
      if constexpr (F::NBUF == 1) __syncthreads();
      if (cc + 1 < nch) put(cc + 1);
      if (cc + 2 < nch) fetch(cc + 2);
      __syncthreads();
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
  const int tz = (4 * grp + (l16 >> 2)) * F::LDX + 8 * (l16 & 3);
  const int ldv = p.H * V, wcol = 16 * wave;
  const int64_t vrow = (sr.t0 * p.H + h) * V + col0;
  const T *const oc = reinterpret_cast<const T *>(p.v) + vrow;  // d_o
  float *const uc = p.rows_out + vrow;
  const uint32_t go = qin ? (uint32_t)((4 * grp * ldv + wcol + l16) * SZ) : kOffNone;

  ColumnRows<T, NC> fo;
  auto fetch_o = [&](int cc) {
    fo.load(tile_rsrc(oc + start_of(cc) * ldv, (uint32_t)(((rows_of(cc) - 1) * ldv + ncol) * SZ)), go, ldv);
  };
  auto states_at = [&](int cc) {  // behind chunk cc of the walk
    return p.states + (delta_slot(p.N, n, sr.t0, sr.t0 + start_of(cc), C) * p.H + h) * K * V;
  };
  if (nch > 0) {
    store_state<F::NT>(states_at(0), K, V, grp, q, S);
    fetch_o(0);
  }
  __syncthreads();
  __syncthreads();
  __syncthreads();
  for (int cc = 0; cc < nch; ++cc) {
    const int L = rows_of(cc);
    const int64_t t0 = start_of(cc);
    const bf16_t *const sX = rows_at(cc), *const sZ = sX + F::nX / 2, *const sT = inverse_at(cc), *const sP = scores_at(cc);
    const float *const tab = tab_at(cc);

    // as in the forward walk, what LDS has is asked for before its use and the order pinned
    bf16x8_t kf[NC][IN], sb[2][3];
    auto read_rows = [&](int s) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int pl = 0; pl < IN; ++pl) kf[i][pl] = row_frag(sZ + pl * F::XPL + 16 * i * F::LDX + ax + 32 * s);
    };
    auto split_state = [&](int s) { split_pair<3>(S[2 * s], S[2 * s + 1], sb[s & 1]); };
    read_rows(0);
    // ---- d_o as an operand, and scale 2^b d_o in parts ----
    bf16x8_t w[KS][IN], wc[KS][3];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const f32x4_t o0 = fo.get(2 * s), o1 = fo.get(2 * s + 1);
      const f32x4_t a0 = *reinterpret_cast<const f32x4_t *>(tab + 128 + 32 * s + 4 * grp);
      const f32x4_t a1 = *reinterpret_cast<const f32x4_t *>(tab + 128 + 32 * s + 16 + 4 * grp);
      split_pair<IN>(o0, o1, w[s]);
      split_pair<3>(o0 * a0, o1 * a1, wc[s]);
    }
    if (cc + 1 < nch) fetch_o(cc + 1);
    split_state(0);
    pin();

    // ---- d0 = c (k D) + scores^T d_o ----
    f32x4_t z[NC], u[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) z[i] = zero4();
#pragma unroll
    for (int s = 0; s < F::PS; ++s) {
      mma_cols<NC>(kf, sb[s & 1], z);
      if (s + 1 < F::PS) {
        split_state(s + 1);
        pin();
        read_rows(s + 1);
      }
    }
    InverseTimes<C, true> ti;  // the scores, and then the inverse: both of the same shape
    ti.read(sP, lane, 0);
#pragma unroll
    for (int i = 0; i < NC; ++i) z[i] *= *reinterpret_cast<const f32x4_t *>(tab + 192 + 16 * i + 4 * grp);
    pin();
    // two tiles of the state at a time, products into one accumulator two apart
    bf16x8_t zt[2][KS][IN];  // channels of two state tiles by the chunk's rows
    auto read_channels = [&](const bf16_t *src, int t) {
#pragma unroll
      for (int w2 = 0; w2 < 2; ++w2)
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int pl = 0; pl < IN; ++pl)
            zt[w2][s][pl] = load_frag32_at(src + pl * F::XPL + 32 * s * F::LDX + state_channel(t + w2, 0), F::LDX, tz);
    };
    auto add_channels = [&](const bf16x8_t (&x)[KS][3], int t) {
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = IN - 1; i >= 0; --i)
#pragma unroll
          for (int j = 2; j >= 0; --j)
            if (i + j < 3) {
#pragma unroll
              for (int w2 = 0; w2 < 2; ++w2) S[t + w2] = Mma<bf16_t>::mma(zt[w2][s][i], x[s][j], S[t + w2]);
            }
    };
    const float dec = tab[320];
#pragma unroll
    for (int t = 0; t < F::NT; ++t) S[t] *= dec;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
#pragma unroll
      for (int a = 2; a >= 0; --a)
#pragma unroll
        for (int b = IN - 1; b >= 0; --b)
          if (a + b < 3) {
#pragma unroll
            for (int i = 0; i < NC; ++i)
              if (InverseTimes<C, true>::has(i, s)) z[i] = Mma<bf16_t>::mma(ti.t[i][a], w[s][b], z[i]);
          }
      ti.read(s + 1 < KS ? sP : sT, lane, s + 1 < KS ? s + 1 : 0);
      pin();
    }
    // ---- du = T^T d0; what q and d_o add to the state fills the pauses of the chain ----
    read_channels(sX, 0);
    bf16x8_t wu[KS][3];
#pragma unroll
    for (int s = 0; s < KS; ++s) split_pair<3>(z[2 * s], z[2 * s + 1], wu[s]);
#pragma unroll
    for (int i = 0; i < NC; ++i) u[i] = zero4();
    pin();
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      ti.add(wu[s], u, s);
      if (s + 1 < KS) {
        ti.read(sT, lane, s + 1);
        pin();
      }
    }
#pragma unroll
    for (int t = 0; t < F::NT; t += 2) {
      add_channels(wc, t);
      if (t + 2 < F::NT) read_channels(sX, t + 2);
    }
    read_channels(sZ, 0);
    pin();
#pragma unroll
    for (int s = 0; s < KS; ++s) {  // -beta 2^b du in parts
      const f32x4_t b0 = *reinterpret_cast<const f32x4_t *>(tab + 256 + 32 * s + 4 * grp);
      const f32x4_t b1 = *reinterpret_cast<const f32x4_t *>(tab + 256 + 32 * s + 16 + 4 * grp);
      split_pair<3>(-(u[2 * s] * b0), -(u[2 * s + 1] * b1), wu[s]);
    }
    {
      const auto rs = tile_rsrc(uc + t0 * ldv, (uint32_t)(((L - 1) * ldv + ncol) * 4));
      uint32_t off = qin ? (uint32_t)((4 * grp * ldv + wcol + l16) * 4) : kOffNone;
      asm volatile("" : "+v"(off));  // formed here, not held in registers over the chunks
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(u[i][e]), rs, (int)(off + (16 * i + e) * ldv * 4), 0, 0);
    }
    if constexpr (F::NBUF == 2) __syncthreads();
    // ---- the state's gradient, which leaves for the next chunk as it is done ----
    const auto rs_next = tile_rsrc(cc + 1 < nch ? states_at(cc + 1) : nullptr, cc + 1 < nch ? (uint32_t)(K * V * 4) : 0u);
#pragma unroll
    for (int t = 0; t < F::NT; t += 2) {
      add_channels(wu, t);
      if (t + 2 < F::NT) read_channels(sZ, t + 2);
      if (t > 0) store_tiles(rs_next, K, V, grp, q, t - 2, S[t - 2], S[t - 1]);
    }
    store_tiles(rs_next, K, V, grp, q, F::NT - 2, S[F::NT - 2], S[F::NT - 1]);
    pin();
    if constexpr (F::NBUF == 1) {
      __syncthreads();  // q and k are done with
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
