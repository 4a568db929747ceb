// Gated delta rule: the forward walk over a sequence's chunks. With the inverse T
// of every chunk's system at hand (delta_prep.hip), S the state at a chunk's start
// and b its cumulative log2 decays,
//
//     u = T beta (v - 2^b k S),
//     o = scale (2^b q S + scores u),   S' = 2^{b_L} S + k^T (2^{b_L - b} u).
//
// One workgroup owns a (sequence, head, block of 16 NW columns) and keeps its FP32
// state in matrix accumulators, a wave 16 columns of every 16-row tile
// (linear_walk.h's layout: an accumulator column is, unchanged, an operand of the
// next product). A wave's columns need no other wave's: the whole chain k S, r,
// T r, k^T u runs in its registers, v and o go between memory and registers, and the
// one barrier a chunk hands over q, k, T and scores, which four helper waves bring and
// form a chunk ahead; a chunk's scores meet its u in the next one's time.
//
// Products on the bf16 matrix cores, an fp32 operand as a sum of three bf16 parts (24
// bits), of whose products with another's those of at most 2^-24 are left out. So for o of
// bf16 inputs too: with two parts in the state's copy, the scores and u (16 bits), 0.3% of
// its values were rounded to the neighbour of the nearest bf16 value, in place of 0.01%; it
// costs 4 to 8% of a call (b4 t4096 h64 d128: 40 us).
//
// Bound by the chain of a chunk's steps, which one or two state waves a SIMD hide little of
// (matrix cores busy 46% of the time, vector units 41%): a chunk of 128 x 128 takes 7.1 us
// with every compute unit at work, at a clock that falls under this load, 5.7 us where half
// of them are. b4 t4096 h64 d128: 440 to 460 us (the case's bytes take 215); in two periods
// a chunk with two barriers 497 when one took 405. u and states kept, b4 t2048 h32 d128: 135
// to 140 us for 700 MB.
#pragma once

#include "delta_chunk.h"

namespace kda {

namespace {

// With o; with u and the states kept (the gradient's); of a segment, nothing but the
// state, or the map, left at the boundary behind it.
enum DeltaMode : int { kDeltaOut = 0, kDeltaKeep = 1, kDeltaState = 2 };

template <typename T, int PT_, int NW_, int MODE_>
struct DeltaCfg {
  static constexpr bool F32 = sizeof(T) == 4;
  static constexpr int PT = PT_, NW = NW_, MODE = MODE_;
  static constexpr int IN = F32 ? 3 : 1, C = delta_chunk(PT, !F32);
  static constexpr int NC = C / 16, KS = C / 32, PS = PT / 32, NT = PT / 16, QT = 16 * NW, NF = delta_frags(C);
  static constexpr int HELPERS = 4, THREADS = 64 * (NW + HELPERS), HT = 64 * HELPERS;
  static constexpr int LDX = PT + 16, XPL = C * LDX;
  static constexpr bool OUT = MODE == kDeltaOut;
  static constexpr unsigned nX = OUT ? 2u * IN * XPL : 0u, nZ = 2u * IN * XPL, rows = nX + nZ;
  static constexpr unsigned nT = InverseMove<C>::bytes;
  static constexpr unsigned nP = OUT ? NF * 3 * 1024u : 0u;  // scores, as pieces like the inverse's
  static constexpr unsigned tab = 4u * (6 * 64 + 4);  // hi, lo, a scale, c, a (with u kept: beta a, beta); the chunk's decay
  static constexpr unsigned oB = 2 * (nT + nP + tab);
  // two chunks of everything; one chunk's q and k rows where two do not fit
  static constexpr int NBUF = 2 * rows + oB <= 160 * 1024 ? 2 : 1;
  static constexpr unsigned oT = NBUF * rows, oP = oT + 2 * nT, oTab = oP + 2 * nP, total = oTab + 2 * tab;
  static_assert(total <= 160 * 1024, "LDS");
};

// One workgroup a compute unit, with all its registers; but a state pass by 64 columns,
// which needs fewer, may share one (fp32, 2 x 1000 tokens, 8 heads of 72 x 40: 24 us for 31).
template <typename T, int PT, int NW, int MODE>
__global__ __launch_bounds__(64 * (NW + 4)) __attribute__((amdgpu_waves_per_eu((NW + 7) / 4, MODE == kDeltaState && NW == 4 ? 4 : (NW + 7) / 4)))
void delta_walk_kernel(DeltaWalk p) {
  using F = DeltaCfg<T, PT, NW, MODE>;
  constexpr int C = F::C, NC = F::NC, KS = F::KS, IN = F::IN, QT = F::QT, NB = NC * (NC + 1) / 2;
  constexpr bool OUT = F::OUT, KEEP = MODE == kDeltaKeep;
  using MX = RowsMove<T, F::HT, C, PT>;
  extern __shared__ __align__(16) char smem[];

  // Workgroups that read the same q/k rows go to one XCD, next to each other; whole
  // segments come before the sequences' first, which may be short. Of a state pass, maps
  // come before all states, and a head's segments are dealt over the XCDs: most maps are
  // not walked and most states only from a segment's last chunks on, while those of a head
  // that decays slowly would else start behind a round of others, or on one XCD.
  const int G = p.H / p.Hk, nvb = (p.V + QT - 1) / QT;
  const int seg = KEEP ? 0 : p.seg;
  const int64_t n_items = p.N + (seg ? ((int64_t)p.B * p.T) / seg : 0);
  const int64_t maps = MODE == kDeltaState ? (n_items * p.Hk + 7) / 8 * 8 * G * ((p.K + QT - 1) / QT) : 0;  // workgroups
  const bool map = MODE == kDeltaState && blockIdx.x < maps;  // columns of M, not of B
  const int64_t block = map ? blockIdx.x : blockIdx.x - maps;
  const int ncb = map ? (p.K + QT - 1) / QT : nvb, U = G * ncb;
  const int64_t unit = (block >> 3) / U * 8 + (block & 7);
  const int member = (int)((block >> 3) % U);
  const int64_t item = n_items - 1 - unit / p.Hk;
  const int hk = (int)((MODE == kDeltaState ? unit + item : unit) % p.Hk), h = hk * G + member / ncb, cb = member % ncb;
  SegLoc sg;
  if (item < 0 || !locate_part(p, item, seg, sg)) return;
  if (MODE == kDeltaState && sg.out < 0) return;  // nothing follows the last segment
  if (map && sg.in < 0) return;                   // a first segment starts from its own state
  const int n = sg.n;
  int skip = 0;
  if constexpr (MODE == kDeltaState) {
    // What lies before a chunk from which on the decays leave nothing (under 2^-160, the
    // chunks' bounds summed) does not reach the segment's end: its state is walked from
    // there on, and its map is zero. So it is for most heads of a gated model over a few
    // thousand tokens.
    const int ln = threadIdx.x & 63, chunks = (int)(sg.hi - sg.lo) / C;
    float behind = 0.f;
    for (int base = (chunks - 1) / 64 * 64; base >= 0 && skip == 0; base -= 64) {
      const int c = base + ln;
      float b = c < chunks ? p.bound[delta_slot(p.N, n, sg.a, sg.lo + (int64_t)c * C, C) * p.H + h] : 0.f;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {  // of this chunk and those behind it
        const float x = __shfl_down(b, off);
        b += ln + off < 64 ? x : 0.f;
      }
      b += behind;
      const unsigned long long none = __ballot(c < chunks && b <= -160.f);
      if (none) skip = base + 64 - __clzll(none);  // one past the last such chunk's place
      behind = __shfl(b, 0);
    }
    if (map) {
      if (cb == 0 && threadIdx.x == 0) p.seg_zero[(int64_t)sg.out * p.H + h] = skip > 0;
      if (skip) return;
    } else if (skip) {
      sg.lo += (int64_t)(skip - 1) * C;
    }
  }
  const int len = (int)(sg.hi - sg.lo);

  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int grp = lane >> 4, l16 = lane & 15;
  const int K = p.K, V = map ? p.K : p.V, col0 = cb * QT, ncol = min(QT, V - col0);  // V: the state's columns
  const int64_t sbase = ((int64_t)n * p.H + h) * K * V;

  constexpr int SZ = sizeof(T);
  const int nch = (len + C - 1) / C;
  auto rows_of = [&](int cc) { return min(C, len - cc * C); };
  auto rows_at = [&](int cc) { return reinterpret_cast<bf16_t *>(smem + (F::NBUF == 2 && (cc & 1) ? F::rows : 0u)); };
  auto inverse_at = [&](int cc) { return reinterpret_cast<bf16_t *>(smem + F::oT + ((cc & 1) ? F::nT : 0u)); };
  auto scores_at = [&](int cc) { return reinterpret_cast<bf16_t *>(smem + F::oP + ((cc & 1) ? F::nP : 0u)); };
  auto tab_at = [&](int cc) { return reinterpret_cast<float *>(smem + F::oTab + ((cc & 1) ? F::tab : 0u)); };

  if (wave >= NW) {
    // =================================== helper waves ===================================
    // What a helper holds up, all state waves wait for. With two state waves to a helper on
    // a SIMD (b4 t4096 h64) a call takes 543 us for 546; with one each the state wave is the
    // later one (b4 t2048 h32, u and states kept: 140 us without, 150 with).
    if constexpr (NW == 8) __builtin_amdgcn_s_setprio(2);
    const int hw = wave - NW, ht = tid - 64 * NW;
    const int ldx = p.Hk * K;  // row stride, elements
    const uint32_t gx = MX::lane_offset(ht, ldx, K);
    const uint32_t rx = (uint32_t)(MX::RPI * ldx * SZ);
    const int px = MX::lds_offset(ht, F::LDX);
    const int ax = l16 * F::LDX + 8 * grp;  // a row of q or k as an operand
    const T *xf = reinterpret_cast<const T *>(p.q) + (sg.lo * p.Hk + hk) * K;
    const T *zf = reinterpret_cast<const T *>(p.k) + (sg.lo * p.Hk + hk) * K;
    const float *gf = p.g + sg.lo * p.H + h, *bf = p.beta + sg.lo * p.H + h;
    using MI = InverseMove<C>;
    u32x4_t fx[OUT ? MX::IT : 1], fz[MX::IT], ft[MI::IT];
    float fg = 0.f, fb = 0.f;
    constexpr int DW = 3;  // the helper that forms the decays: one with fewer blocks of the scores
    auto fetch = [&](int cc) {
      const int L = rows_of(cc);
      if constexpr (OUT) MX::load(fx, xf, ldx, L, K, gx, rx);
      MX::load(fz, zf, ldx, L, K, gx, rx);
      if (hw == DW) {
        if (p.g) fg = row_scalar(gf, lane, L, p.H);
        if constexpr (KEEP) fb = row_scalar(bf, lane, L, p.H);
      }
      xf += (int64_t)C * ldx;
      zf += (int64_t)C * ldx;
      gf += (int64_t)C * p.H;
      bf += (int64_t)C * p.H;
      const int64_t slot = delta_slot(p.N, n, sg.a, sg.lo + (int64_t)cc * C, C);
      MI::load(ft, p.inv + (slot * p.H + h) * delta_inverse_bytes(C), ht);
    };
    auto put = [&](int cc) {
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
        t[256 + lane] = KEEP ? fb * d.from : d.from;
        if constexpr (KEEP) t[320 + lane] = fb;
        if (lane == 0) t[384] = d.all;
      }
      MI::template put<false>(ft, inverse_at(cc), hw, lane);
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
          const int f = C == 32 ? i : (i < 2 ? i : 2 * i - 2 + (j >> 1));
          put_parts<3>(v, sP + (f * 192 + lane) * 8 + 4 * (j & 1), 512);
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
    for (int cc = 0; cc < nch; ++cc) {  // beside chunk cc of the state waves
      if constexpr (OUT) scores(cc);
      if constexpr (F::NBUF == 1) __syncthreads();
      if (cc + 1 < nch) put(cc + 1);
      if (cc + 2 < nch) fetch(cc + 2);
      __syncthreads();
    }
    return;
  }

  // ==================================== state waves ====================================
  // this lane's state column: q
  const int wcol = 16 * wave, q = col0 + wcol + l16;
  const bool qin = q < V;

  // ---- the state at the start: channels state_channel(t, grp) + e of its column ----
  f32x4_t S[F::NT];
  {
    // over a boundary, or the sequence's own start: h0 or its copy, made by the state
    // pass where the final state goes over it
    const float *src = sg.in >= 0 ? p.seg_state + ((int64_t)sg.in * p.H + h) * K * V
                       : MODE != kDeltaState && p.seg_first && sg.out >= 0 ? p.seg_first + sbase
                       : p.s0 ? p.s0 + sbase : nullptr;
    if (MODE == kDeltaState && sg.in >= 0) src = nullptr;  // its own change only
    load_state<F::NT>(src, K, V, grp, q, S);
    if (map) {
#pragma unroll
      for (int t = 0; t < F::NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) S[t][e] = state_channel(t, grp) + e == q ? 1.f : 0.f;
    }
    if (MODE == kDeltaState && sg.in < 0 && p.seg_first) store_state<F::NT>(p.seg_first + sbase, K, V, grp, q, S);
    if (skip) {
#pragma unroll
      for (int t = 0; t < F::NT; ++t) S[t] = zero4();
    }
  }

  const int ax = l16 * F::LDX + 8 * grp;  // a row of q or k as an operand
  const int tz = (4 * grp + (l16 >> 2)) * F::LDX + 8 * (l16 & 3);
  const int ldv = p.H * p.V;
  const int64_t vrow = map ? 0 : (sg.lo * p.H + h) * V + col0;
  const T *vc = reinterpret_cast<const T *>(p.v) + vrow;
  const uint32_t gv = qin && !map ? (uint32_t)((4 * grp * ldv + wcol + l16) * SZ) : kOffNone;
  T *yc = reinterpret_cast<T *>(p.o) + vrow;
  const uint32_t gy = wcol + 4 * grp < ncol ? (uint32_t)((l16 * ldv + wcol + 4 * grp) * SZ) : kOffNone;
  float *uc = KEEP ? p.rows_out + vrow : nullptr;

  ColumnRows<T, NC> fv;
  auto fetch_v = [&](int cc) {
    fv.load(tile_rsrc(vc, (uint32_t)(((rows_of(cc) - 1) * ldv + ncol) * SZ)), gv, ldv);
    vc += (int64_t)C * ldv;
  };
  f32x4_t y[OUT ? NC : 1];
  bf16x8_t ub[KS][3];
  // o of chunk cc: y, which holds 2^b q S by then, and its scores times u; a lane has
  // four neighbouring columns of row l16 of each tile
  auto finish = [&](int cc) {
    const bf16_t *const sP = scores_at(cc);
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int i = 0; i < NC; ++i)
        if (s <= i / 2) {
          bf16x8_t a[3];
#pragma unroll
          for (int pl = 0; pl < 3; ++pl) a[pl] = row_frag(sP + ((frag_index<C>(i, s, false) * 3 + pl) * 64 + lane) * 8);
          y[i] = mma_parts(ub[s], a, y[i]);
        }
  };
  auto store = [&](int cc) {
    const auto rs = tile_rsrc(yc, (uint32_t)(((rows_of(cc) - 1) * ldv + ncol) * SZ));
    yc += (int64_t)C * ldv;
    uint32_t off = gy;
    asm volatile("" : "+v"(off));
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int at = (int)(off + 16 * i * ldv * SZ);
      if constexpr (SZ == 4)
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, y[i]), rs, at, 0, 0);
      else
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2_t, to_bf16x4(y[i])), rs, at, 0, 0);
    }
  };

  if (nch > 0) fetch_v(0);
  __syncthreads();
  __syncthreads();
  for (int cc = 0; cc < nch; ++cc) {
    const int L = rows_of(cc);
    const bf16_t *const sX = rows_at(cc), *const sZ = sX + F::nX / 2, *const sT = inverse_at(cc);
    const float *const tab = tab_at(cc);

    if constexpr (KEEP) {  // the state at the chunk's start
      const int64_t slot = delta_slot(p.N, n, sg.a, sg.lo + (int64_t)cc * C, C);
      store_state<F::NT>(p.states + (slot * p.H + h) * K * V, K, V, grp, q, S);
    }

    // What LDS has is asked for well before its use and the order pinned: left to itself
    // the compiler moves a read next to its use, and a SIMD has one or two of these waves,
    // which hide little.
    bf16x8_t kf[NC][IN], qf[OUT ? NC : 1][IN], sb[2][3];
    auto read_rows = [&](bf16x8_t (&f)[NC][IN], const bf16_t *src, int s) {
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int pl = 0; pl < IN; ++pl) f[i][pl] = row_frag(src + pl * F::XPL + 16 * i * F::LDX + ax + 32 * s);
    };
    auto split_state = [&](int s) { split_pair<3>(S[2 * s], S[2 * s + 1], sb[s & 1]); };
    // ---- the last chunk's o, beside the split of the state ----
    read_rows(kf, sZ, 0);
    if (OUT && cc > 0) finish(cc - 1);
    split_state(0);
    if (OUT && cc > 0) store(cc - 1);
    pin();

    // ---- z = k S and y = (q S)^T ----
    f32x4_t z[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      z[i] = zero4();
      if constexpr (OUT) y[i] = zero4();
    }
#pragma unroll
    for (int s = 0; s < F::PS; ++s) {
      if constexpr (OUT) read_rows(qf, sX, s);
      pin();
      mma_cols<NC>(kf, sb[s & 1], z);
      if (!OUT && s + 1 < F::PS) split_state(s + 1);
      pin();
      if (s + 1 < F::PS) read_rows(kf, sZ, s + 1);
      if constexpr (OUT) {
        if (s + 1 < F::PS) split_state(s + 1);
        mma_rows<NC>(sb[s & 1], qf, y);
        pin();
      }
    }

    // ---- u = T r, r = beta (v - a z) (unless u is kept, T has taken beta) ----
    InverseTimes<C, false> ti;
    f32x4_t za[NC], u[NC];
    bf16x8_t rb[KS][3], uc3[KS][3];
    ti.read(sT, lane, 0);
#pragma unroll
    for (int i = 0; i < NC; ++i) za[i] = *reinterpret_cast<const f32x4_t *>(tab + 256 + 16 * i + 4 * grp);
    const float dec = tab[384];
    pin();
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      f32x4_t r[2];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int i = 2 * s + half;
        f32x4_t v = fv.get(i);
        if constexpr (KEEP) v *= *reinterpret_cast<const f32x4_t *>(tab + 320 + 16 * i + 4 * grp);
        r[half] = v - za[i] * z[i];
      }
      split_pair<3>(r[0], r[1], rb[s]);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) u[i] = zero4();
    pin();
    ti.add(rb[0], u, 0);
    if (cc + 1 < nch) fetch_v(cc + 1);
    if constexpr (KS > 1) {
      ti.read(sT, lane, 1);
      pin();
    }
#pragma unroll
    for (int t = 0; t < F::NT; ++t) S[t] *= dec;
    if constexpr (KS > 1) ti.add(rb[KS - 1], u, KS - 1);
    if constexpr (KEEP) {
      const auto rs = tile_rsrc(uc, (uint32_t)(((L - 1) * ldv + ncol) * 4));
      uc += (int64_t)C * ldv;
      uint32_t off = qin ? (uint32_t)((4 * grp * ldv + wcol + l16) * 4) : kOffNone;
      asm volatile("" : "+v"(off));  // formed here, not held in registers over the chunks
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(u[i][e]), rs, (int)(off + (16 * i + e) * ldv * 4), 0, 0);
    }
    // ---- the state: u's parts times c, two tiles at a time (products into one
    // accumulator lie two apart); for o, u's own parts ----
    bf16x8_t zt[2][KS][IN];  // channels of two state tiles by the chunk's rows
    auto read_channels = [&](int t) {
#pragma unroll
      for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int pl = 0; pl < IN; ++pl)
            zt[w][s][pl] = load_frag32_at(sZ + pl * F::XPL + 32 * s * F::LDX + state_channel(t + w, 0), F::LDX, tz);
    };
    read_channels(0);
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const f32x4_t c0 = *reinterpret_cast<const f32x4_t *>(tab + 192 + 32 * s + 4 * grp);
      const f32x4_t c1 = *reinterpret_cast<const f32x4_t *>(tab + 192 + 32 * s + 16 + 4 * grp);
      if constexpr (OUT) split_pair<3>(u[2 * s], u[2 * s + 1], ub[s]);
      split_pair<3>(u[2 * s] * c0, u[2 * s + 1] * c1, uc3[s]);
    }
    pin();
    if constexpr (OUT) {
#pragma unroll
      for (int i = 0; i < NC; ++i) y[i] *= tab[128 + 16 * i + l16];
    }
#pragma unroll
    for (int t = 0; t < F::NT; t += 2) {
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int i = IN - 1; i >= 0; --i)
#pragma unroll
          for (int j = 2; j >= 0; --j)
            if (i + j < 3) {
#pragma unroll
              for (int w = 0; w < 2; ++w) S[t + w] = Mma<bf16_t>::mma(zt[w][s][i], uc3[s][j], S[t + w]);
            }
      if (t + 2 < F::NT) read_channels(t + 2);
    }
    pin();
    if constexpr (F::NBUF == 1) __syncthreads();
    __syncthreads();
  }
  if (OUT && nch > 0) {
    finish(nch - 1);
    store(nch - 1);
  }

  if constexpr (MODE == kDeltaState) {
    const int64_t at = (int64_t)sg.out * p.H + h;
    store_state<F::NT>((map ? p.seg_map : p.seg_state) + at * K * V, K, V, grp, q, S);
  } else if (sg.out < 0) {
    if (p.sT && !(nch == 0 && p.sT == p.s0)) store_state<F::NT>(p.sT + sbase, K, V, grp, q, S);
  }
}

template <typename T, int PT, int NW, int MODE>
hipError_t launch_delta_one(const DeltaWalk &p, hipStream_t st) {
  using F = DeltaCfg<T, PT, NW, MODE>;
  auto kern = delta_walk_kernel<T, PT, NW, MODE>;
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kern), hipFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)F::total);
  if (e != hipSuccess) {
    (void)hipGetLastError();  // do not leave the error for the next launch to report
    return e;
  }
  const int ncb = (p.V + F::QT - 1) / F::QT + (MODE == kDeltaState ? (p.K + F::QT - 1) / F::QT : 0);
  const int64_t grid = delta_walk_blocks(p, ncb);
  if (grid == 0) return hipSuccess;
  if (grid > most_blocks(F::THREADS)) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(F::THREADS), F::total, st, p);
  return hipGetLastError();
}

template <typename T, int PT, int NW>
hipError_t launch_delta_mode(const DeltaWalk &p, hipStream_t st) {
  if (!p.o) return launch_delta_one<T, PT, NW, kDeltaKeep>(p, st);
  if (p.seg) {
    hipError_t e = launch_delta_one<T, PT, NW, kDeltaState>(p, st);
    if (e == hipSuccess) e = launch_delta_chain(p, st);
    if (e != hipSuccess) return e;
  }
  return launch_delta_one<T, PT, NW, kDeltaOut>(p, st);
}

template <typename T, int PT>
hipError_t launch_delta_cols(const DeltaWalk &p, hipStream_t st) {
  int ncb;
  const int cols = delta_cols(p, &ncb);
  if constexpr (sizeof(T) == 2) {
    if (cols == 128) return launch_delta_mode<T, PT, 8>(p, st);
  }
  return launch_delta_mode<T, PT, 4>(p, st);
}

template <typename T>
hipError_t launch_delta_width(const DeltaWalk &p, hipStream_t st) {
  switch (linear_tile(p.K)) {
    case 64: return launch_delta_cols<T, 64>(p, st);
    case 128: return launch_delta_cols<T, 128>(p, st);
    default: return launch_delta_cols<T, 256>(p, st);
  }
}

}  // namespace

}  // namespace kda
