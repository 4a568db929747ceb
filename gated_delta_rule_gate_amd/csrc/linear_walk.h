// Chunked linear attention with one decay per head: the walk over a sequence's
// chunks that gives the forward and, with other operands or in reverse, each
// gradient (linear_launch.h).
//
// One workgroup owns a (sequence or segment, head, block of 16 NW columns) and
// keeps its FP32 state in matrix accumulators: wave w holds columns 16w..16w+15
// of every 16-row state tile. With the channels of a tile pair dealt as
// state_channel() does, an accumulator column is, unchanged, an operand of the
// next product, so the state never leaves registers.
//
// Arithmetic. Every product runs on the bf16 matrix cores. An fp32 operand is
// a sum of bf16 parts (three parts hold all 24 bits), and products of parts
// that together lie below fp32 rounding are left out: bf16 inputs take one
// part, fp32 inputs three, the decayed w rows of the state update three (a
// state carries fp32 rounding only), the scores and the state's copy in the
// output OPL. Decays enter as fp32 factors of accumulators or of w rows, so q
// and k stay exact. Within a chunk b is summed in fp64 and kept as an integer
// and a fraction: differences of far larger sums stay exact to fp32, and the
// exponent of every pair is formed on its own, so no decay is too strong.
//
// Bound by issue: its vector instructions (46% of cycles, half of them the
// splitting of the state and of w into parts) and its matrix instructions (38%),
// on three waves a SIMD. 4 x 4096 tokens of 64 heads, 128 x 128 bf16: 275 us, 4.0
// TB/s; 206 us with loads and stores left out, where its rows alone would take
// 234 us at the rate of a large copy and 188 at that of a scaling in place.
#pragma once

#include "chunk_fused_tiles.h"
#include "linear_launch.h"
#include "linear_segments.h"

namespace kda {

namespace {

// x as the sum of NP bf16 parts, largest first.
template <int NP>
__device__ __forceinline__ void split8(const float (&x)[8], bf16x8_t (&part)[NP]) {
  float r[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = x[e];
#pragma unroll
  for (int pl = 0; pl < NP; ++pl) {
    part[pl] = pack_bf16x8(r);
    if (pl + 1 < NP) {
#pragma unroll
      for (int e = 0; e < 8; ++e) r[e] -= static_cast<float>(part[pl][e]);
    }
  }
}

__device__ __forceinline__ bf16x8_t join8(const bf16x4_t &lo, const bf16x4_t &hi) {
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Slots of a 32-deep step. An operand read from a row holds elements 8 grp..
// 8 grp + 7 of 32 in slots 0..7 (one 16-byte read). A state tile pair is laid out
// to match, so that its accumulators are the other operand as they stand: row
// 4 grp + e of tile t is channel 32 (t / 2) + 8 grp + 4 (t % 2) + e. Tokens keep
// the order of Mma<bf16_t>::kidx (16 rows to a transposing read), and the scores
// are stored in it.
__device__ __forceinline__ int state_channel(int t, int grp) { return 32 * (t >> 1) + 8 * grp + 4 * (t & 1); }
__device__ __forceinline__ bf16x8_t row_frag(const bf16_t *src) { return *reinterpret_cast<const bf16x8_t *>(src); }

// acc += A B over the parts of both that matter: with three parts on either
// side, products of parts i and j with i + j <= 2.
template <int NA, int NB_>
__device__ __forceinline__ f32x4_t mma_parts(const bf16x8_t (&a)[NA], const bf16x8_t (&b)[NB_], f32x4_t acc) {
  constexpr int M = NA > NB_ ? NA : NB_;
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB_ - 1; j >= 0; --j)
      if (i + j < M) acc = Mma<bf16_t>::mma(a[i], b[j], acc);
  return acc;
}

// What a walk does beside its state: y (kOut), y with the rows' dots and the
// states that anchor dg (kDots), or nothing, the state being left at the
// boundary behind the segment (kState).
enum WalkMode : int { kOut = 0, kState = 1, kDots = 2 };

// y[i] += S^T x_i over the parts of both that matter, part by part: products
// into one accumulator lie NC apart.
template <int NC, int NA, int NB_>
__device__ __forceinline__ void mma_rows(const bf16x8_t (&s)[NA], const bf16x8_t (&x)[NC][NB_], f32x4_t (&y)[NC]) {
  constexpr int M = NA > NB_ ? NA : NB_;
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int j = NB_ - 1; j >= 0; --j)
      if (i + j < M) {
#pragma unroll
        for (int r = 0; r < NC; ++r) y[r] = Mma<bf16_t>::mma(s[i], x[r][j], y[r]);
      }
}

// Inclusive sum over the wave's 64 lanes in fp64: within rows of 16 by row
// shifts, across them by the broadcasts of a row's and a half's last lane, all
// on the VALU (lane shuffles through the LDS unit took four times as long).
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_or_zero(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, ROWS, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, ROWS, 0xf, false);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double wave_scan(double x) {
  x += dpp_or_zero<0x111, 0xf>(x);  // row_shr:1, 2, 4, 8
  x += dpp_or_zero<0x112, 0xf>(x);
  x += dpp_or_zero<0x114, 0xf>(x);
  x += dpp_or_zero<0x118, 0xf>(x);
  x += dpp_or_zero<0x142, 0xa>(x);  // row_bcast:15 into rows 1 and 3
  x += dpp_or_zero<0x143, 0xc>(x);  // row_bcast:31 into rows 2 and 3
  return x;
}
__device__ __forceinline__ double last_lane(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, 63), hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}

// Sum over the wave's four rows of 16 lanes, in every row (two VALU swaps).
__device__ __forceinline__ float rows4_sum(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  const unsigned h = __float_as_uint(__uint_as_float(r[0]) + __uint_as_float(r[1]));
  const auto t = __builtin_amdgcn_permlane32_swap(h, h, false, false);
  return __uint_as_float(t[0]) + __uint_as_float(t[1]);
}

// Geometry of one walk.
template <typename T, int PT_, int NW_, int OPL_, int MODE_>
struct WalkCfg {
  static constexpr bool F32 = sizeof(T) == 4;
  static constexpr int PT = PT_, NW = NW_, OPL = OPL_, MODE = MODE_;
  static constexpr int IN = F32 ? 3 : 1;  // bf16 parts of an input
  static constexpr int C = (F32 || PT == 256) ? 32 : 64;
  static constexpr int NC = C / 16, KS = C / 32, PS = PT / 32, NT = PT / 16, QT = 16 * NW;
  static constexpr int HELPERS = 4, THREADS = 64 * (NW + HELPERS), HT = 64 * HELPERS;
  // Row strides are 32 bytes past a multiple of 128. LDS instructions measured
  // on MI355X at this stride, in cycles a wave with eight waves reading: 16 rows
  // by 16-byte reads 4.5 (8.0 at 16 bytes past), transposing reads at 8-byte
  // steps 3.2, at 16-byte steps 4.2 (8.0); two 8-byte reads in one instruction 32.
  static constexpr int LDX = PT + 16, LDW = QT + 16, LDP = C + 16;
  static constexpr int XPL = C * LDX, WPL = C * LDW, PPL = C * LDP;  // elements of one part
  static constexpr unsigned nX = MODE != kState ? 2u * IN * XPL : 0u, nZ = 2u * IN * XPL, nW = 2u * IN * WPL;
  static constexpr unsigned rows = nX + nZ + nW;  // one chunk's rows
  static constexpr unsigned nP = MODE != kState ? 2u * OPL * PPL : 0u;
  static constexpr unsigned tab = 4u * (4 * 64 + 4);  // hi, lo, a, c of every row, and the chunk's decay
  static constexpr unsigned red = MODE == kDots ? 2 * 4u * NW * 64 + 64 : 64u;  // row dots of every wave; <h, dh>
  // two chunks' rows, and two chunks' scores, where they fit
  static constexpr int NBUF = 2 * rows + nP + 2 * tab + red <= 160 * 1024 ? 2 : 1;
  static constexpr int PBUF = NBUF == 2 && 2 * (rows + nP + tab) + red <= 160 * 1024 ? 2 : 1;
  // y leaves through x's place in LDS, which its chunk no longer needs, so that
  // the helpers store whole rows (a state wave's 32-byte pieces of 16 rows cost
  // four times the address work)
  static constexpr bool STAGE = !F32 && MODE != kState && NBUF == 2 && QT <= PT;
  static constexpr unsigned oP = NBUF * rows, oTab = oP + PBUF * nP, oRed = oTab + 2 * tab, total = oRed + red;
  static_assert(total <= 160 * 1024, "LDS");
};

// Rows of one chunk on their way to LDS: 16-byte loads at offsets that do not
// change from chunk to chunk (the resource's base does), columns past the
// width at an offset that reads zeros, rows past the chunk past its end.
template <typename T, int NT, int ROWS, int COLS>
struct RowsMove {
  static constexpr int EPV = 16 / (int)sizeof(T);
  static constexpr int VPR = COLS / EPV, NV = ROWS * VPR, IT = (NV + NT - 1) / NT;
  static_assert(NV % NT == 0 && NT % VPR == 0, "whole rows per round");
  static constexpr int RPI = NT / VPR;  // rows of one round

  static __device__ __forceinline__ uint32_t lane_offset(int tid, int64_t ldg, int ncol) {
    const int r = tid / VPR, c = (tid % VPR) * EPV;
    return c < ncol ? (uint32_t)((r * ldg + c) * (int64_t)sizeof(T)) : kOffNone;
  }
  static __device__ __forceinline__ int lds_offset(int tid, int lds) { return (tid / VPR) * lds + (tid % VPR) * EPV; }
  // rows [0, L) from base; `round` is RPI rows in bytes
  static __device__ __forceinline__ void load(u32x4_t (&buf)[IT], const T *base, int64_t ldg, int L, int ncol,
                                              uint32_t off, uint32_t round) {
    const auto rs = tile_rsrc(base, (uint32_t)(((int64_t)(L - 1) * ldg + ncol) * (int64_t)sizeof(T)));
#pragma unroll
    for (int it = 0; it < IT; ++it)
      buf[it] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, (int)(off + it * round), 0, 0));
  }
  static __device__ __forceinline__ void put(const u32x4_t (&buf)[IT], bf16_t *s, int lds, int plane) {
#pragma unroll
    for (int it = 0; it < IT; ++it) {
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<u32x4_t *>(s + it * RPI * lds) = buf[it];
      } else {
        f32x4_t x = __builtin_bit_cast(f32x4_t, buf[it]);
#pragma unroll
        for (int pl = 0; pl < 3; ++pl) {
          const bf16x4_t h = to_bf16x4(x);
          *reinterpret_cast<bf16x4_t *>(s + pl * plane + it * RPI * lds) = h;
          x -= to_f32x4(h);
        }
      }
    }
  }
};

// NW state waves each keep 16 columns of the state; four helper waves, one a
// SIMD beside two state waves, bring rows to LDS, form decays and the scores.
// A chunk takes two periods between barriers:
//   state waves   y = a (x S) of chunk c        | y += scores w, y out, S updated and
//                 w decayed                     | split for the next x S
//   helper waves  rows of c + 1 (loaded a chunk | scores of c + 1
//                 ago) to LDS, its decays, the
//                 loads of c + 2
// so the state's chain holds no load, no decay and no score. Where LDS holds one
// chunk's scores the helpers form those of c beside a (x S) and bring c + 1
// afterwards; where it holds one chunk's rows (fp32 by 128 columns or 256
// wide), those go to LDS in a period of their own. Products that give y and scores are taken
// transposed, so that a lane holds four neighbouring columns of one row and both
// leave in 8-byte pieces.
template <typename T, int PT, int NW, bool REV, int OPL, int MODE>
__global__ __launch_bounds__(64 * (NW + 4)) __attribute__((amdgpu_waves_per_eu((NW + 4) / 4, (NW + 4) / 4)))
void linear_walk_kernel(LinearWalk p) {
  using F = WalkCfg<T, PT, NW, OPL, MODE>;
  constexpr int C = F::C, NC = F::NC, KS = F::KS, IN = F::IN, QT = F::QT, NB = NC * (NC + 1) / 2;
  using MX = RowsMove<T, F::HT, C, PT>;
  using MW = RowsMove<T, F::HT, C, QT>;
  extern __shared__ __align__(16) char smem[];

  // Workgroups that read the same q/k rows (a group's heads, a head's column
  // blocks) go to one XCD, next to each other: ids are dealt to the eight XCDs
  // in turn. Whole segments come before the sequences' first, which may be short.
  const int ncb = (p.Q + QT - 1) / QT;
  const int G = p.H / p.Hk, U = G * ncb;
  const int xcd = blockIdx.x & 7, sl = blockIdx.x >> 3;
  const int64_t unit = (int64_t)(sl / U) * 8 + xcd;
  const int member = sl % U;
  const int64_t n_items = p.N + (p.seg ? ((int64_t)p.B * p.T) / p.seg : 0);
  const int64_t item = n_items - 1 - unit / p.Hk;
  const int h = (int)(unit % p.Hk) * G + member / ncb, cb = member % ncb;
  SegLoc sg;
  if (item < 0 || !locate_segment(p, item, REV, sg)) return;
  if (MODE == kState && sg.out < 0) return;  // nothing follows the last segment

  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int grp = lane >> 4, l16 = lane & 15;
  const int P = p.P, Q = p.Q, col0 = cb * QT, ncol = min(QT, Q - col0);
  const int64_t rows = (int64_t)p.B * p.T;

  const int64_t sbase = ((int64_t)sg.n * p.H + h) * P * Q;

  constexpr int SZ = sizeof(T);
  const int nch = (int)((sg.hi - sg.lo + C - 1) / C);
  const int tail = (int)(sg.hi - sg.lo) - (nch - 1) * C;  // rows of the last chunk in token order
  const int64_t first = sg.lo + (REV ? (int64_t)(nch - 1) * C : 0);
  constexpr int STEP = REV ? -C : C;
  auto rows_of = [&](int cc) { return (REV ? cc == 0 : cc == nch - 1) ? tail : C; };
  auto rows_at = [&](int cc) { return reinterpret_cast<bf16_t *>(smem + (F::NBUF == 2 && (cc & 1) ? F::rows : 0u)); };
  auto scores_at = [&](int cc) {
    return reinterpret_cast<bf16_t *>(smem + F::oP + (F::PBUF == 2 && (cc & 1) ? F::nP : 0u));
  };
  auto tab_at = [&](int cc) { return reinterpret_cast<float *>(smem + F::oTab + ((cc & 1) ? F::tab : 0u)); };
  float *const sRed = reinterpret_cast<float *>(smem + F::oRed);
  double *const sAnc = reinterpret_cast<double *>(sRed + (MODE == kDots ? 2 * NW * 64 : 0));  // a value of every state wave
  // whole multiples of kLinearAnchor tokens into the sequence, before its end
  auto anchored = [&](int64_t t0, int L) {
    return MODE == kDots && (((uint32_t)(t0 - sg.a) + L) % kLinearAnchor) == 0 && t0 + L < sg.e;
  };

  if (wave >= NW) {
    // =================================== helper waves ===================================
    // what a helper holds up, eight state waves wait for (1.5 to 3.5% shorter walks)
    __builtin_amdgcn_s_setprio(2);
    const int hw = wave - NW, ht = tid - 64 * NW;
    const int ldx = p.Hx * P, ldw = p.Hw * Q;  // row strides, elements
    const uint32_t gx = MX::lane_offset(ht, ldx, P), gw = MW::lane_offset(ht, ldw, ncol);
    const uint32_t rx = (uint32_t)(MX::RPI * ldx * SZ), rw = (uint32_t)(MW::RPI * ldw * SZ);
    const int px = MX::lds_offset(ht, F::LDX), pw = MW::lds_offset(ht, F::LDW);
    const int ax = l16 * F::LDX + 8 * grp;  // a row of x or z as an operand
    const T *xf = reinterpret_cast<const T *>(p.x) + (first * p.Hx + h / (p.H / p.Hx)) * P;
    const T *zf = reinterpret_cast<const T *>(p.z) + (first * p.Hx + h / (p.H / p.Hx)) * P;
    const T *wf = reinterpret_cast<const T *>(p.w) + (first * p.Hw + h / (p.H / p.Hw)) * Q + col0;
    const float *gf = p.g + (p.g_head ? h : first * p.H + h);
    const int64_t dx = (int64_t)STEP * ldx, dw = (int64_t)STEP * ldw, dg = p.g_head ? 0 : (int64_t)STEP * p.H;
    // loads run a chunk ahead (two ahead changed nothing where only the state is
    // walked, and spilled otherwise)
    u32x4_t fx[MODE != kState ? MX::IT : 1], fz[MX::IT], fw[MW::IT];
    float fg = 0.f;
    double total = 0.0;  // log2 decay of the whole segment (the decays' wave)
    constexpr int DW = 3;  // the helper that forms the decays: one with fewer blocks of the scores
    auto fetch = [&](int cc) {  // chunk after chunk in the walk's order
      const int L = rows_of(cc);
      if constexpr (MODE != kState) MX::load(fx, xf, ldx, L, P, gx, rx);
      MX::load(fz, zf, ldx, L, P, gx, rx);
      MW::load(fw, wf, ldw, L, ncol, gw, rw);
      if (hw == DW) {
        const auto rs = tile_rsrc(gf, (uint32_t)(p.g_head ? 4 : ((L - 1) * p.H + 1) * 4));
        fg = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
            rs, lane < L ? (p.g_head ? 0 : lane * p.H * 4) : (int)kOffNone, 0, 0));
      }
      xf += dx;
      zf += dx;
      wf += dw;
      gf += dg;
    };
    // The chunk's decays: b summed in fp64, as an integer and a fraction; a is
    // the factor of x S, c that of z in the state. The scale goes with y, in
    // reverse with z. A decay below 2^-160 is none at all and counts as
    // 2^-32768: differences across it give zero, those beyond it stay exact.
    auto decays = [&](int cc) {
      if (hw != DW) return;
      double b = (double)fg * 1.4426950408889634073599;
      if (b <= -160.0) b = -32768.0;
      b = wave_scan(b);
      const double bl = last_lane(b);
      const double hi = rint(b);
      const float from = fast_exp2((float)b), rest = fast_exp2((float)(bl - b));
      float *t = tab_at(cc);
      t[lane] = (float)hi;
      t[64 + lane] = (float)(b - hi);
      t[128 + lane] = REV ? rest : from * p.scale;
      t[192 + lane] = REV ? from * p.scale : rest;
      if (lane == 0) t[256] = fast_exp2((float)bl);
      total += bl;
    };
    auto bring = [&](int cc) {  // rows and decays of cc to LDS, the loads of the chunk after it
      bf16_t *s = rows_at(cc);
      if constexpr (MODE != kState) MX::put(fx, s + px, F::LDX, F::XPL);
      MX::put(fz, s + F::nX / 2 + px, F::LDX, F::XPL);
      MW::put(fw, s + (F::nX + F::nZ) / 2 + pw, F::LDW, F::WPL);
      decays(cc);
      if (cc + 1 < nch) fetch(cc + 1);
    };
    // scores of the causal 16 x 16 blocks, decayed and scaled, a wave taking
    // every fourth: lane has row l16 of x, four rows of z
    auto scores = [&](int cc) {
      const bf16_t *const sX = rows_at(cc), *const sZ = sX + F::nX / 2;
      const float *const tab = tab_at(cc);
      bf16_t *const sP = scores_at(cc);
#pragma unroll
      for (int b0 = 0; b0 < NB; b0 += F::HELPERS) {
        const int blk = b0 + hw;
        if (b0 + F::HELPERS <= NB || blk < NB) {
          const int i = blk < 1 ? 0 : (blk < 3 ? 1 : (blk < 6 ? 2 : 3)), j = blk - i * (i + 1) / 2;
          const int ri = REV ? j : i, cj = REV ? i : j;
          const bf16_t *xs = sX + 16 * ri * F::LDX + ax, *zs = sZ + 16 * cj * F::LDX + ax;
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
          const float hr = tab[16 * ri + l16], lr = tab[64 + 16 * ri + l16];
          const f32x4_t hs = *reinterpret_cast<const f32x4_t *>(tab + 16 * cj + 4 * grp);
          const f32x4_t ls = *reinterpret_cast<const f32x4_t *>(tab + 64 + 16 * cj + 4 * grp);
          f32x4_t v;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float d = REV ? (hs[e] - hr) + (ls[e] - lr) : (hr - hs[e]) + (lr - ls[e]);
            const bool keep = i != j || (REV ? 4 * grp + e >= l16 : 4 * grp + e <= l16);
            v[e] = keep ? acc[e] * (fast_exp2(d) * p.scale) : 0.f;
          }
          bf16_t *dst = sP + (16 * ri + l16) * F::LDP + 32 * (cj >> 1) + 8 * grp + 4 * (cj & 1);
#pragma unroll
          for (int pl = 0; pl < OPL; ++pl) {
            const bf16x4_t part = to_bf16x4(v);
            *reinterpret_cast<bf16x4_t *>(dst + pl * F::PPL) = part;
            if (pl + 1 < OPL) v -= to_f32x4(part);
          }
        }
      }
    };
    // y of chunk cc, row by row, from where the state waves left it: a thread
    // reads the places that its own rows of x go to next
    const int ldy = p.H * Q;
    const int yr = ht / MX::VPR, yq = (ht % MX::VPR) * MX::EPV;
    char *yc = reinterpret_cast<char *>(p.y) + ((first * p.H + h) * Q + col0) * 2;
    const int64_t dy = (int64_t)STEP * ldy * 2;
    auto store_rows = [&](int cc) {
      if (p.y_f32) return;
      const auto rs = tile_rsrc(yc, (uint32_t)(((rows_of(cc) - 1) * ldy + ncol) * 2));
      yc += dy;
      const bf16_t *s = rows_at(cc) + px;
      u32x4_t v[MX::IT];
#pragma unroll
      for (int it = 0; it < MX::IT; ++it) v[it] = *reinterpret_cast<const u32x4_t *>(s + it * MX::RPI * F::LDX);
#pragma unroll
      for (int it = 0; it < MX::IT; ++it)
      {
        const int r = yr + it * MX::RPI, c = yq ^ (((r >> 3) & 1) * 8);  // where the state waves put it
        __builtin_amdgcn_raw_buffer_store_b128(v[it], rs, c < ncol && yq < QT ? (r * ldy + c) * 2 : (int)kOffNone, 0, 0);
      }
    };
    auto dots = [&](int cc) {  // the row dots of chunk cc, whole and of a (x S): every state wave's part
      const int L = rows_of(cc), r = ht & 63, which = ht >> 6;
      if (which < 2 && r < L) {
        float d = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) d += sRed[(which * NW + w) * 64 + r];
        float *dst = which ? p.dot_far : p.dot;
        dst[((int64_t)cb * p.H + h) * rows + first + (int64_t)cc * STEP + r] = d;
      }
    };
    auto anchor = [&](int cc) {  // <h, dh> behind chunk cc
      const int L = rows_of(cc);
      const int64_t t0 = first + (int64_t)cc * STEP;
      if (anchored(t0, L) && ht == 0) {
        double d = 0.0;
#pragma unroll
        for (int w = 0; w < NW; ++w) d += sAnc[w];
        p.anchor_dot[(((t0 + L) / kLinearAnchor) * p.H + h) * ncb + cb] = (float)d;
      }
    };

    if (nch > 0) fetch(0);
    if constexpr (MODE != kState) {
      // the blocks of the scores beyond the triangle stay zero
      for (int i = ht; i < (int)(F::PBUF * F::nP / 4); i += F::HT) reinterpret_cast<unsigned *>(smem + F::oP)[i] = 0u;
    }
    if (nch > 0) bring(0);
    __syncthreads();
    if constexpr (F::PBUF == 2 && MODE != kState) {
      if (nch > 0) scores(0);
      __syncthreads();
    }
    for (int cc = 0; cc < nch; ++cc) {  // beside chunk cc of the state waves
      if (MODE == kDots && cc > 0) dots(cc - 1);
      if (F::STAGE && cc > 0) store_rows(cc - 1);
      if constexpr (F::PBUF == 2 && MODE != kState) {
        if (cc + 1 < nch) bring(cc + 1);
        __syncthreads();
        if (MODE == kDots && REV) anchor(cc);
        if (cc + 1 < nch) scores(cc + 1);
        __syncthreads();
      } else {
        if constexpr (MODE != kState) {
          scores(cc);
          __syncthreads();
          if (MODE == kDots && REV) anchor(cc);
        }
        if constexpr (F::NBUF == 1) __syncthreads();
        if (cc + 1 < nch) bring(cc + 1);
        __syncthreads();
      }
    }
    if (MODE == kDots && nch > 0) dots(nch - 1);
    if (F::STAGE && nch > 0) store_rows(nch - 1);
    if (MODE == kState && hw == DW && lane == 0 && cb == 0) p.seg_decay[sg.out * p.H + h] = total;
    if (MODE == kDots && p.end_dot && sg.out < 0) {
      __syncthreads();
      if (ht == 0) {
        double d = 0.0;
        for (int w = 0; w < NW; ++w) d += sAnc[w];
        p.end_dot[((int64_t)sg.n * p.H + h) * ncb + cb] = (float)d;
      }
    }
    return;
  }

  // ==================================== state waves ====================================
  const int q = col0 + 16 * wave + l16;  // this lane's state column
  const int64_t frag = ((int64_t)h * ncb + cb) * (PT * QT) + ((int64_t)wave * F::NT * 64 + lane) * 4;
  const int64_t fragH = (int64_t)p.H * ncb * (PT * QT);  // elements of one boundary

  // ---- the state at the segment's start: channels state_channel(t, grp) + e of column q ----
  f32x4_t S[F::NT];
  {
    // over a boundary, or the sequence's own start: h0 or its copy, made by the
    // state pass where the final state goes over it
    const float *src = sg.in >= 0 ? p.seg_state + ((int64_t)sg.in * p.H + h) * P * Q
                       : MODE != kState && p.seg_first && sg.out >= 0 ? p.seg_first + sbase
                       : p.s0 ? p.s0 + sbase : nullptr;
    if (MODE == kState && sg.in >= 0) src = nullptr;  // its own change only
#pragma unroll
    for (int t = 0; t < F::NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = state_channel(t, grp) + e;
        S[t][e] = (src && r < P && q < Q) ? src[r * p.sp + q * p.sq] : 0.f;
      }
    if (MODE == kState && sg.in < 0 && p.seg_first) {
#pragma unroll
      for (int t = 0; t < F::NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = state_channel(t, grp) + e;
          if (r < P && q < Q) p.seg_first[sbase + r * p.sp + q * p.sq] = S[t][e];
        }
    }
  }

  const int ax = l16 * F::LDX + 8 * grp;  // a row of x as an operand
  const int tz = (4 * grp + (l16 >> 2)) * F::LDX + 8 * (l16 & 3), tw = cfrag_lane_off(F::LDW) + 16 * wave;
  const int ap = l16 * F::LDP + 8 * grp;  // a row of the scores
  // y and its partner u: four neighbouring columns of row l16 of each 16
  const int ldu = p.Hu * Q, ldy = p.H * Q, ysz = SZ == 4 || p.y_f32 ? 4 : 2;
  const bool yin = 16 * wave + 4 * grp < ncol;
  const uint32_t gu = yin ? (uint32_t)((l16 * ldu + 16 * wave + 4 * grp) * SZ) : kOffNone;
  const uint32_t gy = yin ? (uint32_t)((l16 * ldy + 16 * wave + 4 * grp) * ysz) : kOffNone;
  const T *uc = reinterpret_cast<const T *>(p.u) + (first * p.Hu + h / (p.H / p.Hu)) * Q + col0;
  char *yc = reinterpret_cast<char *>(p.y) + ((first * p.H + h) * Q + col0) * ysz;
  const int64_t du = (int64_t)STEP * ldu, dy = (int64_t)STEP * ldy * ysz;

  f32x4_t y[NC];
  bf16x4_t uh[NC];
  f32x4_t uf[NC];
  // The state as an operand of x S: split beside the matrix products that update
  // it, so that x S starts with products; split there where 256 rows of state
  // or the dots leave no registers to hold it.
  constexpr bool KEEP = MODE == kOut && PT <= 128;
  bf16x8_t sb[KEEP ? F::PS : 1][OPL];
  auto split_state = [&](int s) {
    const float sv[8] = {S[2 * s][0], S[2 * s][1], S[2 * s][2], S[2 * s][3],
                         S[2 * s + 1][0], S[2 * s + 1][1], S[2 * s + 1][2], S[2 * s + 1][3]};
    split8<OPL>(sv, sb[KEEP ? s : 0]);
  };
  if constexpr (KEEP) {
#pragma unroll
    for (int s = 0; s < F::PS; ++s) split_state(s);
  }
  // w as an operand, and decayed to the chunk's end in three parts
  bf16x8_t wf[KS][IN], wc[KS][3];
  auto decay_w = [&](int cc, int s) {
    const bf16_t *const sW = rows_at(cc) + (F::nX + F::nZ) / 2;
    const float *const tab = tab_at(cc);
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int pl = IN - 1; pl >= 0; --pl) {
      wf[s][pl] = load_frag32_at(sW + pl * F::WPL + 32 * s * F::LDW, F::LDW, tw);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] += static_cast<float>(wf[s][pl][e]);
    }
    const f32x4_t c0 = *reinterpret_cast<const f32x4_t *>(tab + 192 + 32 * s + 4 * grp);
    const f32x4_t c1 = *reinterpret_cast<const f32x4_t *>(tab + 192 + 32 * s + 16 + 4 * grp);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] *= c0[e];
      x[e + 4] *= c1[e];
    }
    split8<3>(x, wc[s]);
  };

  __syncthreads();
  if constexpr (F::PBUF == 2 && MODE != kState) __syncthreads();
  for (int cc = 0; cc < nch; ++cc) {
    const int L = rows_of(cc);
    const int64_t t0 = first + (int64_t)cc * STEP;
    const bf16_t *const sX = rows_at(cc), *const sZ = sX + F::nX / 2;
    const float *const tab = tab_at(cc);

    // Half of the state behind an anchored chunk loads beside a (x S), the other
    // half afterwards: all of it there spilled and was no faster, none of it there
    // left 7% of the walk waiting.
    constexpr int CK = MODE == kDots && REV ? F::NT / 2 : 1;
    const float *const ck_src = p.ckpt + ((t0 + L) / kLinearAnchor) * fragH + frag;
    f32x4_t ck[CK];
    if constexpr (MODE != kState) {
      if constexpr (MODE == kDots) {
        if (REV && anchored(t0, L)) {  // h behind this chunk, on its way beside a (x S)
#pragma unroll
          for (int t = 0; t < CK; ++t) ck[t] = *reinterpret_cast<const f32x4_t *>(ck_src + t * 256);
        }
        // the row dots' partners: four columns of a row a lane
        const auto rs = tile_rsrc(uc, (uint32_t)(((L - 1) * ldu + ncol) * SZ));
        uc += du;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int off = (int)(gu + 16 * i * ldu * SZ);
          if constexpr (SZ == 2) uh[i] = __builtin_bit_cast(bf16x4_t, __builtin_amdgcn_raw_buffer_load_b64(rs, off, 0, 0));
          else uf[i] = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(rs, off, 0, 0));
        }
      }
      // ---- y = a (x S), and w's parts beside the products ----
#pragma unroll
      for (int i = 0; i < NC; ++i) y[i] = zero4();
#pragma unroll
      for (int s = 0; s < F::PS; ++s) {
        bf16x8_t a[NC][IN];
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int pl = 0; pl < IN; ++pl) a[i][pl] = row_frag(sX + pl * F::XPL + 16 * i * F::LDX + ax + 32 * s);
        if (s < KS) decay_w(cc, s);
        if constexpr (!KEEP) split_state(s);
        mma_rows<NC>(sb[KEEP ? s : 0], a, y);
      }
#pragma unroll
      for (int i = 0; i < NC; ++i) y[i] *= tab[128 + 16 * i + l16];
      if (MODE == kDots && REV && anchored(t0, L)) {  // <h, dh> behind this chunk
        float d = 0.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
#pragma unroll
          for (int t = 0; t < CK; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) d += ck[t][e] * S[half * CK + t < F::NT ? half * CK + t : 0][e];
          if (half == 0)
#pragma unroll
            for (int t = 0; t < CK; ++t) ck[t] = *reinterpret_cast<const f32x4_t *>(ck_src + (CK + t) * 256);
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) d += __shfl_xor(d, off);
        if (lane == 0) sAnc[wave] = d;
      }
      // w's parts are formed in this period, beside x S: left to itself the
      // compiler moves them behind the barrier, before their use (with the dots'
      // registers it has to: holding them spills)
      if constexpr (MODE == kOut) {
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int pl = 0; pl < 3; ++pl) {
            u32x4_t v = __builtin_bit_cast(u32x4_t, wc[s][pl]);
            asm volatile("" : "+v"(v));
            wc[s][pl] = __builtin_bit_cast(bf16x8_t, v);
          }
      }
      __syncthreads();
    } else {
#pragma unroll
      for (int s = 0; s < KS; ++s) decay_w(cc, s);
    }

    if constexpr (MODE != kState) {
      // ---- y += scores w, out ----
      const bf16_t *const sP = scores_at(cc);
      const auto rs = tile_rsrc(yc, (uint32_t)(((L - 1) * ldy + ncol) * ysz));
      yc += dy;
      auto row_dots = [&](int which) {  // this wave's columns of the rows' dots; u is zero past the width
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const f32x4_t u = SZ == 2 ? to_f32x4(uh[i]) : uf[i];
          float d = (y[i][0] * u[0] + y[i][1] * u[1]) + (y[i][2] * u[2] + y[i][3] * u[3]);
          d = rows4_sum(d);
          if (grp == 0) sRed[(which * NW + wave) * 64 + 16 * i + l16] = d;
        }
      };
      if constexpr (MODE == kDots) row_dots(1);
      // every operand first, so that their reads are in flight together (of three
      // parts, those of half the tokens: registers)
      constexpr int GROUP = OPL == 3 ? 1 : KS;
#pragma unroll
      for (int s0 = 0; s0 < KS; s0 += GROUP) {
        bf16x8_t a[NC][GROUP][OPL];
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
          for (int s = s0; s < s0 + GROUP; ++s)
            if (REV ? s >= i / 2 : s <= i / 2) {
#pragma unroll
              for (int pl = 0; pl < OPL; ++pl) a[i][s - s0][pl] = row_frag(sP + pl * F::PPL + 16 * i * F::LDP + ap + 32 * s);
            }
#pragma unroll
        for (int s = s0; s < s0 + GROUP; ++s)
#pragma unroll
          for (int i = 0; i < NC; ++i)
            if (REV ? s >= i / 2 : s <= i / 2) y[i] = mma_parts(wf[s], a[i][s - s0], y[i]);
      }
      if (F::STAGE && ysz == 2) {
        // rows 8..15 of 16 swap 16-byte neighbours: 16 rows then cover all banks
        bf16_t *dst = rows_at(cc) + l16 * F::LDX + ((16 * wave + 4 * grp) ^ (l16 & 8));
#pragma unroll
        for (int i = 0; i < NC; ++i) *reinterpret_cast<bf16x4_t *>(dst + 16 * i * F::LDX) = to_bf16x4(y[i]);
      } else if (ysz == 4) {
#pragma unroll
        for (int i = 0; i < NC; ++i)
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4_t, y[i]), rs, (int)(gy + 16 * i * ldy * ysz), 0, 0);
      } else {
#pragma unroll
        for (int i = 0; i < NC; ++i)
          __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2_t, to_bf16x4(y[i])), rs,
                                                (int)(gy + 16 * i * ldy * ysz), 0, 0);
      }
      if constexpr (MODE == kDots) row_dots(0);
    }

    // ---- the state ----
    const float dec = tab[256];
    // two tiles at a time: products into one accumulator lie two apart
#pragma unroll
    for (int t = 0; t < F::NT; t += 2) {
      bf16x8_t a[2][KS][IN];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int pl = 0; pl < IN; ++pl)
            a[u][s][pl] = load_frag32_at(sZ + pl * F::XPL + 32 * s * F::LDX + state_channel(t + u, 0), F::LDX, tz);
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
              for (int u = 0; u < 2; ++u) S[t + u] = Mma<bf16_t>::mma(a[u][s][i], wc[s][j], S[t + u]);
            }
      if (KEEP) split_state(t / 2);
    }
    if (!REV && anchored(t0, L)) {
      float *dst = p.ckpt + ((t0 + L) / kLinearAnchor) * fragH + frag;
#pragma unroll
      for (int t = 0; t < F::NT; ++t) *reinterpret_cast<f32x4_t *>(dst + t * 256) = S[t];
    }
    if constexpr (F::NBUF == 1) __syncthreads();
    __syncthreads();
  }

  if constexpr (MODE == kState) {
    float *dst = p.seg_state + ((int64_t)sg.out * p.H + h) * P * Q;
#pragma unroll
    for (int t = 0; t < F::NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = state_channel(t, grp) + e;
        if (r < P && q < Q) dst[r * p.sp + q * p.sq] = S[t][e];
      }
  } else if (sg.out < 0) {
    if (p.sT && !(nch == 0 && p.sT == p.s0)) {
#pragma unroll
      for (int t = 0; t < F::NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = state_channel(t, grp) + e;
          if (r < P && q < Q) p.sT[sbase + r * p.sp + q * p.sq] = S[t][e];
        }
    }
    if (MODE == kDots && p.end_dot) {
      // fp64: in fp32 a lane's 32 or 64 sums in a row were off by twice what the states are.
      // (the P axis of these states is the inner one: four channels to a load)
      double d = 0.0;
#pragma unroll
      for (int t = 0; t < F::NT; ++t) {
        const int r = state_channel(t, grp);
        if (r < P && q < Q) {
          const f32x4_t u = *reinterpret_cast<const f32x4_t *>(p.s_dot + sbase + r + q * p.sq);
#pragma unroll
          for (int e = 0; e < 4; ++e) d += (double)S[t][e] * (double)u[e];
        }
      }
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) d += __shfl_xor(d, off);
      if (lane == 0) sAnc[wave] = d;
      __syncthreads();
    }
  }
}

template <typename T, int PT, int NW, bool REV, int OPL, int MODE>
hipError_t launch_one(const LinearWalk &p, hipStream_t st) {
  using F = WalkCfg<T, PT, NW, OPL, MODE>;
  auto kern = linear_walk_kernel<T, PT, NW, REV, OPL, MODE>;
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kern), hipFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)F::total);
  if (e != hipSuccess) {
    (void)hipGetLastError();  // do not leave the error for the next launch to report
    return e;
  }
  const int ncb = (p.Q + F::QT - 1) / F::QT;
  const int64_t grid = linear_walk_blocks(p, ncb);
  if (grid > most_blocks(F::THREADS)) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(F::THREADS), F::total, st, p);
  return hipGetLastError();
}

template <typename T, int PT, int NW, bool REV, int OPL, int MODE>
hipError_t launch_modes(const LinearWalk &p, hipStream_t st) {
  if (p.seg && !p.seg_ready) {
    // The state pass's segments (all but a sequence's last; packed, about the
    // multiples of seg) by 64 columns where by 128 they leave half the compute
    // units idle: the same waves, two to a SIMD less (one segment of 1024 tokens
    // on each of 128 (sequence, head) pairs: 43 us by 128, 36 us by 64).
    const int64_t segs = p.cu ? ((int64_t)p.B * p.T) / p.seg : (int64_t)p.N * ((p.T + p.seg - 1) / p.seg - 1);
    const bool halves = NW > 4 && segs * p.H * ((p.Q + 127) / 128) * 2 <= device_cus();
    hipError_t e = halves ? launch_one<T, PT, 4, REV, 1, kState>(p, st) : launch_one<T, PT, NW, REV, 1, kState>(p, st);
    if (e != hipSuccess) return e;
    if ((e = launch_linear_chain(p, REV, st)) != hipSuccess) return e;
  }
  return launch_one<T, PT, NW, REV, OPL, MODE>(p, st);
}

template <typename T, int PT, bool REV, int OPL, int MODE>
hipError_t launch_cols(const LinearWalk &p, hipStream_t st) {
  int ncb;
  if constexpr (sizeof(T) == 2 || PT <= 128) {
    if (linear_cols(p.P, p.Q, p.is_bf16, (int64_t)p.N * p.H, &ncb) == 128)
      return launch_modes<T, PT, 8, REV, OPL, MODE>(p, st);
  }
  return launch_modes<T, PT, 4, REV, OPL, MODE>(p, st);
}

template <typename T, bool REV, int OPL, int MODE>
hipError_t launch_width(const LinearWalk &p, hipStream_t st) {
  switch (linear_tile(p.P)) {
    case 64: return launch_cols<T, 64, REV, OPL, MODE>(p, st);
    case 128: return launch_cols<T, 128, REV, OPL, MODE>(p, st);
    default: return launch_cols<T, 256, REV, OPL, MODE>(p, st);
  }
}

}  // namespace

}  // namespace kda
