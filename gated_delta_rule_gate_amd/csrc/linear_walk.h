// Chunked linear attention with one decay per head: the walk over a sequence's
// chunks that gives the forward and, with other operands or in reverse, each
// gradient (linear_launch.h).
//
// One workgroup owns a (sequence or segment, head, block of 16 NW columns) and
// keeps its FP32 state in matrix accumulators: wave w holds columns 16w..16w+15
// of every 16-row state tile. A C-layout accumulator column is, unchanged, a B
// operand of the next product under the slot order of Mma<bf16_t>::kidx, so
// the state never leaves registers.
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

template <typename T, int PT_, int NW_, int OPL_>
struct WalkCfg {
  static constexpr bool F32 = sizeof(T) == 4;
  static constexpr int PT = PT_, NW = NW_, OPL = OPL_;
  static constexpr int IN = F32 ? 3 : 1;  // bf16 parts of an input
  static constexpr int C = (F32 || PT == 256) ? 32 : 64;
  static constexpr int NC = C / 16, KS = C / 32, PS = PT / 32, NT = PT / 16, QT = 16 * NW, THREADS = 64 * NW;
  // row strides: 16 bytes past a multiple of 256, so the 16 rows of an operand read lie in 16 bank groups
  static constexpr int LDX = PT + 8, LDW = QT + 8, LDP = C + 8, LDY = QT + 4;
  static constexpr int XPL = C * LDX, WPL = C * LDW, PPL = C * LDP;  // elements of one part
  static constexpr unsigned oX = 0, oZ = oX + 2u * IN * XPL, oW = oZ + 2u * IN * XPL, oP = oW + 2u * IN * WPL,
                            oY = oP + 2u * OPL * PPL, oTab = oY + 4u * C * LDY, oRed = oTab + 4u * 4 * 64 + 16,
                            total = oRed + 4u * 2 * NW + 16;
};

// Rows fetched into registers, written to LDS as bf16 parts.
template <typename T, int NT, int ROWS, int COLS>
struct PartsFetch : RowsFetch<T, NT, ROWS, COLS> {
  using Base = RowsFetch<T, NT, ROWS, COLS>;
  __device__ __forceinline__ void put_parts(bf16_t *s, int lds, int plane) const {
    if constexpr (sizeof(T) == 2) {
      Base::put(s, lds);
    } else {
#pragma unroll
      for (int it = 0; it < Base::IT; ++it) {
        const int idx = it * NT + tid_opaque();
        const int r = idx / Base::VPR, c = (idx % Base::VPR) * 4;
        if (Base::NV % NT == 0 || idx < Base::NV) {
          f32x4_t x = __builtin_bit_cast(f32x4_t, this->buf[it]);
#pragma unroll
          for (int pl = 0; pl < 3; ++pl) {
            const bf16x4_t h = to_bf16x4(x);
            *reinterpret_cast<bf16x4_t *>(s + pl * plane + r * lds + c) = h;
            x -= to_f32x4(h);
          }
        }
      }
    }
  }
};

// MODE 0: the whole walk; 1: the state only, left at the boundary behind the segment.
template <typename T, int PT, int NW, bool REV, int OPL, int MODE>
__global__ __launch_bounds__(64 * NW) void linear_walk_kernel(LinearWalk p) {
  using F = WalkCfg<T, PT, NW, OPL>;
  constexpr int C = F::C, NC = F::NC, KS = F::KS, IN = F::IN, QT = F::QT;
  extern __shared__ __align__(16) char smem[];
  bf16_t *sX = reinterpret_cast<bf16_t *>(smem + F::oX);
  bf16_t *sZ = reinterpret_cast<bf16_t *>(smem + F::oZ);
  bf16_t *sW = reinterpret_cast<bf16_t *>(smem + F::oW);
  bf16_t *sP = reinterpret_cast<bf16_t *>(smem + F::oP);
  float *sY = reinterpret_cast<float *>(smem + F::oY);
  float *sHi = reinterpret_cast<float *>(smem + F::oTab), *sLo = sHi + 64, *sA = sHi + 128, *sC = sHi + 192;
  float *sDec = sHi + 256;
  float *sRed = reinterpret_cast<float *>(smem + F::oRed);

  // Workgroups that read the same q/k rows (a group's heads, a head's column
  // blocks) go to one XCD, next to each other: ids are dealt to the eight XCDs
  // in turn.
  const int ncb = (p.Q + QT - 1) / QT;
  const int G = p.H / p.Hk, U = G * ncb;
  const int xcd = blockIdx.x & 7, sl = blockIdx.x >> 3;
  const int64_t unit = (int64_t)(sl / U) * 8 + xcd;
  const int member = sl % U;
  const int64_t item = unit / p.Hk;
  const int h = (int)(unit % p.Hk) * G + member / ncb, cb = member % ncb;
  SegLoc sg;
  const int64_t n_items = p.N + (p.seg ? ((int64_t)p.B * p.T) / p.seg : 0);
  if (item >= n_items || !locate_segment(p, item, REV, sg)) return;
  if (MODE == 1 && sg.out < 0) return;  // nothing follows the last segment

  const int tid = threadIdx.x, lane = tid & 63, wave = wave_id();
  const int grp = lane >> 4, l16 = lane & 15;
  const int P = p.P, Q = p.Q, col0 = cb * QT, ncol = min(QT, Q - col0);
  const int64_t rows = (int64_t)p.B * p.T;
  const int q = col0 + 16 * wave + l16;  // this lane's state column
  const int64_t frag = ((int64_t)h * ncb + cb) * (PT * QT) + ((int64_t)wave * F::NT * 64 + lane) * 4;
  const int64_t fragH = (int64_t)p.H * ncb * (PT * QT);  // elements of one boundary

  // ---- the state at the segment's start ----
  f32x4_t S[F::NT];
  const int64_t sbase = ((int64_t)sg.n * p.H + h) * P * Q;
  if (MODE == 0 && sg.in >= 0) {
    const float *src = p.seg_state + sg.in * fragH + frag;
#pragma unroll
    for (int t = 0; t < F::NT; ++t) S[t] = *reinterpret_cast<const f32x4_t *>(src + t * 256);
  } else if (MODE == 0 && p.seg_first && sg.out >= 0) {
    const float *src = p.seg_first + sg.n * fragH + frag;
#pragma unroll
    for (int t = 0; t < F::NT; ++t) S[t] = *reinterpret_cast<const f32x4_t *>(src + t * 256);
  } else {
    const bool from = p.s0 && sg.in < 0;
#pragma unroll
    for (int t = 0; t < F::NT; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = 16 * t + 4 * grp + e;
        S[t][e] = (from && r < P && q < Q) ? p.s0[sbase + r * p.sp + q * p.sq] : 0.f;
      }
    if (MODE == 1 && sg.in < 0 && p.seg_first) {
      float *dst = p.seg_first + sg.n * fragH + frag;
#pragma unroll
      for (int t = 0; t < F::NT; ++t) *reinterpret_cast<f32x4_t *>(dst + t * 256) = S[t];
    }
  }

  const float yscale = REV ? 1.f : p.scale, wscale = REV ? p.scale : 1.f;
  const int nch = (int)((sg.hi - sg.lo + C - 1) / C);
  PartsFetch<T, F::THREADS, C, PT> fx, fz;
  PartsFetch<T, F::THREADS, C, QT> fw;
  float fg = 0.f;
  double total = 0.0;  // log2 decay of the whole segment (wave 0)
  auto fetch = [&](int c) {
    const int64_t t0 = sg.lo + (int64_t)c * C;
    const int L = (int)min((int64_t)C, sg.hi - t0);
    if constexpr (MODE == 0)
      fx.fetch(reinterpret_cast<const T *>(p.x) + (t0 * p.Hx + h / (p.H / p.Hx)) * P, (int64_t)p.Hx * P, L, P);
    fz.fetch(reinterpret_cast<const T *>(p.z) + (t0 * p.Hz + h / (p.H / p.Hz)) * P, (int64_t)p.Hz * P, L, P);
    fw.fetch(reinterpret_cast<const T *>(p.w) + (t0 * p.Hw + h / (p.H / p.Hw)) * Q + col0, (int64_t)p.Hw * Q, L, ncol);
    if (wave == 0) fg = lane < L ? (p.g_head ? p.g[h] : p.g[(t0 + lane) * p.H + h]) : 0.f;
  };
  if (nch > 0) fetch(REV ? nch - 1 : 0);

  if constexpr (MODE == 0) {
    // the blocks of the scores beyond the triangle stay zero
    for (int i = tid; i < OPL * F::PPL / 2; i += F::THREADS) reinterpret_cast<unsigned *>(sP)[i] = 0u;
  }

  for (int cc = 0; cc < nch; ++cc) {
    const int c = REV ? nch - 1 - cc : cc;
    const int64_t t0 = sg.lo + (int64_t)c * C;
    const int L = (int)min((int64_t)C, sg.hi - t0);

    // ---- this chunk's rows and decays to LDS ----
    if constexpr (MODE == 0) fx.put_parts(sX, F::LDX, F::XPL);
    fz.put_parts(sZ, F::LDX, F::XPL);
    fw.put_parts(sW, F::LDW, F::WPL);
    if (wave == 0) {
      // b in fp64; a decay below 2^-160 is none at all and counts as 2^-32768:
      // differences across it give zero, those beyond it stay exact
      double b = (double)fg * 1.4426950408889634073599;
      if (b <= -160.0) b = -32768.0;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const double up = __shfl_up(b, off);
        if (lane >= off) b += up;
      }
      const double bl = __shfl(b, 63);
      const double hi = rint(b);
      const float first = fast_exp2((float)b), rest = fast_exp2((float)(bl - b));
      sHi[lane] = (float)hi;
      sLo[lane] = (float)(b - hi);
      sA[lane] = REV ? rest : first;
      sC[lane] = REV ? first * p.scale : rest;
      if (lane == 0) sDec[0] = fast_exp2((float)bl);
      total += bl;
    }
    if (MODE == 0 && REV && p.ckpt) {  // <h, dh> behind this chunk
      const int64_t end = t0 + L;
      if (end < sg.e && (end - sg.a) % p.anchor == 0) {
        const float *src = p.ckpt + (end / p.anchor) * fragH + frag;
        float d = 0.f;
#pragma unroll
        for (int t = 0; t < F::NT; ++t) {
          const f32x4_t x = *reinterpret_cast<const f32x4_t *>(src + t * 256);
#pragma unroll
          for (int e = 0; e < 4; ++e) d += x[e] * S[t][e];
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) d += __shfl_xor(d, off);
        if (lane == 0) sRed[wave] = d;
      }
    }
    __syncthreads();
    if (MODE == 0 && REV && p.ckpt && tid == 0) {
      const int64_t end = t0 + L;
      if (end < sg.e && (end - sg.a) % p.anchor == 0) {
        float d = 0.f;
#pragma unroll
        for (int w = 0; w < NW; ++w) d += sRed[w];
        p.anchor_dot[((end / p.anchor) * p.H + h) * ncb + cb] = d;
      }
    }
    if (cc + 1 < nch) fetch(REV ? c - 1 : c + 1);

    f32x4_t y[NC];
    if constexpr (MODE == 0) {
      // ---- scores of the causal 16 x 16 blocks, dealt to the waves ----
#pragma unroll
      for (int b0 = 0; b0 < NC * (NC + 1) / 2; b0 += NW) {
        const int blk = b0 + wave;
        if (blk < NC * (NC + 1) / 2) {
          const int i = blk < 1 ? 0 : (blk < 3 ? 1 : (blk < 6 ? 2 : 3)), j = blk - i * (i + 1) / 2;
          const int ri = REV ? j : i, cj = REV ? i : j;
          f32x4_t acc = zero4();
#pragma unroll
          for (int s = 0; s < F::PS; ++s) {
            bf16x8_t a[IN], bz[IN];
#pragma unroll
            for (int pl = 0; pl < IN; ++pl) {
              a[pl] = *reinterpret_cast<const bf16x8_t *>(sX + pl * F::XPL + (16 * ri + l16) * F::LDX + 32 * s + 8 * grp);
              bz[pl] = *reinterpret_cast<const bf16x8_t *>(sZ + pl * F::XPL + (16 * cj + l16) * F::LDX + 32 * s + 8 * grp);
            }
            acc = mma_parts(a, bz, acc);
          }
          const f32x4_t hr = *reinterpret_cast<const f32x4_t *>(sHi + 16 * ri + 4 * grp);
          const f32x4_t lr = *reinterpret_cast<const f32x4_t *>(sLo + 16 * ri + 4 * grp);
          const float hs = sHi[16 * cj + l16], ls = sLo[16 * cj + l16];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float d = REV ? (hs - hr[e]) + (ls - lr[e]) : (hr[e] - hs) + (lr[e] - ls);
            const int r = 4 * grp + e;
            const bool keep = i != j || (REV ? l16 >= r : l16 <= r);
            float v = keep ? acc[e] * fast_exp2(d) * wscale : 0.f;
#pragma unroll
            for (int pl = 0; pl < OPL; ++pl) {
              const bf16_t hv = static_cast<bf16_t>(v);
              sP[pl * F::PPL + (16 * ri + r) * F::LDP + 16 * cj + l16] = hv;
              v -= static_cast<float>(hv);
            }
          }
        }
      }
      // ---- y = a (x S) ----
#pragma unroll
      for (int i = 0; i < NC; ++i) y[i] = zero4();
#pragma unroll
      for (int s = 0; s < F::PS; ++s) {
        bf16x8_t sb[OPL];
        const float sv[8] = {S[2 * s][0], S[2 * s][1], S[2 * s][2], S[2 * s][3],
                             S[2 * s + 1][0], S[2 * s + 1][1], S[2 * s + 1][2], S[2 * s + 1][3]};
        split8<OPL>(sv, sb);
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          bf16x8_t a[IN];
#pragma unroll
          for (int pl = 0; pl < IN; ++pl) {
            const bf16_t *src = sX + pl * F::XPL + (16 * i + l16) * F::LDX + 32 * s + 4 * grp;
            a[pl] = join8(*reinterpret_cast<const bf16x4_t *>(src), *reinterpret_cast<const bf16x4_t *>(src + 16));
          }
          y[i] = mma_parts(a, sb, y[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < NC; ++i) y[i] *= *reinterpret_cast<const f32x4_t *>(sA + 16 * i + 4 * grp);
      __syncthreads();
    }

    // ---- w as an operand, and decayed to the chunk's end in three parts ----
    bf16x8_t wf[KS][IN], wc[KS][3];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int pl = IN - 1; pl >= 0; --pl) {
        wf[s][pl] = load_frag32(sW + pl * F::WPL, F::LDW, 32 * s, 16 * wave);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] += static_cast<float>(wf[s][pl][e]);
      }
      const f32x4_t c0 = *reinterpret_cast<const f32x4_t *>(sC + 32 * s + 4 * grp);
      const f32x4_t c1 = *reinterpret_cast<const f32x4_t *>(sC + 32 * s + 16 + 4 * grp);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] *= c0[e];
        x[e + 4] *= c1[e];
      }
      split8<3>(x, wc[s]);
    }

    if constexpr (MODE == 0) {
      // ---- y += scores w; staged for whole-row stores ----
#pragma unroll
      for (int i = 0; i < NC; ++i) {
#pragma unroll
        for (int s = REV ? i / 2 : 0; s <= (REV ? KS - 1 : i / 2); ++s) {
          bf16x8_t a[OPL];
#pragma unroll
          for (int pl = 0; pl < OPL; ++pl) {
            const bf16_t *src = sP + pl * F::PPL + (16 * i + l16) * F::LDP + 32 * s + 4 * grp;
            a[pl] = join8(*reinterpret_cast<const bf16x4_t *>(src), *reinterpret_cast<const bf16x4_t *>(src + 16));
          }
          y[i] = mma_parts(a, wf[s], y[i]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) sY[(16 * i + 4 * grp + e) * F::LDY + 16 * wave + l16] = y[i][e] * yscale;
      }
    }

    // ---- the state ----
    const float dec = sDec[0];
#pragma unroll
    for (int t = 0; t < F::NT; ++t) {
      S[t] *= dec;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        bf16x8_t a[IN];
#pragma unroll
        for (int pl = 0; pl < IN; ++pl) a[pl] = load_frag32(sZ + pl * F::XPL, F::LDX, 32 * s, 16 * t);
        S[t] = mma_parts(a, wc[s], S[t]);
      }
    }
    if (MODE == 0 && !REV && p.ckpt) {
      const int64_t end = t0 + L;
      if (end < sg.e && (end - sg.a) % p.anchor == 0) {
        float *dst = p.ckpt + (end / p.anchor) * fragH + frag;
#pragma unroll
        for (int t = 0; t < F::NT; ++t) *reinterpret_cast<f32x4_t *>(dst + t * 256) = S[t];
      }
    }
    __syncthreads();

    if constexpr (MODE == 0) {
      // ---- rows out, eight columns a thread, and their dots with u ----
      constexpr int TPR = QT / 8;
#pragma unroll
      for (int i0 = 0; i0 < C * TPR; i0 += F::THREADS) {
        const int idx = i0 + tid, r = idx / TPR, cq = 8 * (idx % TPR);
        const bool ok = r < L && cq < ncol;
        float v[8];
        *reinterpret_cast<f32x4_t *>(v) = *reinterpret_cast<const f32x4_t *>(sY + r * F::LDY + cq);
        *reinterpret_cast<f32x4_t *>(v + 4) = *reinterpret_cast<const f32x4_t *>(sY + r * F::LDY + cq + 4);
        const int64_t at = ((t0 + r) * p.H + h) * Q + col0 + cq;
        if (ok) {
          if constexpr (sizeof(T) == 2) {
            if (p.y_f32) {
              float *dst = reinterpret_cast<float *>(p.y) + at;
              *reinterpret_cast<f32x4_t *>(dst) = *reinterpret_cast<const f32x4_t *>(v);
              *reinterpret_cast<f32x4_t *>(dst + 4) = *reinterpret_cast<const f32x4_t *>(v + 4);
            } else {
              *reinterpret_cast<bf16x8_t *>(reinterpret_cast<bf16_t *>(p.y) + at) = pack_bf16x8(v);
            }
          } else {
            float *dst = reinterpret_cast<float *>(p.y) + at;
            *reinterpret_cast<f32x4_t *>(dst) = *reinterpret_cast<const f32x4_t *>(v);
            *reinterpret_cast<f32x4_t *>(dst + 4) = *reinterpret_cast<const f32x4_t *>(v + 4);
          }
        }
        if (p.u) {
          float d = 0.f;
          if (ok) {
            const T *us = reinterpret_cast<const T *>(p.u) + ((t0 + r) * p.Hu + h / (p.H / p.Hu)) * Q + col0 + cq;
#pragma unroll
            for (int e = 0; e < 8; ++e) d += v[e] * to_f32(us[e]);
          }
#pragma unroll
          for (int off = TPR / 2; off > 0; off >>= 1) d += __shfl_xor(d, off);
          if (ok && cq == 0) p.dot[((int64_t)cb * p.H + h) * rows + t0 + r] = d;
        }
      }
    }
  }

  if constexpr (MODE == 1) {
    float *dst = p.seg_state + sg.out * fragH + frag;
#pragma unroll
    for (int t = 0; t < F::NT; ++t) *reinterpret_cast<f32x4_t *>(dst + t * 256) = S[t];
    if (tid == 0 && cb == 0) p.seg_decay[sg.out * p.H + h] = total;
  } else if (sg.out < 0) {
    if (p.sT && !(nch == 0 && p.sT == p.s0)) {
#pragma unroll
      for (int t = 0; t < F::NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 16 * t + 4 * grp + e;
          if (r < P && q < Q) p.sT[sbase + r * p.sp + q * p.sq] = S[t][e];
        }
    }
    if (p.end_dot) {
      float d = 0.f;
#pragma unroll
      for (int t = 0; t < F::NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 16 * t + 4 * grp + e;
          if (r < P && q < Q) d += S[t][e] * p.s_dot[sbase + r * p.sp + q * p.sq];
        }
#pragma unroll
      for (int off = 32; off > 0; off >>= 1) d += __shfl_xor(d, off);
      __syncthreads();
      if (lane == 0) sRed[wave] = d;
      __syncthreads();
      if (tid == 0) {
        float s = 0.f;
        for (int w = 0; w < NW; ++w) s += sRed[w];
        p.end_dot[((int64_t)sg.n * p.H + h) * ncb + cb] = s;
      }
    }
  }
}

template <typename T, int PT, int NW, bool REV, int OPL, int MODE>
hipError_t launch_one(const LinearWalk &p, hipStream_t st) {
  using F = WalkCfg<T, PT, NW, OPL>;
  auto kern = linear_walk_kernel<T, PT, NW, REV, OPL, MODE>;
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kern), hipFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)F::total);
  if (e != hipSuccess) {
    (void)hipGetLastError();  // do not leave the error for the next launch to report
    return e;
  }
  const int ncb = (p.Q + F::QT - 1) / F::QT;
  const int64_t items = p.N + (p.seg ? ((int64_t)p.B * p.T) / p.seg : 0);
  const int64_t grid = (items * p.Hk + 7) / 8 * 8 * (p.H / p.Hk) * ncb;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(F::THREADS), F::total, st, p);
  return hipGetLastError();
}

template <typename T, int PT, int NW, bool REV, int OPL>
hipError_t launch_modes(const LinearWalk &p, hipStream_t st) {
  if (p.seg) {
    hipError_t e = launch_one<T, PT, NW, REV, 1, 1>(p, st);
    if (e != hipSuccess) return e;
    const int ncb = (p.Q + 16 * NW - 1) / (16 * NW);
    if ((e = launch_linear_chain(p, REV, (int64_t)ncb * PT * 16 * NW, st)) != hipSuccess) return e;
  }
  return launch_one<T, PT, NW, REV, OPL, 0>(p, st);
}

template <typename T, int PT, bool REV, int OPL>
hipError_t launch_cols(const LinearWalk &p, hipStream_t st) {
  int ncb;
  if (linear_cols(p.Q, &ncb) == 64) return launch_modes<T, PT, 4, REV, OPL>(p, st);
  return launch_modes<T, PT, 8, REV, OPL>(p, st);
}

template <typename T, bool REV, int OPL>
hipError_t launch_width(const LinearWalk &p, hipStream_t st) {
  switch (linear_tile(p.P)) {
    case 64: return launch_cols<T, 64, REV, OPL>(p, st);
    case 128: return launch_cols<T, 128, REV, OPL>(p, st);
    default: return launch_cols<T, 256, REV, OPL>(p, st);
  }
}

}  // namespace

}  // namespace kda
