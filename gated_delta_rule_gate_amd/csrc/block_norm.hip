// The norms round an attention block (include/kda_norm.h), forward and
// backward:
//
//   n = w x rho,  rho = (mean x^2 + eps)^-1/2 (L2: sum);   y = res + s n act(gate)
//   z = w2 y rho2,  rho2 = (mean y^2 + eps)^-1/2
//
// and, with t the total gradient of y,
//
//   t  = dy + rho2 (w2 dz - y rho2^2 mean(w2 dz y))
//   dres = t,  dgate = s t n act'(gate),  dn = s t act(gate)
//   dx = rho (w dn - x rho^2 mean(w dn x))       (L2: sum)
//   dw = sum over rows of dn x rho,  ds = of t n act(gate),  dw2 = of dz y rho2
//
// Bound by the bytes of the rows: each input is read once into registers, the
// row sums are taken there, and each output is written once. A row of D values
// is held by LPR lanes of eight values each: up to 512 values by part of a wave
// or a wave (no barrier), longer rows by a whole workgroup of 128 to 512
// threads, which past 4096 values take two or four vectors a lane (NV).
// Parameter gradients stay in registers while a workgroup walks its rows; its
// sums go to the workspace and are added over workgroups in order.
// Forward 1048576 x 128 with a gate, bf16: 140 us, 5.7 TB/s. Backward 262144 x
// 128 with a gate: 84 us, 4.0 TB/s; 8192 x 4096 with gate, residual, channel
// scale and next norm: 115 us, 4.6 TB/s; 8192 x 8192: 321 us, 3.3 TB/s. Past
// 8192 columns the backward spills 50 to 310 registers a lane (4096 x 16384: 920
// us, 1.2 TB/s), and in fp32 with the next norm 28 past 4096 (8192 x 8192: 630
// us, 3.4 TB/s).
#include "kda_device.h"
#include "linear_launch.h"

namespace kda {

namespace {

template <typename T>
__device__ __forceinline__ void load8(const void *p, int64_t at, float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    const bf16x8_t v = *reinterpret_cast<const bf16x8_t *>(reinterpret_cast<const bf16_t *>(p) + at);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = static_cast<float>(v[e]);
  } else {
    const f32x4_t *v = reinterpret_cast<const f32x4_t *>(reinterpret_cast<const float *>(p) + at);
    const f32x4_t a = v[0], b = v[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = a[e];
      x[e + 4] = b[e];
    }
  }
}
template <typename T>
__device__ __forceinline__ void store8(void *p, int64_t at, const float (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<bf16x8_t *>(reinterpret_cast<bf16_t *>(p) + at) = pack_bf16x8(x);
  } else {
    f32x4_t *v = reinterpret_cast<f32x4_t *>(reinterpret_cast<float *>(p) + at);
    v[0] = f32x4_t{x[0], x[1], x[2], x[3]};
    v[1] = f32x4_t{x[4], x[5], x[6], x[7]};
  }
}
__device__ __forceinline__ void fill8(float (&x)[8], float v) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = v;
}

// Sums of a row's lanes: within the wave by shuffles, over a workgroup's waves
// through LDS (two buffers in turn, so one barrier a sum is enough).
constexpr int block_threads(int lpr) { return lpr >= 128 ? lpr : 256; }

template <int LPR, int NS>
__device__ __forceinline__ void row_sums(float (&s)[NS], float (*red)[2][16], int &turn) {
#pragma unroll
  for (int off = (LPR < 64 ? LPR : 64) / 2; off > 0; off >>= 1)
#pragma unroll
    for (int i = 0; i < NS; ++i) s[i] += __shfl_xor(s[i], off);
  if constexpr (LPR > 64) {
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < NS; ++i) red[turn][i][wave] = s[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      s[i] = 0.f;
#pragma unroll
      for (int w = 0; w < LPR / 64; ++w) s[i] += red[turn][i][w];
    }
    turn ^= 1;
  }
}

__device__ __forceinline__ float act_of(bool silu, float g) {
  const float s = sigmoid_f32(g);
  return silu ? g * s : s;
}

template <typename Tx, typename Tr, int LPR, int NV>
__global__ __launch_bounds__(block_threads(LPR)) void block_norm_fwd_kernel(BlockNorm p) {
  constexpr int RPB = block_threads(LPR) / LPR;  // rows of a workgroup at a time
  __shared__ float red[2][2][16];
  int turn = 0;
  const int lane = threadIdx.x % LPR;
  const float inv = p.l2 ? 1.0f : 1.0f / (float)p.D, inv2 = 1.0f / (float)p.D;
  for (int64_t row0 = (int64_t)blockIdx.x * RPB; row0 < p.rows; row0 += (int64_t)gridDim.x * RPB) {
    const int64_t row = row0 + threadIdx.x / LPR;
    const bool live = row < p.rows;
    const int64_t base = row * p.D;
    float x[NV][8], gt[NV][8], y[NV][8];
    float s[1] = {0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * LPR + lane) * 8;
      const bool ok = live && c < p.D;
      fill8(x[v], 0.f);
      fill8(gt[v], 0.f);
      fill8(y[v], 0.f);
      if (ok) {
        load8<Tx>(p.x, base + c, x[v]);
        if (p.gate) load8<Tx>(p.gate, base + c, gt[v]);
        if (p.residual) load8<Tr>(p.residual, base + c, y[v]);
      }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += x[v][e] * x[v][e];
    row_sums<LPR, 1>(s, red, turn);
    const float rho = 1.0f / sqrtf(s[0] * inv + p.eps);
    float s2[1] = {0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * LPR + lane) * 8;
      if (!live || c >= p.D) continue;
      float w[8], sc[8];
      if (p.weight) load8<float>(p.weight, c, w);
      else fill8(w, 1.f);
      if (p.scale_vec) load8<float>(p.scale_vec, c, sc);
      else fill8(sc, p.scale);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float n = x[v][e] * rho * w[e];
        if (p.gate) n *= act_of(p.silu, gt[v][e]);
        y[v][e] += n * sc[e];
        s2[0] += y[v][e] * y[v][e];
      }
      store8<Tr>(p.y, base + c, y[v]);
    }
    if (!p.z) continue;
    row_sums<LPR, 1>(s2, red, turn);
    const float rho2 = 1.0f / sqrtf(s2[0] * inv2 + p.eps);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = (v * LPR + lane) * 8;
      if (!live || c >= p.D) continue;
      float w[8];
      if (p.next_weight) load8<float>(p.next_weight, c, w);
      else fill8(w, 1.f);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] *= y[v][e] * rho2;
      store8<Tx>(p.z, base + c, w);
    }
  }
}

// Eight values as they lie in memory.
template <typename T>
struct Raw8 {
  u32x4_t v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const void *p, int64_t at) {
    const u32x4_t *src = reinterpret_cast<const u32x4_t *>(reinterpret_cast<const T *>(p) + at);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v[i] = src[i];
  }
  // hides the value's origin, so that its uses on either side are converted apart
  __device__ __forceinline__ void renew() {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) asm volatile("" : "+v"(v[i]));
  }
  __device__ __forceinline__ void keep(bool ok) {  // or zeros
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) v[i] = ok ? v[i] : u32x4_t{0u, 0u, 0u, 0u};
  }
  __device__ __forceinline__ void get(float (&x)[8], bool ok) const {  // zeros where !ok
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      unsigned u;
      if constexpr (sizeof(T) == 2) u = e & 1 ? v[0][e / 2] & 0xffff0000u : v[0][e / 2] << 16;
      else u = v[e / 4][e % 4];
      x[e] = __uint_as_float(ok ? u : 0u);
    }
  }
};

// The next rows' loads are in flight while a workgroup computes on its rows:
// with the registers this takes, few waves share a SIMD, and their number alone
// does not cover the loads (262144 x 128 with a SiLU gate: 169 us without).
template <typename Tx, typename Tr, int LPR, int NV, bool NEXT>
__global__ __launch_bounds__(block_threads(LPR)) void block_norm_bwd_kernel(BlockNorm p) {
  constexpr int RPB = block_threads(LPR) / LPR;
  __shared__ float red[2][2][16];
  int turn = 0;
  const int lane = threadIdx.x % LPR;
  const float inv = p.l2 ? 1.0f : 1.0f / (float)p.D, inv2 = 1.0f / (float)p.D;
  const bool has_dy = p.dy, has_gate = p.gate, has_res = p.residual;
  float aw[NV][8], as[NV][8], an[NEXT ? NV : 1][8];  // sums over this lane's rows
  // One vector a lane leaves registers for the next rows and for the weights;
  // with more, weights come from the cache for every use, and inputs stay as
  // they lie in memory until used.
  constexpr bool AHEAD = NV == 1;
  float kw[AHEAD ? 3 : 1][8];
  auto weight_of = [&](int i, int v, float(&o)[8]) {  // 0: weight, 1: scale, 2: next weight
    const float *const src[3] = {p.weight, p.scale_vec, p.next_weight};
    fill8(o, i == 1 ? p.scale : 1.f);
    if (src[i]) load8<float>(src[i], min((v * LPR + lane) * 8, p.D - 8), o);
  };
  auto weight = [&](int i, int v, float(&o)[8]) {
    if constexpr (AHEAD) {
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = kw[i][e];
    } else {
      weight_of(i, v, o);
    }
  };
  if constexpr (AHEAD) {
#pragma unroll
    for (int i = 0; i < (NEXT ? 3 : 2); ++i) weight_of(i, 0, kw[i]);
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    fill8(aw[v], 0.f);
    fill8(as[v], 0.f);
    if constexpr (NEXT) fill8(an[v], 0.f);
  }
  Raw8<Tx> rx[NV], rg[NV], rz[NEXT ? NV : 1];
  Raw8<Tr> rt[NV], rr[NEXT ? NV : 1];
  auto fetch = [&](int64_t row0) {  // rows and columns past the end repeat the last
    const int64_t base = min(row0 + threadIdx.x / LPR, p.rows - 1) * p.D;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int64_t at = base + min((v * LPR + lane) * 8, p.D - 8);
      rx[v].load(p.x, at);
      if (has_gate) rg[v].load(p.gate, at);
      if (has_dy) rt[v].load(p.dy, at);
      if constexpr (NEXT) {
        rz[v].load(p.dz, at);
        if (has_res) rr[v].load(p.residual, at);
      }
    }
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row0 = (int64_t)blockIdx.x * RPB;
  if (AHEAD && row0 < p.rows) fetch(row0);
  for (; row0 < p.rows; row0 += step) {
    if constexpr (!AHEAD) fetch(row0);
    const int64_t row = row0 + threadIdx.x / LPR;
    const bool live = RPB == 1 || row < p.rows;
    const int64_t base = row * p.D;
    Raw8<Tx> cx[NV], cg[NV], cz[NEXT ? NV : 1];
    float t[NV][8], y[NEXT ? NV : 1][8];
    bool ok[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      ok[v] = live && (v * LPR + lane) * 8 < p.D;
      cx[v] = rx[v];
      cg[v] = rg[v];
      if constexpr (sizeof(Tx) == 2) cg[v].keep(ok[v]);
      rt[v].get(t[v], ok[v] && has_dy);
      if constexpr (NEXT) {
        cz[v] = rz[v];
        rr[v].get(y[v], ok[v] && has_res);
      }
    }
    if (AHEAD && row0 + step < p.rows) fetch(row0 + step);

    // Past the last row and column every input is taken as zero, and a row there has
    // no norm: with eps = 0 its statistic would be infinite, and its zeros NaN, which
    // the parameters' sums would keep. (A bf16 gate is zeroed as it lies in memory, an
    // fp32 gate where it is used: 8192 x 8192 with every part, bf16 323 us against 328
    // the other way, fp32 628 us against 668.)
    auto norm_of = [&](float mean) { return live ? 1.0f / sqrtf(mean + p.eps) : 0.f; };
    // act(gate) and its derivative; no gate: 1 and 0
    auto gate = [&](int v, float(&act)[8], float(&dact)[8]) {
      cg[v].get(act, has_gate && (sizeof(Tx) == 2 || ok[v]));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float g = act[e], sg = sigmoid_f32(g), ds = sg * (1.0f - sg);
        act[e] = !has_gate ? 1.f : (p.silu ? g * sg : sg);
        dact[e] = p.silu ? sg + g * ds : ds;
      }
    };
    // between the passes over a row, wide rows keep neither converted inputs nor
    // weights: held, they spill (8192 x 8192: 850 us)
    auto apart = [&]() {
      if constexpr (AHEAD) return;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        cx[v].renew();
        cg[v].renew();
        if constexpr (NEXT) cz[v].renew();
      }
      asm volatile("" ::: "memory");
    };
    float rho = 0.f;
    if constexpr (NEXT) {
      float s[1] = {0.f};
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float x[8];
        cx[v].get(x, ok[v]);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] += x[e] * x[e];
      }
      row_sums<LPR, 1>(s, red, turn);
      rho = norm_of(s[0] * inv);
      apart();
      float s2[2] = {0.f, 0.f};
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float x[8], w[8], sc[8], w2[8], act[8], dact[8], dz[8];
        cx[v].get(x, ok[v]);
        cz[v].get(dz, ok[v]);
        weight(0, v, w);
        weight(1, v, sc);
        weight(2, v, w2);
        gate(v, act, dact);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          y[v][e] += x[e] * rho * w[e] * act[e] * sc[e];
          s2[0] += y[v][e] * y[v][e];
          s2[1] += y[v][e] * dz[e] * w2[e];
        }
      }
      row_sums<LPR, 2>(s2, red, turn);
      const float rho2 = norm_of(s2[0] * inv2), m = s2[1] * inv2 * rho2 * rho2;
      apart();
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float w2[8], dz[8];
        cz[v].get(dz, ok[v]);
        weight(2, v, w2);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          an[v][e] += dz[e] * y[v][e] * rho2;
          t[v][e] += rho2 * (dz[e] * w2[e] - y[v][e] * m);
        }
      }
    }
    // t is the whole gradient of y from here on
    apart();
    float s3[2] = {0.f, 0.f};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float x[8], w[8], sc[8], act[8], dact[8];
      cx[v].get(x, ok[v]);
      weight(0, v, w);
      weight(1, v, sc);
      gate(v, act, dact);
      if (p.dresidual && ok[v]) store8<Tr>(p.dresidual, base + (v * LPR + lane) * 8, t[v]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        s3[0] += x[e] * x[e];
        s3[1] += t[v][e] * sc[e] * act[e] * x[e] * w[e];
      }
    }
    row_sums<LPR, 2>(s3, red, turn);
    if constexpr (!NEXT) rho = norm_of(s3[0] * inv);
    const float m = s3[1] * inv * rho * rho;
    apart();
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float x[8], w[8], sc[8], act[8], dact[8], dg[8], dx[8];
      cx[v].get(x, ok[v]);
      weight(0, v, w);
      weight(1, v, sc);
      gate(v, act, dact);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xr = x[e] * rho, n = xr * w[e], dn = t[v][e] * sc[e] * act[e];
        aw[v][e] += dn * xr;
        as[v][e] += t[v][e] * n * act[e];
        dg[e] = t[v][e] * sc[e] * n * dact[e];
        dx[e] = rho * (dn * w[e] - x[e] * m);
      }
      if (ok[v]) {
        if (p.dgate) store8<Tx>(p.dgate, base + (v * LPR + lane) * 8, dg);
        store8<Tx>(p.dx, base + (v * LPR + lane) * 8, dx);
      }
    }
  }

  // ---- parameter gradients: rows of this workgroup, then the workspace ----
  float *part = p.part + (int64_t)blockIdx.x * 3 * p.D;
  __shared__ float sums[RPB > 1 ? 256 : 1][8];
  float *const wanted[3] = {p.dweight, p.dscale_vec, p.dnext_weight};
#pragma unroll
  for (int i = 0; i < (NEXT ? 3 : 2); ++i) {
    if (!wanted[i]) continue;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      float(&a)[8] = i == 0 ? aw[v] : (i == 1 ? as[v] : an[NEXT ? v : 0]);
      const int c = (v * LPR + lane) * 8;
      if constexpr (RPB > 1) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[threadIdx.x][e] = a[e];
        __syncthreads();
        if ((int)threadIdx.x < LPR && c < p.D) {
          for (int r = 1; r < RPB; ++r)
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] += sums[r * LPR + threadIdx.x][e];
          store8<float>(part, (int64_t)i * p.D + c, a);
        }
      } else if (c < p.D) {
        store8<float>(part, (int64_t)i * p.D + c, a);
      }
    }
  }
}

// Sums over the workgroups' parts in a fixed order: 64 columns a workgroup,
// sixteen waves each taking every sixteenth part, eight parts in flight (one
// part at a time, a wave's loads alone took 60 us for 1024 parts).
__global__ __launch_bounds__(1024) void block_norm_params_kernel(BlockNorm p, int blocks) {
  __shared__ double red[16][64];
  float *const wanted[3] = {p.dweight, p.dscale_vec, p.dnext_weight};
  float *out = wanted[blockIdx.y];
  if (!out) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane;
  const float *src = p.part + (int64_t)blockIdx.y * p.D + min(c, p.D - 1);
  double s = 0.0;
  for (int b = wave; b < blocks; b += 128) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = src[(int64_t)min(b + 16 * i, blocks - 1) * 3 * p.D];
#pragma unroll
    for (int i = 0; i < 8; ++i) s += b + 16 * i < blocks ? (double)v[i] : 0.0;
  }
  red[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < p.D) {
    for (int w = 1; w < 16; ++w) s += red[w][lane];
    out[c] = (float)s;
  }
}

// Lanes a row.
int row_lanes(int D) {
  int lpr = 1;
  while (lpr < 512 && lpr * 8 < D) lpr *= 2;
  return lpr;
}

// Workgroups of the backward: enough to fill the device, few enough that their
// parts stay small beside the rows.
int bwd_blocks(int64_t rows, int D) {
  const int lpr = row_lanes(D), rpb = block_threads(lpr) / lpr;
  const int64_t need = (rows + rpb - 1) / rpb;
  const int64_t most = (int64_t)device_cus() * (D > 4096 ? 1 : (D > 512 ? 1024 / lpr : 4));
  return (int)(need < most ? (need > 0 ? need : 1) : most);
}

template <typename Tx, typename Tr, int LPR, int NV>
hipError_t launch_nv(const BlockNorm &p, bool bwd, hipStream_t st) {
  constexpr int RPB = block_threads(LPR) / LPR;
  const int64_t need = (p.rows + RPB - 1) / RPB;
  if (bwd) {
    const int blocks = bwd_blocks(p.rows, p.D);
    if (p.dz || p.dnext_weight)  // without rows dz has no address, and dnext_weight is zero
      hipLaunchKernelGGL((block_norm_bwd_kernel<Tx, Tr, LPR, NV, true>), dim3(blocks), dim3(block_threads(LPR)), 0, st, p);
    else
      hipLaunchKernelGGL((block_norm_bwd_kernel<Tx, Tr, LPR, NV, false>), dim3(blocks), dim3(block_threads(LPR)), 0, st, p);
  } else {
    if (need == 0) return hipSuccess;
    const int64_t most = most_blocks(block_threads(LPR)), grid = need < most ? need : most;
    hipLaunchKernelGGL((block_norm_fwd_kernel<Tx, Tr, LPR, NV>), dim3((unsigned)grid), dim3(block_threads(LPR)), 0, st, p);
  }
  return hipGetLastError();
}

template <typename Tx, typename Tr>
hipError_t launch_rows(const BlockNorm &p, bool bwd, hipStream_t st) {
  switch (row_lanes(p.D)) {
    case 1: return launch_nv<Tx, Tr, 1, 1>(p, bwd, st);
    case 2: return launch_nv<Tx, Tr, 2, 1>(p, bwd, st);
    case 4: return launch_nv<Tx, Tr, 4, 1>(p, bwd, st);
    case 8: return launch_nv<Tx, Tr, 8, 1>(p, bwd, st);
    case 16: return launch_nv<Tx, Tr, 16, 1>(p, bwd, st);
    case 32: return launch_nv<Tx, Tr, 32, 1>(p, bwd, st);
    case 64: return launch_nv<Tx, Tr, 64, 1>(p, bwd, st);
    case 128: return launch_nv<Tx, Tr, 128, 1>(p, bwd, st);
    case 256: return launch_nv<Tx, Tr, 256, 1>(p, bwd, st);
    default:
      if (p.D <= 4096) return launch_nv<Tx, Tr, 512, 1>(p, bwd, st);
      return p.D <= 8192 ? launch_nv<Tx, Tr, 512, 2>(p, bwd, st) : launch_nv<Tx, Tr, 512, 4>(p, bwd, st);
  }
}

hipError_t launch_types(const BlockNorm &p, bool bwd, hipStream_t st) {
  if (!p.is_bf16) return launch_rows<float, float>(p, bwd, st);
  return p.res_f32 ? launch_rows<bf16_t, float>(p, bwd, st) : launch_rows<bf16_t, bf16_t>(p, bwd, st);
}

}  // namespace

size_t block_norm_bwd_part_bytes(int64_t rows, int D) {
  return (size_t)bwd_blocks(rows, D) * 3 * (size_t)D * sizeof(float);
}

hipError_t launch_block_norm_fwd(const BlockNorm &p, hipStream_t st) { return launch_types(p, false, st); }

hipError_t launch_block_norm_bwd(const BlockNorm &p, hipStream_t st) {
  hipError_t e = launch_types(p, true, st);
  if (e != hipSuccess || !(p.dweight || p.dscale_vec || p.dnext_weight)) return e;
  hipLaunchKernelGGL(block_norm_params_kernel, dim3((p.D + 63) / 64, 3), dim3(1024), 0, st, p,
                     bwd_blocks(p.rows, p.D));
  return hipGetLastError();
}

}  // namespace kda
