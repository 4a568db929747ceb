// Token-sequential linear attention with one decay per head (decoding).
//
// One workgroup of 256 threads owns a (sequence, head, block of BV value
// columns) and scans its tokens with the [K, BV] FP32 state in registers:
//
//   S = 2^a S + k v^T,     o = scale S^T q.
//
// Bound by the state's bytes, read and written once. A thread holds RPT rows
// of four adjacent columns, so a wave's 16-byte state accesses cover whole
// runs of a row; they bypass the caches' retention (touched once a call).
// A column's sum over K runs over the lanes that share it, then over the four
// waves through LDS. Column blocks of 128 read the state in its own order;
// where those would leave compute units idle, blocks of 32 spread a (sequence,
// head) over four times the workgroups. 256 sequences, 64 heads, 128 x 128, one
// token: 376 us, 5.76 TB/s (an in-place scaling reaches 5.9); one sequence of 16
// heads: 4 us.
#include "kda_device.h"
#include "linear_launch.h"

namespace kda {

namespace {

__device__ __forceinline__ f32x4_t load_once(const float *p) {
  return __builtin_nontemporal_load(reinterpret_cast<const f32x4_t *>(p));
}
__device__ __forceinline__ void store_once(float *p, f32x4_t v) {
  __builtin_nontemporal_store(v, reinterpret_cast<f32x4_t *>(p));
}

// FULL: K == KP and V a multiple of BV: no masks. ONE: every sequence has one
// token (a dense decode step): no loop and nothing prefetched, so fewer
// registers and more workgroups a compute unit.
template <typename T, int KP, int BV, bool FULL, bool ONE>
__global__ __launch_bounds__(256) void linear_recurrent_kernel(LinearRecurrent p) {
  constexpr int CG = BV / 4, RG = 256 / CG, RPT = KP / RG;
  static_assert(256 % CG == 0 && KP % RG == 0 && CG <= 64, "tile");
  const int K = FULL ? KP : p.K;
  const int nvb = FULL ? p.V / BV : (p.V + BV - 1) / BV;
  const int vb = blockIdx.x % nvb;
  const int nh = blockIdx.x / nvb;
  const int n = nh / p.H, h = nh % p.H, hk = h / (p.H / p.Hk);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int cg = tid % CG, rg = tid / CG, row0 = rg * RPT, col0 = vb * BV + cg * 4;
  const bool col_ok = FULL || col0 < p.V;
  SlotRange sr = slot_range(ONE ? nullptr : p.cu, n, ONE ? 1 : p.T);
  const int64_t sbase = (int64_t)(n * (int64_t)p.H + h) * K * p.V;

  const T *qp = reinterpret_cast<const T *>(p.q), *kp = reinterpret_cast<const T *>(p.k);
  const T *vp = reinterpret_cast<const T *>(p.v);
  T *op = reinterpret_cast<T *>(p.o);

  float nk = 0.f, nq = 0.f, nv = 0.f, ng = 0.f;  // the next token's inputs
  auto fetch = [&](int i) {
    const int64_t t = sr.t0 + i;
    if (tid < K) {
      nk = to_f32(kp[(t * p.Hk + hk) * K + tid]);
      nq = to_f32(qp[(t * p.Hk + hk) * K + tid]);
    }
    if (tid < BV && (FULL || vb * BV + tid < p.V)) nv = to_f32(vp[(t * p.H + h) * p.V + vb * BV + tid]);
    ng = p.g_head ? p.g[h] : p.g[t * p.H + h];
  };
  if (sr.len > 0) fetch(0);

  f32x4_t S[RPT];
#pragma unroll
  for (int r = 0; r < RPT; ++r)
    S[r] = (p.h0 && (FULL || (col_ok && row0 + r < K))) ? load_once(p.h0 + sbase + (int64_t)(row0 + r) * p.V + col0)
                                                        : f32x4_t{0.f, 0.f, 0.f, 0.f};

  __shared__ float s_k[2][KP], s_q[2][KP];
  __shared__ __align__(16) float s_v[2][BV];
  __shared__ __align__(16) float s_red[2][4][BV];
  for (int i = 0; i < sr.len; ++i) {
    const int buf = i & 1;
    if (tid < KP) {  // channels past K hold zeros
      s_k[buf][tid] = nk;
      s_q[buf][tid] = nq;
    }
    if (tid < BV) s_v[buf][tid] = nv;
    const float a = fast_exp2(ng * kLog2e);
    if (!ONE && i + 1 < sr.len) fetch(i + 1);
    __syncthreads();
    const f32x4_t v4 = *reinterpret_cast<const f32x4_t *>(&s_v[buf][cg * 4]);
    f32x4_t o4 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < RPT; ++r) {
      S[r] = S[r] * a + s_k[buf][row0 + r] * v4;
      o4 += S[r] * s_q[buf][row0 + r];
    }
#pragma unroll
    for (int off = CG; off < 64; off <<= 1)
#pragma unroll
      for (int e = 0; e < 4; ++e) o4[e] += __shfl_xor(o4[e], off);
    if (lane < CG) *reinterpret_cast<f32x4_t *>(&s_red[buf][wave][cg * 4]) = o4;
    __syncthreads();
    if (tid < BV && (FULL || vb * BV + tid < p.V)) {
      const float s = (s_red[buf][0][tid] + s_red[buf][1][tid]) + (s_red[buf][2][tid] + s_red[buf][3][tid]);
      op[((sr.t0 + i) * p.H + h) * p.V + vb * BV + tid] = from_f32<T>(p.scale * s);
    }
  }
  if (p.ht && !(sr.len == 0 && p.ht == p.h0)) {
#pragma unroll
    for (int r = 0; r < RPT; ++r)
      if (FULL || (col_ok && row0 + r < K)) store_once(p.ht + sbase + (int64_t)(row0 + r) * p.V + col0, S[r]);
  }
}

template <typename T, int KP, int BV>
hipError_t launch_rec(const LinearRecurrent &p, hipStream_t st) {
  const int64_t grid = (int64_t)p.N * p.H * ((p.V + BV - 1) / BV);
  if (grid == 0) return hipSuccess;
  if (grid > most_blocks(256)) return hipErrorInvalidValue;
  const bool full = p.K == KP && p.V % BV == 0, one = !p.cu && p.T == 1;
  auto kern = full ? (one ? linear_recurrent_kernel<T, KP, BV, true, true> : linear_recurrent_kernel<T, KP, BV, true, false>)
                   : (one ? linear_recurrent_kernel<T, KP, BV, false, true> : linear_recurrent_kernel<T, KP, BV, false, false>);
  hipLaunchKernelGGL(kern, dim3((unsigned)grid), dim3(256), 0, st, p);
  return hipGetLastError();
}

template <typename T, int KP>
hipError_t launch_rec_k(const LinearRecurrent &p, hipStream_t st) {
  if ((int64_t)p.N * p.H * ((p.V + 127) / 128) < 2 * device_cus()) return launch_rec<T, KP, 32>(p, st);
  return launch_rec<T, KP, 128>(p, st);
}

template <typename T>
hipError_t launch_rec_t(const LinearRecurrent &p, hipStream_t st) {
  if (p.K <= 64) return launch_rec_k<T, 64>(p, st);
  if (p.K <= 128) return launch_rec_k<T, 128>(p, st);
  return launch_rec_k<T, 256>(p, st);
}

}  // namespace

// (blocks of 32 columns are for launches far below the limit)
bool linear_recurrent_fits(const LinearRecurrent &p) {
  return (int64_t)p.N * p.H * ((p.V + 127) / 128) <= most_blocks(256);
}

hipError_t launch_linear_recurrent(const LinearRecurrent &p, hipStream_t st) {
  return p.is_bf16 ? launch_rec_t<bf16_t>(p, st) : launch_rec_t<float>(p, st);
}

}  // namespace kda
