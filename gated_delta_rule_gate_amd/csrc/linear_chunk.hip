// Linear attention with one decay per head: the passes round the chunk walk
// (linear_walk.h) -- chaining segments, summing the gradients of shared q/k
// heads, the decay's gradient -- and the choice of segments.
#include <algorithm>
#include <cmath>

#include "chunk_fused_tiles.h"
#include "linear_launch.h"
#include "linear_segments.h"

namespace kda {

namespace {

// The segments' own state changes chained into the state at every boundary, in
// place and in the walk's order: S_j += 2^{decay of the segment before j} S_{j-1}.
// Four elements a thread; a boundary's next state is in flight while one is added.
// Bound by the states' bytes, read and written once: 10 us for 15 boundaries of 16
// heads, 128 x 128 (31 MB), half of it the launch and the serial chain.
__global__ __launch_bounds__(256) void linear_chain_kernel(LinearWalk p, bool rev, int64_t elems) {
  const int64_t per = (elems / 4 + 255) / 256;
  const int n = (int)(blockIdx.x / (per * p.H));
  const int h = (int)(blockIdx.x / per % p.H);
  const int64_t el = ((int64_t)(blockIdx.x % per) * 256 + threadIdx.x) * 4;
  const SlotRange sr = slot_range(p.cu, n, p.T);
  const int64_t nb = sr.len > 0 ? (sr.len - 1) / p.seg : 0;  // boundaries inside the sequence
  if (nb < 2 || el >= elems) return;
  const int64_t first = sr.t0 / p.seg + 1, step = (int64_t)p.H * elems;
  float *at = p.seg_state + (int64_t)h * elems + el;
  int64_t j = rev ? first + nb - 1 : first;
  const int64_t d = rev ? -1 : 1;
  f32x4_t s = *reinterpret_cast<const f32x4_t *>(at + j * step);
  f32x4_t next = *reinterpret_cast<const f32x4_t *>(at + (j + d) * step);
  for (int64_t i = 1; i < nb; ++i) {
    j += d;
    const f32x4_t own = next;
    if (i + 1 < nb) next = *reinterpret_cast<const f32x4_t *>(at + (j + d) * step);
    const float f = fast_exp2((float)p.seg_decay[j * p.H + h]);
    s = own + f * s;
    *reinterpret_cast<f32x4_t *>(at + j * step) = s;
  }
}

// Gradients of shared q/k heads: the group's fp32 parts added in order. Bound by
// bytes: 6 us for 4999 tokens of 16 heads on 8, 64 wide (26 MB).
template <typename T>
__global__ __launch_bounds__(256) void linear_group_sum_kernel(const float *in, T *out, const int32_t *cu, int N,
                                                               int64_t rows, int H, int Hk, int D) {
  const int G = H / Hk;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // of [rows, Hk, D / 4]
  const int64_t rk = i / (D / 4), row = rk / Hk;
  if (row >= rows) return;
  if (cu && (row < cu[0] || row >= cu[N])) return;
  const float *src = in + (rk * G) * D + (i % (D / 4)) * 4;
  f32x4_t s = *reinterpret_cast<const f32x4_t *>(src);
  for (int g = 1; g < G; ++g) s += *reinterpret_cast<const f32x4_t *>(src + (int64_t)g * D);
  T *dst = out + rk * D + (i % (D / 4)) * 4;
  if constexpr (sizeof(T) == 2) *reinterpret_cast<bf16x4_t *>(dst) = to_bf16x4(s);
  else *reinterpret_cast<f32x4_t *>(dst) = s;
}

// dg over one anchored stretch of one (sequence, head): a wave takes the
// stretch, a lane kDgPer neighbouring tokens, all of one chunk; sums in fp64.
// Each token's value comes from the side whose squares add up to less: a large
// <ht, dht> at the end is then not carried to tokens that it has decayed away from,
// where only its error would be left (fp32, 256 x 256, 1000 tokens: dg off by 3.2e-6
// of its norm summed from the end, by 0.8e-6 so).
// 9 us for 4 x 2048 tokens of 32 heads (5 MB of dots): latency of its few waves.
constexpr int kDgPer = kLinearAnchor / 64;
static_assert(32 % kDgPer == 0, "a lane's tokens lie in one chunk");
__global__ __launch_bounds__(256) void linear_dg_kernel(LinearDg p) {
  const int h = (int)(blockIdx.x % ((p.H + 3) / 4)) * 4 + (threadIdx.x >> 6);
  const int64_t item = blockIdx.x / ((p.H + 3) / 4);
  if (h >= p.H) return;
  const int lane = threadIdx.x & 63;
  LinearWalk w{};
  w.cu = p.cu;
  w.B = p.B;
  w.T = p.T;
  w.N = p.N;
  w.seg = kLinearAnchor;
  SegLoc sg;
  const bool ok = locate_segment(w, item, false, sg);
  double sum = 0.0;
  if (ok) {
    const int64_t rows = (int64_t)p.B * p.T;
    double before = 0.0, behind = 0.0;  // <h, dh> at the stretch's ends
    for (int cb = 0; cb < p.ncb; ++cb) {
      const int64_t slot = ((int64_t)sg.n * p.H + h) * p.ncb + cb;
      if (sg.in >= 0) before += p.anchor_dot[(sg.in * p.H + h) * p.ncb + cb];
      else if (p.start_dot) before += p.start_dot[slot];
      if (sg.out >= 0) behind += p.anchor_dot[(sg.out * p.H + h) * p.ncb + cb];
      else if (p.end_dot) behind += p.end_dot[slot];
    }
    // of each token a - b and a^2 + b^2, and over the lane's tokens the same of the far parts
    double x[kDgPer], m[kDgPer], own = 0.0, own_m = 0.0, far = 0.0, far_m = 0.0;
#pragma unroll
    for (int i = 0; i < kDgPer; ++i) {
      const int64_t t = sg.lo + lane * kDgPer + i;
      double a = 0.0, b = 0.0, fa = 0.0, fb = 0.0;
      if (t < sg.hi)
        for (int cb = 0; cb < p.ncb; ++cb) {
          const int64_t at = ((int64_t)cb * p.H + h) * rows + t;
          a += p.a[at];
          b += p.b[at];
          fa += p.a_far[at];
          fb += p.b_far[at];
        }
      own += x[i] = a - b;
      own_m += m[i] = a * a + b * b;
      far += fa - fb;
      far_m += fa * fa + fb * fb;
    }
    const int lanes = p.chunk / kDgPer, place = lane % lanes;
    // of this lane's tokens and all later ones: to the chunk's end, and of the far parts to the stretch's
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const double v = __shfl_down(far, off), vm = __shfl_down(far_m, off);
      if (lane + off < 64) far += v, far_m += vm;
      if (off < lanes) {
        const double w = __shfl_down(own, off), wm = __shfl_down(own_m, off);
        if (place + off < lanes) own += w, own_m += wm;
      }
    }
    const int head = lane - place, next = head + lanes;  // first lanes of this chunk and of the next
    const double all = __shfl(far, 0), all_m = __shfl(far_m, 0);
    const double here = __shfl(far, head), here_m = __shfl(far_m, head);
    double later = __shfl(far, next & 63), later_m = __shfl(far_m, next & 63);
    if (next >= 64) later = later_m = 0.0;
    const double whole = __shfl(own, head), whole_m = __shfl(own_m, head);
    // from the end, and from the start, where <h, dh> less all that came before is what is left
    double back = behind + later + own, back_m = behind * behind + later_m + own_m;
    double fore = before - (all - here) - (whole - own), fore_m = before * before + (all_m - here_m) + (whole_m - own_m);
#pragma unroll
    for (int i = 0; i < kDgPer; ++i) {
      const int64_t t = sg.lo + lane * kDgPer + i;
      const double d = fore_m < back_m ? fore : back;
      if (t < sg.hi) {
        sum += d;
        if (!p.g_head) p.dg[t * p.H + h] = (float)d;
      }
      back -= x[i], back_m -= m[i];
      fore -= x[i], fore_m += m[i];
    }
  }
  if (p.g_head) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
    if (lane == 0) p.part[item * p.H + h] = sum;
  }
}

// Head decays: the stretches' sums added in a fixed order, one workgroup a head.
__global__ __launch_bounds__(256) void linear_dg_head_kernel(const double *part, float *dg, int64_t items, int H) {
  __shared__ double red[256];
  const int h = blockIdx.x;
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < items; i += 256) s += part[i * H + h];
  red[threadIdx.x] = s;
  __syncthreads();
  for (int off = 128; off > 0; off >>= 1) {
    if ((int)threadIdx.x < off) red[threadIdx.x] += red[threadIdx.x + off];
    __syncthreads();
  }
  if (threadIdx.x == 0) dg[h] = (float)red[0];
}

}  // namespace

int linear_tile(int width) { return width <= 64 ? 64 : (width <= 128 ? 128 : 256); }

// By 128 columns x and z are read once where by 64 they are read twice. fp32
// takes 64 where 256 rows of state would spill by 128 (4 x 2048 tokens, 16
// heads, 256 x 128: 333 us against 561), and for few (sequence, head) pairs,
// where the smaller rows fit LDS twice and more workgroups help more than the
// second read costs (128 x 128, by 64 and by 128: 32 pairs of 2048 tokens 78 and
// 105 us, 64 of 4096 237 and 212, 256 of 2048 348 and 319).
int linear_cols(int P, int width, bool is_bf16, int64_t pairs, int *ncb) {
  const int qt = width <= 64 || (!is_bf16 && (P > 128 || 8 * pairs <= device_cus())) ? 64 : 128;
  *ncb = (width + qt - 1) / qt;
  return qt;
}

// Segments pay where whole sequences leave compute units idle (one workgroup
// each, by LDS). Costs in chunks of a walk that has the device to itself (3.3 us
// with y, 5 us with row dots at 128 wide): a state pass's chunk 0.62 or 0.42 of
// that; chaining and two more launches 12 to 20 us.
// Dense: rounds of equal segments. Packed, lengths unknown: the work shared out
// evenly plus half a segment behind the last, or one segment if that is longer,
// and 7 chunks for each segment's start and end, of which every slot adds about
// 0.6; the longest slot is taken to be as long as four average ones. How well it
// chooses, all in one run: 32 heads, 10 slots, 15872 tokens, segments of 512,
// 768, 1024, 1152 (its choice), 1280, 1408, 1536, 1792, none: 266, 250, 245, 236,
// 215, 215, 222, 248, 306 us; the gradient of 16 heads, 7 slots, 4999 tokens, of
// 256, 320, 384, 448, 512 (its choice), 640, 768: 202, 186, 176, 160, 168, 182,
// 200 us. Dense, its choices are the best measured: 1 x 32768 tokens, 16 heads, of
// 1024, 1536, 2048 (its choice), 4096: 242, 284, 220, 300 us; the gradient of 4 x
// 2048, 32 heads, of 512, 1024 (its choice), none: 428, 353, 434 us.
int linear_segment(int T, int slots, int H, int P, int Q, bool is_bf16, bool packed, bool dots) {
  int ncb;
  linear_cols(P, Q, is_bf16, (int64_t)slots * H, &ncb);
  const double room = device_cus();
  const int64_t pairs = (int64_t)H * ncb;
  const int64_t chunks = (T + 63) / 64;
  if (slots < 1 || chunks < 8) return 0;
  const double rate = dots ? 1.42 : 1.62, join = dots ? 2.4 : 6.0;
  const double share = pairs * chunks / room;
  double best = 0.97 * (packed ? std::max(chunks * std::min(1.0, 4.0 / slots), share)
                               : std::ceil(pairs * slots / room) * chunks);
  int64_t take = 1;
  for (int64_t s = 2; s <= 64 && chunks / s >= 4; ++s) {
    const double len = (double)((chunks + s - 1) / s);
    const double cost = packed ? std::max(len, share + len / 2) * rate + 7 * pairs * (s + 0.6 * slots) / room + join
                               : std::ceil(pairs * slots * s / room) * len * rate + join;
    if (cost < best) {
      best = cost;
      take = s;
    }
  }
  return take == 1 ? 0 : (int)((chunks + take - 1) / take * 64);
}

static int64_t chain_blocks(const LinearWalk &p) { return ((int64_t)p.P * p.Q / 4 + 255) / 256 * p.H * p.N; }

bool linear_walk_fits(const LinearWalk &p) {
  int ncb;
  const int qt = linear_cols(p.P, p.Q, p.is_bf16, (int64_t)p.N * p.H, &ncb);
  return linear_walk_blocks(p, ncb) <= most_blocks(64 * (qt / 16 + 4)) && (!p.seg || chain_blocks(p) <= most_blocks(256));
}

hipError_t launch_linear_chain(const LinearWalk &p, bool rev, hipStream_t st) {
  const int64_t elems = (int64_t)p.P * p.Q, grid = chain_blocks(p);
  if (grid > most_blocks(256)) return hipErrorInvalidValue;
  hipLaunchKernelGGL(linear_chain_kernel, dim3((unsigned)grid), dim3(256), 0, st, p, rev, elems);
  return hipGetLastError();
}

hipError_t launch_linear_walk(const LinearWalk &p, hipStream_t st) {
  if (p.N == 0) return hipSuccess;
  if (p.is_bf16) return p.reverse ? launch_linear_walk_bf16_rev(p, st) : launch_linear_walk_bf16_fwd(p, st);
  return p.reverse ? launch_linear_walk_f32_rev(p, st) : launch_linear_walk_f32_fwd(p, st);
}

static int64_t group_sum_blocks(int64_t rows, int Hk, int D) { return (rows * Hk * (D / 4) + 255) / 256; }

bool linear_group_sum_fits(int64_t rows, int Hk, int D) { return group_sum_blocks(rows, Hk, D) <= most_blocks(256); }

hipError_t launch_linear_group_sum(const float *in, void *out, bool is_bf16, const int32_t *cu, int N, int64_t rows,
                                   int H, int Hk, int D, hipStream_t st) {
  const int64_t grid = group_sum_blocks(rows, Hk, D);
  if (grid == 0) return hipSuccess;
  if (grid > most_blocks(256)) return hipErrorInvalidValue;
  if (is_bf16)
    hipLaunchKernelGGL(linear_group_sum_kernel<bf16_t>, dim3((unsigned)grid), dim3(256), 0, st, in,
                       reinterpret_cast<bf16_t *>(out), cu, N, rows, H, Hk, D);
  else
    hipLaunchKernelGGL(linear_group_sum_kernel<float>, dim3((unsigned)grid), dim3(256), 0, st, in,
                       reinterpret_cast<float *>(out), cu, N, rows, H, Hk, D);
  return hipGetLastError();
}

int linear_chunk_rows(int P, bool is_bf16) { return !is_bf16 || linear_tile(P) == 256 ? 32 : 64; }

int64_t linear_dg_items(int B, int T, int N) { return N + ((int64_t)B * T) / kLinearAnchor; }

bool linear_dg_fits(int64_t items, int H) { return items * ((H + 3) / 4) <= most_blocks(256); }

hipError_t launch_linear_dg(const LinearDg &p, hipStream_t st) {
  const int64_t items = linear_dg_items(p.B, p.T, p.N);
  const int64_t grid = items * ((p.H + 3) / 4);
  if (!linear_dg_fits(items, p.H)) return hipErrorInvalidValue;
  if (grid > 0) {
    hipLaunchKernelGGL(linear_dg_kernel, dim3((unsigned)grid), dim3(256), 0, st, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (p.g_head) hipLaunchKernelGGL(linear_dg_head_kernel, dim3(p.H), dim3(256), 0, st, p.part, p.dg, items, p.H);
  return hipGetLastError();
}

}  // namespace kda
