// The norm of every head's query and key row with the rotation by position
// (include/kda_rope.h), forward and backward:
//
//   n = w x rho,  rho = (mean x^2 + eps)^-1/2 (L2: sum);   y = R n
//   dn = R^T dy;  dw = sum over rows of dn x rho;  dx = rho (w dn - x rho^2 mean(w dn x))  (L2: sum)
//
// A lane holds both channels of VEC pairs, so the rotation never leaves it: its two
// vectors lie rot/2 channels apart (or next to each other), channels that are not turned
// are dealt out the same way, and D / (2 VEC) lanes hold a row. A group of lanes takes one
// token and every HS-th of its heads, the next row on its way beside the one at hand. A
// workgroup's angles (fp64 products and reduction) with their sines and cosines are formed
// once, one by each thread, and handed over in LDS: formed by every group for itself they
// took b4 t4096 h32/8 d128 from 74 to 89 us. Weights' gradients stay in registers over a
// workgroup's rows, leave as one part a workgroup, and are added over workgroups in order.
//
// Bound by the rows' bytes: at b4 t4096 h32/8 d128 the forward takes 72 us and the backward
// 105 + 5 us, where their 336 and 503 MB would take 64 and 97 us at a large copy's 5.2 TB/s;
// the fp32 forward 138 us for 129.
#include "../../include/kda_rope.h"
#include "kda_device.h"
#include "linear_launch.h"
#include "rope_launch.h"

namespace kda {

namespace {

typedef __bf16 bf16x4v_t __attribute__((ext_vector_type(4)));

// VEC values as they lie in memory.
template <typename T, int VEC>
struct Raw {
  static constexpr int W = VEC * (int)sizeof(T) / 4;  // dwords
  uint32_t w[W];
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (W == 2) {
      const u32x2_t v = *reinterpret_cast<const u32x2_t *>(p);
      w[0] = v[0], w[1] = v[1];
    } else {
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        const u32x4_t v = reinterpret_cast<const u32x4_t *>(p)[i];
#pragma unroll
        for (int e = 0; e < 4; ++e) w[4 * i + e] = v[e];
      }
    }
  }
  __device__ __forceinline__ void get(float (&x)[VEC]) const {
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      x[e] = sizeof(T) == 4 ? __uint_as_float(w[e]) : __uint_as_float(e & 1 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
  }
  static __device__ __forceinline__ void store(T *p, const float (&x)[VEC]) {
    uint32_t o[W];
#pragma unroll
    for (int i = 0; i < W; ++i) o[i] = sizeof(T) == 4 ? __float_as_uint(x[i % VEC]) : pack_bf16x2(x[(2 * i) % VEC], x[(2 * i + 1) % VEC]);
    if constexpr (W == 2) {
      *reinterpret_cast<u32x2_t *>(p) = u32x2_t{o[0], o[1]};
    } else {
#pragma unroll
      for (int i = 0; i < W / 4; ++i) reinterpret_cast<u32x4_t *>(p)[i] = u32x4_t{o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]};
    }
  }
};

// What a group of lanes does: its token, its first head, and its lane's channels.
struct Place {
  int j, lanes;   // lane of the row, lanes that hold channels
  int a, b;       // first channels of the lane's two vectors
  bool in, turned;
};
template <int VEC>
__device__ __forceinline__ Place place_of(const QkRope &p, int j) {
  Place l;
  l.j = j;
  l.lanes = p.D / (2 * VEC);
  l.in = j < l.lanes;
  l.turned = j * VEC < p.rot / 2;
  if (p.adjacent) {
    l.a = 2 * j * VEC;
    l.b = l.a + VEC;
  } else if (l.turned) {
    l.a = j * VEC;
    l.b = p.rot / 2 + l.a;
  } else {
    l.a = p.rot + (j * VEC - p.rot / 2);
    l.b = l.a + (p.D - p.rot) / 2;
  }
  return l;
}

// Cosines and sines of `count` tokens from t0 on, each angle by one thread, to LDS: turns in
// fp64, whole quarters taken off there, so that what is rounded to fp32 is at most an eighth
// of a turn (2^-28 of a turn off; half a turn would be 2^-26 off, more than the sines are).
__device__ __forceinline__ void angles(const QkRope &p, int64_t t0, int count, float *cs) {
  const int half = p.rot / 2;
  for (int idx = threadIdx.x; idx < count * half; idx += 256) {
    const int tk = idx / half, i = idx - tk * half;
    const int64_t token = t0 + tk;
    if (token >= p.tokens) break;
    int at = 0;
    if (p.axes > 1) {
      if (p.spread) {
        at = i % p.axes;
        const int lim = at == 0 ? 0 : (at == 1 ? p.sec[1] : (at == 2 ? p.sec[2] : p.sec[3]));
        if (i >= lim) at = 0;
      } else {
        at = (i >= p.sec[0]) + (i >= p.sec[1]) + (i >= p.sec[2]);
      }
    }
    double t = ((double)p.pos[at * p.tokens + token] * (double)p.freq[i]) * 0.15915494309189533577;
    t -= rint(t);
    const double quarters = rint(4.0 * t);
    float sn, c;
    sincospif(2.0f * (float)(t - 0.25 * quarters), &sn, &c);
    const int n = (int)quarters & 3;
    const float x = n & 1 ? sn : c, y = n & 1 ? c : sn;
    cs[idx] = n == 1 || n == 2 ? -x : x;
    cs[count * half + idx] = n & 2 ? -y : y;
  }
}
template <int VEC>
__device__ __forceinline__ void read_angles(const QkRope &p, const Place &l, int tk, int count, const float *cs, float (&c)[VEC],
                                            float (&s)[VEC]) {
  const float *src = cs + tk * (p.rot / 2) + l.j * VEC;
#pragma unroll
  for (int e = 0; e < VEC; e += 4) {
    const f32x4_t x = *reinterpret_cast<const f32x4_t *>(src + e), y = *reinterpret_cast<const f32x4_t *>(src + count * (p.rot / 2) + e);
#pragma unroll
    for (int i = 0; i < 4; ++i) c[e + i] = x[i], s[e + i] = y[i];
  }
}

// (a, b) pairs of the lane turned by +- the angles.
template <int VEC>
__device__ __forceinline__ void turn(bool adjacent, float sign, const float (&c)[VEC], const float (&s)[VEC], float (&a)[VEC],
                                     float (&b)[VEC]) {
  if (!adjacent) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float x = a[e], y = b[e], z = sign * s[e];
      a[e] = x * c[e] - y * z;
      b[e] = y * c[e] + x * z;
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {  // pair e: channels 2 e and 2 e + 1 of the lane's 2 VEC
      float *v = 2 * e < VEC ? &a[(2 * e) % VEC] : &b[(2 * e) % VEC];
      const float x = v[0], y = v[1], z = sign * s[e];
      v[0] = x * c[e] - y * z;
      v[1] = y * c[e] + x * z;
    }
  }
}

template <int VEC>
__device__ __forceinline__ void weight_of(const float *w, const Place &l, float (&a)[VEC], float (&b)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    a[e] = w && l.in ? w[l.a + e] : 1.f;
    b[e] = w && l.in ? w[l.b + e] : 1.f;
  }
}

template <int GL>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int off = GL / 2; off > 0; off >>= 1) x += __shfl_xor(x, off);
  return x;
}

template <typename T, int VEC, int GL>
__global__ __launch_bounds__(256) void qk_rope_fwd_kernel(QkRope p, int HS) {
  const int g = threadIdx.x / GL, tpb = 256 / GL / HS;  // tokens of a workgroup at a time
  const Place l = place_of<VEC>(p, threadIdx.x % GL);
  const float inv = p.l2 ? 1.0f : 1.0f / (float)p.D;
  extern __shared__ __align__(16) float angle_lds[];  // two iterations' cosines and sines
  const int rows = p.H + p.Hk;
  int turn_no = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * tpb; t0 < p.tokens; t0 += (int64_t)gridDim.x * tpb, turn_no ^= 1) {
    const int64_t token = t0 + g / HS;
    const bool live = token < p.tokens && l.in;
    const T *const q = reinterpret_cast<const T *>(p.q) + token * p.qs, *const k = reinterpret_cast<const T *>(p.k) + token * p.ks;
    T *const qo = reinterpret_cast<T *>(p.qo) + token * p.qos, *const ko = reinterpret_cast<T *>(p.ko) + token * p.kos;
    Raw<T, VEC> ra, rb;
    auto fetch = [&](int r) {  // a row: q's heads, then k's
      if (r < rows && live) {
        const T *in = r < p.H ? q + (int64_t)r * p.D : k + (int64_t)(r - p.H) * p.D;
        ra.load(in + l.a);
        rb.load(in + l.b);
      }
    };
    int r = g % HS;
    fetch(r);
    float c[VEC], s[VEC];
    if (p.rot) {
      float *const cs = angle_lds + turn_no * tpb * p.rot;
      angles(p, t0, tpb, cs);
      __syncthreads();
      if (l.turned && live) read_angles<VEC>(p, l, g / HS, tpb, cs, c, s);
    }
    if (token >= p.tokens) continue;  // (a whole group)
    float wa[VEC], wb[VEC];
    weight_of<VEC>(r < p.H ? p.q_weight : p.k_weight, l, wa, wb);
    for (; r < rows; r += HS) {
      float a[VEC], b[VEC];
      ra.get(a);
      rb.get(b);
      fetch(r + HS);  // the next row on its way
      float rho = 1.f;
      if (p.normed) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss += a[e] * a[e] + b[e] * b[e];
        ss = row_sum<GL>(l.in ? ss : 0.f);
        rho = 1.0f / sqrtf(ss * inv + p.eps);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        a[e] = a[e] * rho * wa[e];
        b[e] = b[e] * rho * wb[e];
      }
      if (l.turned) turn<VEC>(p.adjacent, 1.f, c, s, a, b);
      if (l.in) {
        T *const out = r < p.H ? qo + (int64_t)r * p.D : ko + (int64_t)(r - p.H) * p.D;
        Raw<T, VEC>::store(out + l.a, a);
        Raw<T, VEC>::store(out + l.b, b);
      }
      if (r < p.H && r + HS >= p.H) weight_of<VEC>(p.k_weight, l, wa, wb);
    }
  }
}

template <typename T, int VEC, int GL>
__global__ __launch_bounds__(256) void qk_rope_bwd_kernel(QkRope p, int HS) {
  const int g = threadIdx.x / GL, tpb = 256 / GL / HS;
  const Place l = place_of<VEC>(p, threadIdx.x % GL);
  const float inv = p.l2 ? 1.0f : 1.0f / (float)p.D;
  float acc[2][2][VEC];  // weights' gradients of q and k
#pragma unroll
  for (int e = 0; e < VEC; ++e) acc[0][0][e] = acc[0][1][e] = acc[1][0][e] = acc[1][1][e] = 0.f;
  extern __shared__ __align__(16) float angle_lds[];
  const int rows = p.H + p.Hk;
  int turn_no = 0;
  for (int64_t t0 = (int64_t)blockIdx.x * tpb; t0 < p.tokens; t0 += (int64_t)gridDim.x * tpb, turn_no ^= 1) {
    const int64_t token = t0 + g / HS;
    const bool live = token < p.tokens && l.in;
    const T *const q = reinterpret_cast<const T *>(p.q) + token * p.qs, *const k = reinterpret_cast<const T *>(p.k) + token * p.ks;
    const T *const dqo = reinterpret_cast<const T *>(p.dqo) + token * p.qos, *const dko = reinterpret_cast<const T *>(p.dko) + token * p.kos;
    Raw<T, VEC> ra, rb, da, db;
    auto fetch = [&](int r) {  // a row: q's heads, then k's
      if (r < rows && live) {
        const bool of_k = r >= p.H;
        const int64_t at = (int64_t)(of_k ? r - p.H : r) * p.D;
        const T *const in = (of_k ? k : q) + at, *const dy = (of_k ? dko : dqo) + at;
        ra.load(in + l.a);
        rb.load(in + l.b);
        da.load(dy + l.a);
        db.load(dy + l.b);
      }
    };
    int r = g % HS;
    fetch(r);
    float c[VEC], s[VEC];
    if (p.rot) {
      float *const cs = angle_lds + turn_no * tpb * p.rot;
      angles(p, t0, tpb, cs);
      __syncthreads();
      if (l.turned && live) read_angles<VEC>(p, l, g / HS, tpb, cs, c, s);
    }
    if (token >= p.tokens) continue;  // (a whole group)
    float wa[VEC], wb[VEC];
    weight_of<VEC>(r < p.H ? p.q_weight : p.k_weight, l, wa, wb);
    for (; r < rows; r += HS) {
      float a[VEC], b[VEC], ga[VEC], gb[VEC];
      ra.get(a);
      rb.get(b);
      da.get(ga);
      db.get(gb);
      fetch(r + HS);
      if (!l.in) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) a[e] = b[e] = ga[e] = gb[e] = 0.f;
      }
      if (l.turned) turn<VEC>(p.adjacent, -1.f, c, s, ga, gb);
      float rho = 1.f, m = 0.f;
      if (p.normed) {
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          ss += a[e] * a[e] + b[e] * b[e];
          dot += ga[e] * wa[e] * a[e] + gb[e] * wb[e] * b[e];
        }
        ss = row_sum<GL>(ss);
        dot = row_sum<GL>(dot);
        rho = 1.0f / sqrtf(ss * inv + p.eps);
        m = dot * inv * rho * rho;
      }
      if (l.in) {
        auto add = [&](float (&to)[2][VEC]) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            to[0][e] += ga[e] * (a[e] * rho);
            to[1][e] += gb[e] * (b[e] * rho);
          }
        };
        if (r < p.H) add(acc[0]);
        else add(acc[1]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          a[e] = rho * (ga[e] * wa[e] - a[e] * m);
          b[e] = rho * (gb[e] * wb[e] - b[e] * m);
        }
        T *const out = r < p.H ? reinterpret_cast<T *>(p.qo) + (token * p.H + r) * p.D
                               : reinterpret_cast<T *>(p.ko) + (token * p.Hk + r - p.H) * p.D;
        Raw<T, VEC>::store(out + l.a, a);
        Raw<T, VEC>::store(out + l.b, b);
      }
      if (r < p.H && r + HS >= p.H) weight_of<VEC>(p.k_weight, l, wa, wb);
    }
  }
  if (!p.part) return;
  // the groups' sums: over those of a wave by shuffles, over the four waves through LDS
  __shared__ float sums[4][GL][2 * VEC + 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int part = 0; part < 2; ++part) {
#pragma unroll
    for (int off = GL; off < 64; off <<= 1)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        acc[part][0][e] += __shfl_xor(acc[part][0][e], off);
        acc[part][1][e] += __shfl_xor(acc[part][1][e], off);
      }
    __syncthreads();
    if (lane < GL)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        sums[wave][lane][e] = acc[part][0][e];
        sums[wave][lane][VEC + e] = acc[part][1][e];
      }
    __syncthreads();
    float *dst = p.part + ((int64_t)blockIdx.x * 2 + part) * p.D;
    if ((int)threadIdx.x < GL && l.in) {
#pragma unroll
      for (int e = 0; e < 2 * VEC; ++e) {
        const int j = threadIdx.x;
        dst[e < VEC ? l.a + e : l.b + e - VEC] = (sums[0][j][e] + sums[1][j][e]) + (sums[2][j][e] + sums[3][j][e]);
      }
    }
  }
}

// Sums over the workgroups' parts in a fixed order and fp64: 16 channels a workgroup, 64
// lanes of a channel each taking every 64th part, eight of them in flight.
__global__ __launch_bounds__(1024) void qk_rope_params_kernel(QkRope p, int blocks) {
  __shared__ double red[16][16];
  float *out = blockIdx.y ? p.dk_weight : p.dq_weight;
  if (!out) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = blockIdx.x * 16 + (threadIdx.x & 15), first = threadIdx.x >> 4;
  const float *src = p.part + (int64_t)blockIdx.y * p.D + min(c, p.D - 1);
  double s = 0.0;
  for (int b = first; b < blocks; b += 512) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = src[(int64_t)min(b + 64 * i, blocks - 1) * 2 * p.D];
#pragma unroll
    for (int i = 0; i < 8; ++i) s += b + 64 * i < blocks ? (double)v[i] : 0.0;
  }
  s += __shfl_xor(s, 16);
  s += __shfl_xor(s, 32);
  if (lane < 16) red[wave][lane] = s;
  __syncthreads();
  if (threadIdx.x < 16 && c < p.D) {
    s = red[0][lane];
    for (int w = 1; w < 16; ++w) s += red[w][lane];
    out[c] = (float)s;
  }
}

// Pairs of a lane: eight, or four where a vector of eight would not begin on a multiple of eight.
int vec_of(const QkRope &p) { return p.rot % 16 == 0 && p.D % 16 == 0 ? 8 : 4; }
int group_of(const QkRope &p) {
  const int lanes = p.D / (2 * vec_of(p));
  int gl = 1;
  while (gl < lanes) gl *= 2;
  return gl;
}

// Groups that share a token: all of a workgroup's, halved while a group has fewer than
// eight rows and the device stays full. b4 t4096 with 40 heads of 128 channels (a lane row
// has 8 lanes, a workgroup 32 groups), forward and backward kernel: 4 groups a token 70 and
// 109 us, 32 groups 155 and 211, 8 groups 74 and 117, 1 group 82 and 138. 64 tokens: 32
// groups 7 us, 8 groups 10, 1 group 40.
int heads_split(const QkRope &p, int groups) {
  const int rows = p.H + p.Hk;
  int hs = groups;
  while (hs > 1 && rows < 8 * hs && (p.tokens * (hs / 2) / groups >= 8 * device_cus() || hs / 2 >= rows)) hs /= 2;
  return hs;
}

int64_t fwd_blocks(const QkRope &p, int groups, int hs) { return (p.tokens + groups / hs - 1) / (groups / hs); }

// Workgroups of the backward: enough to fill the device, few enough that their parts stay small.
int bwd_blocks(const QkRope &p) {
  const int groups = 256 / group_of(p);
  const int64_t need = fwd_blocks(p, groups, heads_split(p, groups)), most = (int64_t)device_cus() * 4;
  return (int)(need < most ? (need > 0 ? need : 1) : most);
}

template <typename T, int VEC, int GL>
hipError_t launch_gl(const QkRope &p, bool bwd, hipStream_t st) {
  const int groups = 256 / GL, hs = heads_split(p, groups);
  const unsigned lds = 2u * (groups / hs) * p.rot * sizeof(float);  // at most 32 KB: rot channels are a group's lanes' pairs
  if (bwd) {
    hipLaunchKernelGGL((qk_rope_bwd_kernel<T, VEC, GL>), dim3(bwd_blocks(p)), dim3(256), lds, st, p, hs);
  } else {
    const int64_t need = fwd_blocks(p, groups, hs), most = most_blocks(256);
    if (need == 0) return hipSuccess;
    hipLaunchKernelGGL((qk_rope_fwd_kernel<T, VEC, GL>), dim3((unsigned)(need < most ? need : most)), dim3(256), lds, st, p, hs);
  }
  return hipGetLastError();
}

template <typename T, int VEC>
hipError_t launch_vec(const QkRope &p, bool bwd, hipStream_t st) {
  switch (group_of(p)) {
    case 1: return launch_gl<T, VEC, 1>(p, bwd, st);
    case 2: return launch_gl<T, VEC, 2>(p, bwd, st);
    case 4: return launch_gl<T, VEC, 4>(p, bwd, st);
    case 8: return launch_gl<T, VEC, 8>(p, bwd, st);
    case 16: return launch_gl<T, VEC, 16>(p, bwd, st);
    case 32: return launch_gl<T, VEC, 32>(p, bwd, st);
    default:
      if constexpr (VEC == 4) return launch_gl<T, VEC, 64>(p, bwd, st);
      return hipErrorInvalidValue;  // 512 channels by eight pairs a lane are 32 lanes
  }
}

hipError_t launch_types(const QkRope &p, bool bwd, hipStream_t st) {
  if (vec_of(p) == 8) return p.is_bf16 ? launch_vec<bf16_t, 8>(p, bwd, st) : launch_vec<float, 8>(p, bwd, st);
  return p.is_bf16 ? launch_vec<bf16_t, 4>(p, bwd, st) : launch_vec<float, 4>(p, bwd, st);
}

}  // namespace

size_t qk_rope_part_bytes(const QkRope &p) { return (size_t)bwd_blocks(p) * 2 * p.D * sizeof(float); }

hipError_t launch_qk_rope_fwd(const QkRope &p, hipStream_t st) { return launch_types(p, false, st); }

hipError_t launch_qk_rope_bwd(const QkRope &p, hipStream_t st) {
  const hipError_t e = launch_types(p, true, st);
  if (e != hipSuccess || !p.part) return e;
  hipLaunchKernelGGL(qk_rope_params_kernel, dim3((p.D + 15) / 16, 2), dim3(1024), 0, st, p, bwd_blocks(p));
  return hipGetLastError();
}

}  // namespace kda

// ---------------------------------------------------------------------------------------------
// host API
// ---------------------------------------------------------------------------------------------
namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Sizes (also for the workspace query), and the block of sizes that the kernels take.
kda_status base(const kda_qk_args *a, kda::QkRope &p) {
  if (!a) return KDA_ERR_NULL;
  if (a->tokens < 0 || a->tokens > (int64_t)1 << 31 || a->H < 1 || a->Hk < 1 || a->H > 65536 || a->Hk > 65536 || a->D < 1 ||
      a->rot < 0 || a->rot > a->D || a->axes < 1 || a->axes > 4 || !(a->eps >= 0.f))
    return KDA_ERR_SHAPE;
  if (a->dtype != KDA_BF16 && a->dtype != KDA_F32) return KDA_ERR_DTYPE;
  if ((a->norm != KDA_QK_RMS && a->norm != KDA_QK_L2 && a->norm != KDA_QK_NONE) ||
      (a->pairs != KDA_PAIRS_HALF && a->pairs != KDA_PAIRS_ADJACENT))
    return KDA_ERR_GATE;
  if (a->D % 8 != 0 || a->D > 512 || a->rot % 8 != 0) return KDA_ERR_UNSUPPORTED;
  p.tokens = a->tokens;
  p.H = a->H;
  p.Hk = a->Hk;
  p.D = a->D;
  p.rot = a->rot;
  const int64_t nq = (int64_t)a->H * a->D, nk = (int64_t)a->Hk * a->D;
  const int64_t strides[4] = {a->q_stride, a->k_stride, a->qo_stride, a->ko_stride};
  for (int i = 0; i < 4; ++i)
    if (strides[i] != 0 && (strides[i] < (i & 1 ? nk : nq) || strides[i] % 8 != 0 || strides[i] > (int64_t)1 << 31)) return KDA_ERR_SHAPE;
  p.qs = a->q_stride ? a->q_stride : nq;
  p.ks = a->k_stride ? a->k_stride : nk;
  p.qos = a->qo_stride ? a->qo_stride : nq;
  p.kos = a->ko_stride ? a->ko_stride : nk;
  p.axes = a->rot ? a->axes : 1;
  p.spread = a->spread != 0;
  if (p.axes > 1) {
    const int half = a->rot / 2;
    int sum = 0;
    for (int i = 0; i < p.axes; ++i) {
      if (a->sections[i] < 0 || a->sections[i] > half) return KDA_ERR_SHAPE;
      if (p.spread && i > 0 && a->sections[i] > 0 && i + p.axes * (a->sections[i] - 1) >= half) return KDA_ERR_SHAPE;
      sum += a->sections[i];
    }
    if (sum != half) return KDA_ERR_SHAPE;
    int end = 0;
    for (int i = 0; i < 4; ++i) {
      end += i < p.axes ? a->sections[i] : 0;
      p.sec[i] = p.spread ? (i < p.axes ? p.axes * a->sections[i] : 0) : (i < p.axes - 1 ? end : half);
    }
  }
  p.is_bf16 = a->dtype == KDA_BF16;
  p.adjacent = a->pairs == KDA_PAIRS_ADJACENT;
  p.normed = a->norm != KDA_QK_NONE;
  p.l2 = a->norm == KDA_QK_L2;
  p.eps = a->eps;
  return KDA_OK;
}

}  // namespace

extern "C" kda_status kda_qk_norm_rope_fwd(const kda_qk_args *a, const void *q, const void *k, const float *q_weight,
                                           const float *k_weight, const int32_t *positions, const float *inv_freq,
                                           void *q_out, void *k_out, void *stream) {
  kda::QkRope p{};
  const kda_status s = base(a, p);
  if (s != KDA_OK) return s;
  if (p.tokens > 0 && (!q || !k || !q_out || !k_out || (p.rot && (!positions || !inv_freq)))) return KDA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out)) return KDA_ERR_ALIGN;
  p.q = q;
  p.k = k;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.pos = positions;
  p.freq = inv_freq;
  p.qo = q_out;
  p.ko = k_out;
  return kda::report_hip(kda::launch_qk_rope_fwd(p, (hipStream_t)stream));
}

extern "C" size_t kda_qk_norm_rope_bwd_workspace_bytes(const kda_qk_args *a) {
  kda::QkRope p{};
  return base(a, p) == KDA_OK ? kda::qk_rope_part_bytes(p) : 0;
}

extern "C" kda_status kda_qk_norm_rope_bwd(const kda_qk_args *a, const void *q, const void *k, const float *q_weight,
                                           const float *k_weight, const int32_t *positions, const float *inv_freq,
                                           const void *dq_out, const void *dk_out, void *dq, void *dk,
                                           float *dq_weight, float *dk_weight, void *workspace, size_t ws_bytes,
                                           void *stream) {
  kda::QkRope p{};
  const kda_status s = base(a, p);
  if (s != KDA_OK) return s;
  if (p.tokens > 0 && (!q || !k || !dq_out || !dk_out || !dq || !dk || (p.rot && (!positions || !inv_freq)))) return KDA_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(dq_out) || !aligned16(dk_out) || !aligned16(dq) || !aligned16(dk))
    return KDA_ERR_ALIGN;
  if (dq_weight || dk_weight) {
    if (!workspace || ws_bytes < kda::qk_rope_part_bytes(p)) return KDA_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return KDA_ERR_ALIGN;
    p.part = static_cast<float *>(workspace);
  }
  p.q = q;
  p.k = k;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.pos = positions;
  p.freq = inv_freq;
  p.dqo = dq_out;
  p.dko = dk_out;
  p.qo = dq;
  p.ko = dk;
  p.dq_weight = dq_weight;
  p.dk_weight = dk_weight;
  return kda::report_hip(kda::launch_qk_rope_bwd(p, (hipStream_t)stream));
}
