// Gated delta rule: the chain of segments, and the choice of columns and segments.
#include <algorithm>
#include <cmath>

#include "delta_chunk.h"

namespace kda {

namespace {

// The state at every boundary of a sequence from its segments' own, S_j = B_j + M_j S_{j-1},
// in place. One workgroup takes a (sequence, head, 16 columns): its four waves share out the
// 16-row tiles, each an fp32-accurate product of M's rows (three bf16 parts, split as they
// are loaded, the next boundary's in flight) with the last state, which passes between the
// waves through LDS as operands. A chain of short steps, 3.4 us a boundary (1 x 32768
// tokens, 16 heads: 47 us for 14 of them); the next boundary's state and M's parts formed
// a boundary ahead as well took 49.
template <int PT>
__global__ __launch_bounds__(256) void delta_chain_kernel(DeltaWalk p) {
  constexpr int NT = PT / 16, PS = PT / 32, TW = NT / 4;
  constexpr bool AHEAD = PT <= 128;  // 256 rows of M leave no registers for more
  __shared__ __align__(16) bf16_t sB[2][PS * 3 * 512];
  const int ncb = (p.V + 15) / 16;
  const int cb = (int)(blockIdx.x % ncb), h = (int)(blockIdx.x / ncb % p.H), n = (int)(blockIdx.x / ncb / p.H);
  const int lane = threadIdx.x & 63, wave = wave_id(), grp = lane >> 4, l16 = lane & 15;
  const SlotRange sr = slot_range(p.cu, n, p.T);
  const int64_t nb = sr.len > 0 ? (sr.len - 1) / p.seg : 0;  // boundaries inside the sequence
  if (nb < 2) return;
  const int K = p.K, V = p.V, q = 16 * cb + l16;
  int64_t j = sr.t0 / p.seg + 1;

  // tiles 4 x + wave of this wave: rows state_channel(t, grp) + e; as the product's rows
  // a lane's is the one that lies at l16 there
  auto row_of = [&](int t) { return state_channel(t, l16 >> 2) + (l16 & 3); };
  f32x4_t m[TW][PS][2];
  auto fetch_map = [&](int64_t at) {
    const auto rs = tile_rsrc(p.seg_map + (at * p.H + h) * K * K, (uint32_t)(K * K * 4));
#pragma unroll
    for (int x = 0; x < TW; ++x)
#pragma unroll
      for (int s = 0; s < PS; ++s) {
        const int ch = 32 * s + 8 * grp;
        const uint32_t off = ch < K ? (uint32_t)((row_of(4 * x + wave) * K + ch) * 4) : kOffNone;
        m[x][s][0] = __builtin_bit_cast(f32x4_t, tile_load16(rs, off));
        m[x][s][1] = __builtin_bit_cast(f32x4_t, tile_load16(rs, off + 16));
      }
  };
  f32x4_t own[TW];
  auto state_at = [&](int64_t at) { return p.seg_state + (at * p.H + h) * (int64_t)K * V; };
  auto fetch_state = [&](int64_t at) {
    const auto rs = tile_rsrc(state_at(at), (uint32_t)(K * V * 4));
#pragma unroll
    for (int x = 0; x < TW; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = state_channel(4 * x + wave, grp) + e;
        own[x][e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, q < V ? (r * V + q) * 4 : (int)kOffNone, 0, 0));
      }
  };
  auto hand_over = [&](int buf) {
#pragma unroll
    for (int x = 0; x < TW; ++x) {
      const int t = 4 * x + wave;
      put_parts<3>(own[x], sB[buf] + ((t >> 1) * 192 + lane) * 8 + 4 * (t & 1), 512);
    }
  };
  fetch_state(j);
  // whether the map of the segment that ends at a boundary is zero
  auto is_zero = [&](int64_t to) { return p.seg_zero[to * p.H + h] != 0; };
  bool zero = is_zero(j + 1);
  if (AHEAD && !zero) fetch_map(j + 1);
  hand_over(0);
  for (int64_t i = 1; i < nb; ++i) {
    ++j;
    const int buf = (int)(i - 1) & 1;
    fetch_state(j);
    if (!AHEAD && !zero) fetch_map(j);
    __syncthreads();
    const bool next_zero = i + 1 < nb && is_zero(j + 1);
    if (zero) {  // the segment's own state is all there is
      if (AHEAD && i + 1 < nb && !next_zero) fetch_map(j + 1);
      zero = next_zero;
      hand_over(buf ^ 1);
      continue;
    }
    bf16x8_t b[PS][3];
#pragma unroll
    for (int s = 0; s < PS; ++s)
#pragma unroll
      for (int pl = 0; pl < 3; ++pl) b[s][pl] = row_frag(sB[buf] + ((s * 3 + pl) * 64 + lane) * 8);
#pragma unroll
    for (int x = 0; x < TW; ++x)
#pragma unroll
      for (int s = 0; s < PS; ++s) {
        bf16x8_t a[3];
        split_pair<3>(m[x][s][0], m[x][s][1], a);
        own[x] = mma_parts(a, b[s], own[x]);
      }
    if (AHEAD && i + 1 < nb && !next_zero) fetch_map(j + 1);
    zero = next_zero;
    hand_over(buf ^ 1);
    const auto rs = tile_rsrc(state_at(j), (uint32_t)(K * V * 4));
#pragma unroll
    for (int x = 0; x < TW; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = state_channel(4 * x + wave, grp) + e;
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(own[x][e]), rs, q < V ? (r * V + q) * 4 : (int)kOffNone, 0, 0);
      }
  }
}

int64_t chain_blocks(const DeltaWalk &p) { return (int64_t)p.N * p.H * ((p.V + 15) / 16); }

}  // namespace

hipError_t launch_delta_chain(const DeltaWalk &p, hipStream_t st) {
  const int64_t grid = chain_blocks(p);
  if (grid > most_blocks(256)) return hipErrorInvalidValue;
  switch (linear_tile(p.K)) {
    case 64: hipLaunchKernelGGL((delta_chain_kernel<64>), dim3((unsigned)grid), dim3(256), 0, st, p); break;
    case 128: hipLaunchKernelGGL((delta_chain_kernel<128>), dim3((unsigned)grid), dim3(256), 0, st, p); break;
    default: hipLaunchKernelGGL((delta_chain_kernel<256>), dim3((unsigned)grid), dim3(256), 0, st, p); break;
  }
  return hipGetLastError();
}

// Columns of a workgroup: 128, a wave on every SIMD beside another; 64 where V has no
// more, for fp32 inputs, whose three parts leave no registers for more, and where 128
// would leave half the compute units idle (a chunk of 128 x 128 then takes 3.9 us
// instead of 5.7: calls on 128 (sequence, head) pairs of 2048 tokens 163 us by 64, 219 us
// by 128; on 256 pairs of 4096 tokens 602 us by 64, 543 us by 128).
int delta_cols(const DeltaWalk &p, int *ncb) {
  const int64_t parts = p.seg ? (int64_t)p.B * p.T / p.seg : p.N;
  const int64_t wide = std::max<int64_t>(parts, p.N) * p.H * ((p.V + 127) / 128);
  const int qt = p.V <= 64 || !p.is_bf16 || 2 * wide <= device_cus() ? 64 : 128;
  *ncb = (p.V + qt - 1) / qt;
  return qt;
}

bool delta_walk_fits(const DeltaWalk &p) {
  int ncb;
  const int qt = delta_cols(p, &ncb);
  if (p.seg && ((p.K + qt - 1) / qt + ncb) * delta_walk_blocks(p, 1) > most_blocks(64 * (qt / 16 + 4))) return false;
  return delta_walk_blocks(p, ncb) <= most_blocks(64 * (qt / 16 + 4)) && (!p.seg || chain_blocks(p) <= most_blocks(256));
}

// Segments pay where whole sequences leave compute units idle or wait for the longest.
// Costs in microseconds a chunk and workgroup as measured for bf16, 128 x 128, by 128 or 64
// columns when o took two parts: 6.3 or 3.9 (4.8 or 3.1 alone on the device) with o, 0.8 of
// that in the state pass, whose segments (all but a sequence's last) walk V and, but for the
// first, K columns. They serve every width and type, and what o takes now (7.1, 5.7) would
// move the choices below by a chunk at most. Two chunks for a segment's start and end; two
// more launches and a boundary's step of the chain 2.5 us. With decays most maps are zero
// and not walked (delta_walk.h): an eighth is counted. (That states are then walked from a
// segment's last chunks on only is not: the pass waits for the slowest head.)
// What it chooses, and whole calls: 1 x 32768 tokens, 16 heads: 35 chunks, 428 us (31: 509,
// 32: 416, 64: 401, none: 1690); fp32, 2 x 1000 tokens, 8 heads: 5 chunks, 65 us (8: 62,
// none: 91). 15872 packed tokens, 32 heads: 18 chunks whatever the 10 slots' lengths are:
//                              10   13   16   18   20   24   30  none
//     random cuts             496  477  450  450  440  448  483   558 us
//     equal slots             471  392  418  433  448  482  360   342
//     one of 14972, nine 100  597  544  537  539  512  555  530  1308
// Chosen without the slots' own lengths, it bounds what a long one costs, and takes a
// quarter more than the best for equal ones.
int delta_segment(const DeltaWalk &p, bool packed, bool gated) {
  const int C = delta_chunk(linear_tile(p.K), p.is_bf16);
  const double room = device_cus(), maps = gated ? 0.12 : 1.0;
  const int64_t chunks = ((int64_t)p.T + C - 1) / C;  // of a sequence; packed: of the batch
  if (p.N < 1 || chunks < 8) return 0;
  double best = 0.0;
  int64_t take = 1;
  for (int64_t s = 1; s <= 64 && (s == 1 || chunks / s >= 4); ++s) {
    const int64_t len = (chunks + s - 1) / s;
    DeltaWalk w = p;
    w.seg = s == 1 ? 0 : (int)(len * C);
    int ncb;
    const int qt = delta_cols(w, &ncb);
    const int kcb = (p.K + qt - 1) / qt;
    const double busy = qt == 128 ? 6.3 : 3.9, alone = qt == 128 ? 4.8 : 3.1;
    auto pass = [&](double wgs, double length, double rate) {  // wgs workgroups of `length` chunks
      const double rounds = std::max(1.0, std::ceil(wgs / room - 0.02));
      return rounds * (length + (s > 1 ? 2.0 : 0.0)) * rate * (wgs > 0.6 * room ? busy : alone);
    };
    double cost;
    if (!packed) {
      cost = pass((double)p.N * p.H * s * ncb, (double)len, 1.0);
      if (s > 1)
        cost += pass((double)p.N * p.H * ((s - 1) * ncb + (s - 2) * kcb * maps), (double)len, 0.8) + 2.5 * (double)(s + 3);
    } else {
      // lengths unknown: spread as by random cuts (exponentially), the longest slot 3.2
      // average ones. Of a slot's chunks, segments that end inside it hold the sum over
      // i >= 1 of len P(longer than i len); the state pass walks V columns of those and K
      // columns of all of them but the first. Work is shared out evenly, plus half a
      // segment behind the last.
      const double mean = (double)chunks / p.N, l = (double)len, x = std::exp(-l / mean);
      const double share = (double)chunks * p.H * ncb / room, longest = std::min((double)chunks, 3.2 * mean);
      if (s == 1) {
        cost = std::max(longest, share + 0.5 * longest) * busy;
      } else {
        const double cut = l * x / (1.0 - x) / mean;
        const double start = 1.0 + 2.0 / l;
        cost = std::max(l, share * start + 0.5 * l) * busy +
               std::max(l, share * cut * (1.0 + x * maps * kcb / ncb) * start + 0.5 * l) * 0.8 * busy +
               2.5 * (std::max(0.0, longest / l - 1.0) + 3);
      }
    }
    if (s == 1 || cost < best) {
      // (packed, cutting also bounds what a longer slot than supposed costs)
      best = s == 1 ? (packed ? 1.05 : 0.95) * cost : cost;
      take = s;
    }
  }
  return take == 1 ? 0 : (int)((chunks + take - 1) / take * C);
}

}  // namespace kda
