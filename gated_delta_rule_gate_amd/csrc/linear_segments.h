// Where a segment of a sequence lies (linear attention).
#pragma once

#include "kda_device.h"
#include "linear_launch.h"

namespace kda {

// A segment of one sequence: rows [lo, hi) of the token axis, of the sequence
// [a, e), entered over boundary `in` and left over `out` in the walk's order
// (-1: the sequence's own start or end).
struct SegLoc {
  int n;
  int64_t a, e, lo, hi;
  int64_t in, out;
};

// Items are the sequences' first segments, then one for every multiple of seg
// on the token axis: a sequence's boundaries lie seg apart, so each falls into
// a window of its own, and the only sequence with a boundary in window j is
// the one that holds token j * seg.
__device__ __forceinline__ bool locate_segment(const LinearWalk &p, int64_t item, bool rev, SegLoc &s) {
  int64_t k = 0;  // segment within the sequence
  if (item < p.N) {
    s.n = (int)item;
  } else {
    if (!p.seg) return false;
    const int64_t j = item - p.N + 1, tok = j * p.seg;
    if (p.cu) {
      if (tok >= p.cu[p.N] || tok < p.cu[0]) return false;
      int lo = 0, hi = p.N;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.cu[mid] <= tok) lo = mid;
        else hi = mid;
      }
      s.n = lo;
    } else {
      if (tok >= (int64_t)p.B * p.T) return false;
      s.n = (int)(tok / p.T);
    }
    const SlotRange sr = slot_range(p.cu, s.n, p.T);
    k = j - sr.t0 / p.seg;
    if (k < 1 || k * p.seg >= sr.len) return false;
  }
  const SlotRange sr = slot_range(p.cu, s.n, p.T);
  s.a = sr.t0;
  s.e = sr.t0 + sr.len;
  s.lo = s.a;
  s.hi = s.e;
  s.in = s.out = -1;
  if (p.seg) {
    s.lo = s.a + k * p.seg;
    s.hi = min(s.e, s.lo + p.seg);
    const int64_t before = k > 0 ? s.lo / p.seg : -1, behind = s.hi < s.e ? s.hi / p.seg : -1;
    s.in = rev ? behind : before;
    s.out = rev ? before : behind;
  }
  return true;
}

}  // namespace kda
