// The sequence of a packed row, found by a whole warp.
#pragma once

#include "hstu_common.cuh"

namespace hstu {

// The sequence b with off[b] <= t < off[b + 1], for 0 <= t < off[B], by 32-way
// search: every lane reads one of 32 pivots, so a step costs one round trip
// to memory and 1,024 sequences take two.  off must be non-decreasing; with
// offsets that are not, the result is some b in [0, B).
__device__ __forceinline__ int warp_find_sequence(const int64_t* off, int B, int64_t t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;                     // the answer lies in [lo, lo + n)
  while (n > 1) {
    const int step = (int)((unsigned)(n + 31) >> 5);
    const int at = lo + lane * step;     // pivot `lane`: first sequence of its part
    const bool below = lane * step < n && off[at] <= t;
    const unsigned m = __ballot_sync(0xffffffffu, below);
    const int k = m ? 31 - __clz(m) : 0;   // the last part that starts at or before t
    n = min(step, n - k * step);
    lo += k * step;
  }
  return lo;
}

}  // namespace hstu
