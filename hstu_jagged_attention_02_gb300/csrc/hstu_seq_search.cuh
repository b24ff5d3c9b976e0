// The sequence of a packed row, found by a whole warp.
#pragma once

#include "hstu_common.cuh"

namespace hstu {

struct FoundSeq {
  int b;
  int64_t begin, end;   // off[b], off[b + 1]
  int32_t aux;          // aux[b]
};

// The sequence b with off[b] <= t < off[b + 1], for 0 <= t < off[B] and B >= 1, by
// 32-way search: every lane reads one of 32 pivots, so a step costs one round
// trip to memory and 1,000 sequences take two.  The last round reads the
// remaining offsets and their aux entries (NULL: none) at once.  off must be
// non-decreasing; with offsets that are not, the result is some b in [0, B).
__device__ __forceinline__ FoundSeq warp_find_sequence(const int64_t* off, const int32_t* aux, int B, int64_t t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;                     // the answer lies in [lo, lo + n)
  while (n > 31) {
    const int step = (int)((unsigned)(n + 31) >> 5);
    const bool in = lane * step < n;     // pivot `lane`: first sequence of its part
    const unsigned m = __ballot_sync(0xffffffffu, in && off[lo + (in ? lane * step : 0)] <= t);
    const int k = m ? 31 - __clz(m) : 0;   // the last part that starts at or before t
    n = min(step, n - k * step);
    lo += k * step;
  }
  const int64_t o = off[lo + min(lane, n)];
  const int32_t a = aux ? aux[lo + min(lane, n - 1)] : 0;
  const unsigned m = __ballot_sync(0xffffffffu, lane < n && o <= t);
  const int k = m ? 31 - __clz(m) : 0;
  FoundSeq r;
  r.b = lo + k;
  r.begin = __shfl_sync(0xffffffffu, o, k);
  r.end = __shfl_sync(0xffffffffu, o, k + 1);
  r.aux = __shfl_sync(0xffffffffu, a, k);
  return r;
}

}  // namespace hstu
