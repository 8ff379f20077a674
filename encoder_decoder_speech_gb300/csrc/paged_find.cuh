// The look-up of a token's sequence, by a warp.
#pragma once

#include <cuda_runtime.h>

namespace cxa {

// The sequence whose rows hold token t, by the whole warp: the last b with
// q_start[b] <= t, 32 candidates a step. -1 if t lies before the first row.
__device__ __forceinline__ int find_seq(const int* q_start, int B, int t, int lane) {
  int lo = 0, len = B;   // the answer, if any, lies in [lo, lo + len)
  if (__ldg(q_start) > t) return -1;
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int at = lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, at < len && __ldg(q_start + lo + min(at, len - 1)) <= t);
    const int last = 31 - __clz(m | 1u);
    lo += last * step;
    len = min(step, len - last * step);
  }
  return lo;
}

}  // namespace cxa
