// Work that is dealt out by sequence without query rows: every sequence has a number of units (as a
// device function of its index gives), all units are numbered densely, and block c of the grid takes
// an equal range of the numbers.
#pragma once

#include "paged.cuh"
#include "paged_work.cuh"

namespace cxa {

struct SpanScratch {
  int scan[32];
  int b, first;        // the sequence that the block's range starts in, and the number of its first unit
};

struct SpanRange {
  int g0, g1;          // this block's units
  int b, first;
};

// Called by all kThreads threads of the block; false if the block has nothing to do. units(b) >= 0. A
// batch of more units than can be numbered is left out (only numbers that the host cannot see
// bring one).
template <int kThreads, typename F>
__device__ bool span_locate(int B, F units, SpanScratch* sm, SpanRange* r) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = (B + kThreads - 1) / kThreads;
  const int b0 = min(tid * each, B), b1 = min(b0 + each, B);
  int mine = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) mine = count_add(mine, units(b));
  int incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl = count_add(incl, o);
  }
  if (lane == 31) sm->scan[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before = count_add(before, sm->scan[i]);
    total = count_add(total, sm->scan[i]);
  }
  if (total == kCountLimit || total == 0) return false;
  const int blocks = static_cast<int>(gridDim.x), block = static_cast<int>(blockIdx.x);
  const int per = total / blocks, more = total % blocks;     // the first `more` blocks take one more
  r->g0 = per * block + min(block, more);
  r->g1 = r->g0 + per + (block < more ? 1 : 0);
  if (r->g0 >= r->g1) return false;
  int at = before + incl - mine;
  if (r->g0 >= at && r->g0 - at < mine) {
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const int u = units(b);
      if (r->g0 - at < u) {
        sm->b = b;
        sm->first = at;
        break;
      }
      at += u;
    }
  }
  __syncthreads();
  r->b = sm->b;
  r->first = sm->first;
  return true;
}

}  // namespace cxa
