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

// Counts all units, asks want(total) for the number of one of them (the same in every thread; below 0: none),
// and finds the sequence that holds it. Called by all kThreads threads of the block; false if
// there is none, or if there are more units than can be numbered (only numbers that the host cannot see
// bring that). units(b) >= 0.
template <int kThreads, typename F, typename G>
__device__ bool span_find(int B, F units, SpanScratch* sm, G want, int* seq, int* first) {
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
  const int g = want(total);
  if (g < 0) return false;
  int at = before + incl - mine;
  if (g >= at && g - at < mine) {
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const int u = units(b);
      if (g - at < u) {
        sm->b = b;
        sm->first = at;
        break;
      }
      at += u;
    }
  }
  __syncthreads();
  *seq = sm->b;
  *first = sm->first;
  return true;
}

// The block's equal range of all units; false if it has nothing to do.
template <int kThreads, typename F>
__device__ bool span_locate(int B, F units, SpanScratch* sm, SpanRange* r) {
  return span_find<kThreads>(
      B, units, sm,
      [&](int total) {
        const int blocks = static_cast<int>(gridDim.x), block = static_cast<int>(blockIdx.x);
        const int per = total / blocks, more = total % blocks;     // the first `more` blocks take one more
        r->g0 = per * block + min(block, more);
        r->g1 = r->g0 + per + (block < more ? 1 : 0);
        return r->g0 < r->g1 ? r->g0 : -1;
      },
      &r->b, &r->first);
}

}  // namespace cxa
