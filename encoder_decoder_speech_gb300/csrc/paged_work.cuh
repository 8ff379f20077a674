// How the paged attention kernels share out their work.
//
// A work item is a tile of query rows of one (sequence, K/V head): the rows are the
// sequence's new tokens times the G query heads of the K/V head, token by token. Its cost
// is its number of chunks of 64 to 256 keys, the causal limit of its last token deciding how
// many there are; an item without a visible key counts one chunk, in which its rows are
// written as zeros. All chunks of all items are numbered densely, in the order (sequence,
// head, tile, chunk), and block c of the grid takes the numbers [c * per, (c + 1) * per):
// every block has the same number of chunks whatever the lengths, and blocks working on
// one head's tiles run at the same time, so that its keys are read from L2.
//
// An item cut by a block boundary leaves one partial state per block that holds a part of
// it, and the block that arrives last merges them in order of their chunks: the result
// does not depend on who is last. A block has at most two cut items, one that began before
// its range (its partial slot 2c) and one that goes on behind it (2c + 1); the arrival
// counter of a cut item is that of the first block that holds a part of it.
#pragma once

#include "paged.cuh"
#include "ptx.cuh"

namespace cxa {

struct WorkShape {
  int G;              // query heads a K/V head
  int rows;           // rows a tile
  int chunk_shift;    // log2 of the keys a chunk
  bool coarse;        // whether items are cut into fewer, larger chunks (work_locate may set it)
  int cap;            // keys the table's row can hold
  int min_rows, max_rows;   // sequences with fewer or more query rows a head are another kernel's
  bool alone = false;       // no other kernel takes those with more: they are reported
};

// The rows of one K/V head of a sequence; 0 if the sequence is not this kernel's.
__device__ __forceinline__ int work_rows(const PagedSeq& s, const WorkShape& w) {
  const long long m = static_cast<long long>(s.n) * w.G;
  return m < w.min_rows || m > w.max_rows ? 0 : static_cast<int>(m);
}

// Keys visible to token i of a sequence.
__device__ __forceinline__ int visible_keys(const PagedSeq& s, int i, int cap) {
  return max(0, min(cap, s.kv - s.n + i + 1));
}

__device__ __forceinline__ int tile_keys(const PagedSeq& s, const WorkShape& w, int rt) {
  return visible_keys(s, min(s.n - 1, (rt * w.rows + w.rows - 1) / w.G), w.cap);
}

// Steps of 1 << chunk_shift keys of a tile.
__device__ __forceinline__ int tile_steps(const PagedSeq& s, const WorkShape& w, int rt) {
  return max(1, (tile_keys(s, w, rt) + (1 << w.chunk_shift) - 1) >> w.chunk_shift);
}

// Chunks of a tile: its steps, or, coarse, four to seven of them in each.
__device__ __forceinline__ int tile_chunks(const PagedSeq& s, const WorkShape& w, int rt) {
  const int n = tile_steps(s, w, rt);
  return w.coarse ? max(1, n >> 2) : n;
}

// The most chunks a call can have, by what the host knows of it. Kernels count in 31 bits:
// calls that could reach kCountLimit are refused.
inline long long work_bound(const PagedBatch& bt, int page_shift, int Hkv, int G, int rows, int chunk_shift) {
  const long long tiles = bt.B + static_cast<long long>(bt.n_tokens) * G / rows;      // a head
  const long long keys = static_cast<long long>(bt.width) << page_shift;
  const double bound = static_cast<double>(tiles) * Hkv * static_cast<double>((keys >> chunk_shift) + 1);
  return bound < 9e18 ? static_cast<long long>(bound) : 9000000000000000000LL;
}

// Sums that stop at the limit. Sequences overlap where q_start decreases, against its contract;
// their chunks may then pass what the host allowed for, and must not wrap around.
constexpr int kCountLimit = 0x7FFFFFFF;
__device__ __forceinline__ int count_add(int a, int b) {
  return static_cast<int>(min(static_cast<unsigned>(a) + static_cast<unsigned>(b), static_cast<unsigned>(kCountLimit)));
}

// The first step of chunk c of nc.
__device__ __forceinline__ int chunk_step(const WorkShape& w, int c, int nc, int steps) {
  return w.coarse ? static_cast<int>(static_cast<long long>(c) * steps / nc) : c;   // (rare)
}

// The tiles of a head of a sequence with m > 0 query rows in runs of equal numbers of chunks: f(first tile, tiles,
// chunks of each) until it returns false. Later tiles see no fewer keys, so that there are no more runs than
// numbers of chunks. (306 tiles of 64 rows, 153 tokens of 128 heads that share their keys: 139 us one by one, 107 in
// runs. Not for coarse chunks, and a loss of 1 % where tiles are few.)
template <typename F>
__device__ __forceinline__ void each_run(const PagedSeq& s, const WorkShape& w, int m, F f) {
  const int tiles = (m + w.rows - 1) / w.rows;
#pragma unroll 1
  for (int rt = 0; rt < tiles;) {
    const int c = tile_chunks(s, w, rt);
    // the first token that sees enough keys for one chunk more, and the tile with its first row
    const int keys = c << w.chunk_shift;
    const int i = keys - (s.kv - s.n);
    const int next = keys >= w.cap || i >= s.n ? tiles : i * w.G / w.rows;
    if (!f(rt, next - rt, c)) break;
    rt = next;
  }
}

// Chunks of one head of a sequence.
template <bool kRuns>
__device__ __forceinline__ int head_chunks(const PagedSeq& s, const WorkShape& w) {
  const int m = work_rows(s, w);
  int u = 0;
  if constexpr (kRuns)
    each_run(s, w, m, [&](int, int tiles, int c) {
      u += tiles * c;
      return true;
    });
  else
    for (int rt = 0; rt * w.rows < m; ++rt) u += tile_chunks(s, w, rt);
  return u;
}

struct WorkCursor {
  PagedSeq seq;
  int b, h, rt, c;     // c: first chunk of the item in this block's range
  int tiles;           // of a head of the sequence
  int nc;              // chunks of the item
  int first;           // number of the item's first chunk
};

struct WorkRange {
  int g0, g1;          // this block's chunk numbers
  int per;
};

// Scratch in shared memory for work_locate.
struct WorkScratch {
  int scan[2][32];
  WorkCursor cur;
};

// Number the chunks and find this block's range and the item it starts in. Called by all
// kThreads threads of the block; returns false if the block has nothing to do. With
// kMayCoarsen, w becomes coarse where a block would have less than four steps: a merge costs
// as much as some eight of them. With kRuns, tiles are counted in runs (each_run). With a
// status word, sequences whose keys pass their row of the table are reported there, whichever
// kernel they are of, those that no kernel takes, and a q_start that decreases. A batch of more chunks than can be numbered,
// which only such a q_start brings, is left out.
template <int kThreads, bool kMayCoarsen, bool kRuns = false>
__device__ bool work_locate(const PagedBatch& bt, WorkShape& w, int Hkv, WorkScratch* sm, WorkRange* range,
                            WorkCursor* cur, unsigned int* status = nullptr) {
  static_assert(!(kRuns && kMayCoarsen), "runs are of fine chunks");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int kW = kThreads / 32;
  // each thread counts a run of sequences, in fine chunks and in coarse ones
  const int each = (bt.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * each, bt.B), b1 = min(b0 + each, bt.B);
  int mine[2] = {0, 0}, incl[2], before[2] = {0, 0}, total[2] = {0, 0};
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const PagedSeq s = paged_seq(bt.q_start, bt.kv_len, b, bt.n_tokens);
    const int m = work_rows(s, w);
    if (status != nullptr && s.n > 0 && s.kv > w.cap) atomicOr(status, kStatusBadPage);
    if (status != nullptr && bt.q_start[b + 1] < bt.q_start[b]) atomicOr(status, kStatusBadBatch);
    if (status != nullptr && w.alone && static_cast<long long>(s.n) * w.G > w.max_rows) atomicOr(status, kStatusBadBatch);
    if constexpr (kRuns) {
      each_run(s, w, m, [&](int, int tiles, int c) {
        const long long all = static_cast<long long>(tiles) * c * Hkv;
        mine[0] = count_add(mine[0], static_cast<int>(min(all, static_cast<long long>(kCountLimit))));
        return true;
      });
      continue;
    }
#pragma unroll 1
    for (int rt = 0; rt * w.rows < m; ++rt) {
      const int n = tile_steps(s, w, rt);
      mine[0] = count_add(mine[0], n * Hkv);
      mine[1] = count_add(mine[1], max(1, n >> 2) * Hkv);
    }
  }
#pragma unroll
  for (int k = 0; k < (kMayCoarsen ? 2 : 1); ++k) {
    incl[k] = mine[k];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl[k], off);
      if (lane >= off) incl[k] = count_add(incl[k], o);
    }
    if (lane == 31) sm->scan[k][warp] = incl[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < (kMayCoarsen ? 2 : 1); ++k)
#pragma unroll
    for (int i = 0; i < kW; ++i) {
      if (i < warp) before[k] = count_add(before[k], sm->scan[k][i]);
      total[k] = count_add(total[k], sm->scan[k][i]);
    }
  if (total[0] == kCountLimit) return false;    // the same in every thread
  w.coarse = kMayCoarsen && total[0] < 4 * static_cast<int>(gridDim.x);
  const int k = w.coarse ? 1 : 0, blocks = static_cast<int>(gridDim.x), block = static_cast<int>(blockIdx.x);
  const int all = k ? total[1] : total[0], own = k ? mine[1] : mine[0];
  int at = k ? before[1] + incl[1] - own : before[0] + incl[0] - own;
  // (all + blocks - 1 could pass 31 bits)
  range->per = all / blocks + (all % blocks != 0 ? 1 : 0);
  const long long g0 = static_cast<long long>(range->per) * block;
  range->g0 = static_cast<int>(min(g0, static_cast<long long>(all)));
  range->g1 = static_cast<int>(min(g0 + range->per, static_cast<long long>(all)));
  if (range->g0 >= range->g1) return false;     // the same in every thread
  if (range->g0 >= at && range->g0 - at < own) {
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const PagedSeq s = paged_seq(bt.q_start, bt.kv_len, b, bt.n_tokens);
      const int u = head_chunks<kRuns>(s, w);
      if (range->g0 - at < u * Hkv) {
        WorkCursor c;
        c.seq = s;
        c.b = b;
        c.h = (range->g0 - at) / u;
        at += u * c.h;
        c.tiles = (work_rows(s, w) + w.rows - 1) / w.rows;
        if constexpr (kRuns) {
          each_run(s, w, work_rows(s, w), [&](int rt, int tiles, int chunks) {
            // (of one tile, without a division; the last one, if no run is left)
            const int in = tiles == 1 ? 0 : min((range->g0 - at) / chunks, tiles - 1);
            c.rt = rt + in;
            c.nc = chunks;
            at += in * chunks;
            const bool more = range->g0 - at >= chunks && rt + tiles < c.tiles;
            if (more) at += chunks;
            return more;
          });
        } else {
#pragma unroll 1
          for (c.rt = 0;; ++c.rt) {
            c.nc = tile_chunks(s, w, c.rt);
            if (range->g0 - at < c.nc || c.rt + 1 >= c.tiles) break;
            at += c.nc;
          }
        }
        c.first = at;
        c.c = range->g0 - at;
        sm->cur = c;
        break;
      }
      at += u * Hkv;
    }
  }
  __syncthreads();
  *cur = sm->cur;
  return true;
}

// The item after the cursor's; only called while chunks remain in the block's range.
__device__ __forceinline__ void work_next(const PagedBatch& bt, const WorkShape& w, int Hkv, WorkCursor* c) {
  c->first += c->nc;
  c->c = 0;
  if (++c->rt == c->tiles) {
    c->rt = 0;
    if (++c->h == Hkv) {
      c->h = 0;
      do {
        ++c->b;
        if (c->b >= bt.B) return;
        c->seq = paged_seq(bt.q_start, bt.kv_len, c->b, bt.n_tokens);
        c->tiles = (work_rows(c->seq, w) + w.rows - 1) / w.rows;
      } while (c->tiles == 0);
    }
  }
  c->nc = tile_chunks(c->seq, w, c->rt);
}

}  // namespace cxa
