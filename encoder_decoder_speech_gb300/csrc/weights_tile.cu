// The attention weight that keys of a paged bf16 cache gather, as tcgen05 products.
//
//   ref_r = log2 sum_j 2^s_rj,   W_j = decay W_j + sum_r 2^(s_rj - ref_r),   s = scale log2(e) q K^T
//
// Many query rows (prompts), two passes over the scores:
//   weights_ref_kernel   dealt out as the attention is: 256 query rows of a K/V head in two tiles of 128
//                        against 128 keys a step. A thread has a row: its running reference and sum need no
//                        other thread.
//   weights_sum_kernel   the transposed product: a block has 128 keys, a thread one of them, and goes
//                        over all tiles of 128 query rows that see them. A thread adds up its own key's weights,
//                        so that every W is written once and in one order.
// Both are bound by the exponentials, 32 a clock of an SM: 512 clocks for 128 x 128 scores, against 256 (64
// channels) or 512 (128) for their product. 2048 tokens over 8192 keys of 20 heads of 64: 144 us, the exponential
// units busy 44 and 41 % of the two passes: two warps a scheduler do not cover each other's waits and reads of
// tensor memory (registers alone: 82 %). Tried: a second warp for the products and 16 softmax warps, no gain; 64
// columns at a time with the next ones on their way, 183 us; sums with a reference that seldom moves, 170 us.
//
// Few query rows (16 a K/V head at most: single tokens, in a batch of their own or beside prompts, see
// weights_split), bound by reading K:
//   weights_few_kernel   the transposed product again, of 128 keys by 16 rows; a thread has a key, keeps
//                        references and sums of its own until the item's end, and stores the scores (4 bytes a row
//                        and key, against 2 dh bytes of the key itself).
//   weights_add_kernel   (weights_few.cu) reads the scores back and adds the weights to W.
// 64 single tokens, 32 heads on 8 of 128, over 282,119 keys: 124 us, 104 of them the first at 5.7 TB/s.
// Where the scores have no room, the second pass is weights_sum_kernel, which reads K once more (ScoreRule).
//
// Products of bf16 values are exact; sums, references and weights are fp32.
#include <cuda.h>
#include <cuda_bf16.h>

#include <cmath>

#include "paged_work.cuh"
#include "ptx.cuh"
#include "span_work.cuh"
#include "tc_util.cuh"
#include "weights_few.cuh"

namespace cxa {
namespace {

constexpr int kKeys = kFewKeys, kChunkShift = kFewChunkShift;
constexpr int kUnitBytes = 16384;               // 64 channels of 128 keys or query rows
constexpr int kSmemBytes = 232448, kSmallBytes = 6144;
constexpr int kTileRows = 128;

struct WeightsParams {
  const __nv_bfloat16* q;
  long long q_stride;
  float* W;
  float decay, qscale;
  unsigned int* counters;
  float* ref;               // [Hkv][n_tokens][G]
  float* part;              // [2 * grid][rows][2]
  float* scores;            // of chunk c, row r: [c * rule.max_rows + r][kKeys]
  ScoreRule rule;
  unsigned int* status;
  PagedBatch batch;
  int num_pages, Hkv, page_shift;
  WorkShape shape;
};

__device__ __forceinline__ int lookup(const WeightsParams& p, int b, int t) {
  return paged_lookup(p.batch.table + static_cast<size_t>(b) * p.batch.width, p.batch.width, p.page_shift, p.num_pages, t);
}
// A value that every lane has, known as such: operands' addresses need no carrying over from a lane then, which
// takes longer than a product of 32 clocks.
__device__ __forceinline__ uint32_t same_in_all(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ float* refs_of(const WeightsParams& p, const PagedSeq& s, int h) {
  return p.ref + (static_cast<size_t>(h) * p.batch.n_tokens + s.q0) * p.shape.G;
}

// A warp's copies of 128 keys of head h, 64 channels a unit, into units of a ring: a lane a box.
template <int kUnits>
struct KeyCopies {
  int pos;
  uint32_t round, armed, parity;
  int full, empty;           // first barriers of the ring
  int ring;                  // units
  uint32_t base;
  // `bad`, if given, gets the groups of 16 keys whose page is outside the pool. False if a wait ran out.
  __device__ bool step(const WeightsParams& p, const CUtensorMap* map, Waits& w, int b, int h, int key0, int keys,
                       volatile uint32_t* bad) {
    const int lane = threadIdx.x & 31;
    const int box_shift = min(p.page_shift, kChunkShift), box_rows = 1 << box_shift, boxes = kKeys >> box_shift;
    const int box = lane % boxes, at = key0 + box * box_rows;
    const bool want = lane < boxes && at < keys;
    const int page = want ? lookup(p, b, at) : -2;
    const uint32_t good = __ballot_sync(0xffffffffu, page >= 0), gone = __ballot_sync(0xffffffffu, page == -1);
    const int y = at & ((1 << p.page_shift) - 1);
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      if (!w.warp(empty + pos, (round & 1) ^ 1, kStatusTimeout)) return false;
      if (lane == 0) {
        if (u == 0) {
          if (bad != nullptr) {
            uint32_t groups = 0;
            for (uint32_t m = gone; m != 0; m &= m - 1)
              groups |= ((1u << (box_rows / 16)) - 1u) << ((__ffs(m) - 1) * (box_rows / 16));
            *bad = groups;
          }
          if (gone != 0) atomicOr(p.status, kStatusBadPage);
        }
        mbar_arrive_expect_tx(w.bar(full + pos), static_cast<uint32_t>(__popc(good) * box_rows * 128));
      }
      __syncwarp();
      if (page >= 0)
        tma_load_3d(base + pos * kUnitBytes + box * box_rows * 128, map, w.bar(full + pos), u * 64, y, page * p.Hkv + h);
      armed |= 1u << pos;
      parity = (parity & ~(1u << pos)) | (round & 1u) << pos;
      if (++pos == ring) {
        pos = 0;
        ++round;
      }
    }
    return true;
  }
  // After a wait that ran out: the copies under way land before the block ends.
  __device__ void drain(const Waits& w) const {
    for (int b = 0; b < ring; ++b)
      if (armed & (1u << b)) mbar_wait(w.bar(full + b), (parity >> b) & 1u);
  }
};

// ============================================================================ few rows
namespace few {

constexpr int kRows = kScoreRows;
constexpr int kThreads = 6 * 32, kMmaWarp = 4, kTmaWarp = 5;
constexpr int kBufs = 4;               // of S^T
constexpr int kRing = 12;
enum Bars { kQFull = 0, kSFull = 1, kSFree = kSFull + kBufs, kUFull = kSFree + kBufs, kUEmpty = kUFull + kRing, kBars = kUEmpty + kRing };
struct Small {
  uint64_t bars[kBars];
  WorkScratch work;
  uint32_t bad[32];           // (copies run up to 16 steps ahead of who reads it)
  volatile int abort;
  int tmem;
  FewShared few;
};
static_assert(sizeof(Small) <= kSmallBytes, "the small arrays fit");
constexpr uint32_t kTmemCols = 64;

template <int kDh>
__global__ void __launch_bounds__(kThreads, 1)
    weights_few_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ WeightsParams p) {
  constexpr int kUnits = kDh / 64;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t u_base = smem_u32(smem), q_base = u_base + kRing * kUnitBytes;
  Small* sm = reinterpret_cast<Small*>(smem + kSmemBytes - kSmallBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedBatch& bt = p.batch;
  const int G = p.shape.G;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  WorkRange range;
  WorkCursor cur;
  WorkShape shape = p.shape;
  const bool kept = p.rule.ask ? score_ask<kThreads>(p.rule, bt, G, p.Hkv, shape.cap, &sm->work) : p.rule.kept;
  if (!kept && p.rule.others) return;      // these sequences go with those of many
  if (!work_locate<kThreads, false>(bt, shape, p.Hkv, &sm->work, &range, &cur, p.status)) return;
  Waits w = {smem_u32(sm->bars), &sm->abort, p.status, true};
  if (tid == 0) {
    for (int i = 0; i < kBars; ++i) mbar_init(w.bar(i), i == kQFull || (i >= kSFree && i < kUFull) ? 4 : 1);
    fence_mbar_init();
    sm->abort = 0;
  }
  if (warp == kTmaWarp && lane == 0) prefetch_tmap(&tmK);
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&sm->tmem), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = same_in_all(static_cast<uint32_t>(sm->tmem));
  const int n_chunks = range.g1 - range.g0;

  if (warp == kTmaWarp) {
    fence_proxy_async_global();
    KeyCopies<kUnits> kc = {0, 0u, 0u, 0u, kUFull, kUEmpty, kRing / kUnits * kUnits, u_base};
    int c = cur.c;
    for (int i = 0; i < n_chunks; ++i) {
      if (!kc.step(p, &tmK, w, cur.b, cur.h, c * kKeys, tile_keys(cur.seq, shape, cur.rt), &sm->bad[i & 31])) break;
      if (++c == cur.nc && i + 1 < n_chunks) {
        work_next(bt, shape, p.Hkv, &cur);
        c = 0;
      }
    }
    if (!w.ok) kc.drain(w);
  } else if (warp == kMmaWarp) {
    constexpr uint32_t idesc = make_idesc(1u, kKeys, kRows);
    constexpr uint64_t hi = desc_high(1024);
    const uint32_t ub = same_in_all(u_base), qb = same_in_all(q_base);
    int pos = 0, item = 0, c = cur.c;
    uint32_t round = 0;
    bool fresh = true;
    for (int i = 0; i < n_chunks; ++i) {
      if (fresh && !w.warp(kQFull, item & 1, kStatusTimeout)) break;
      fresh = false;
      const int buf = i % kBufs;
      if (!w.warp(kSFree + buf, ((i / kBufs) & 1) ^ 1, kStatusTimeout)) break;
#pragma unroll
      for (int u = 0; u < kUnits; ++u) {
        if (!w.warp(kUFull + pos, round & 1, kStatusTimeout)) break;
        tc_fence_after();
        const int at = __shfl_sync(0xffffffffu, pos | buf << 8, 0);
        const uint32_t al = desc_low(ub + (at & 255) * kUnitBytes, 16), bl = desc_low(qb + u * (kRows * 128), 16);
        const uint32_t d = tmem + (at >> 8) * kRows;
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_bf16(d, hi | (al + 2 * k), hi | (bl + 2 * k), idesc, u + k != 0 ? 1u : 0u);
          tc_commit(w.bar(kUEmpty + pos));
          if (u + 1 == kUnits) tc_commit(w.bar(kSFull + buf));
        }
        __syncwarp();
        if (++pos == kRing / kUnits * kUnits) {
          pos = 0;
          ++round;
        }
      }
      if (!w.ok) break;
      if (++c == cur.nc && i + 1 < n_chunks) {
        work_next(bt, shape, p.Hkv, &cur);
        c = 0;
        ++item;
        fresh = true;
      }
    }
    __syncwarp();
  } else {
    // a key a thread
    const uint32_t my_tmem = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    int i = 0;
    for (;;) {
      const int end = min(range.g1, cur.first + cur.nc), c0 = cur.c, c1 = end - cur.first;
      const PagedSeq seq = cur.seq;
      const int rows = work_rows(seq, shape);      // one tile an item: kRows at most
      const int see_all = visible_keys(seq, 0, shape.cap);
      // the rows' queries (the scores of the item before have been taken)
      for (int e = tid; e < kRows * (kDh / 8); e += 128) {
        const int r = e / (kDh / 8), j = e % (kDh / 8);
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows)
          v = *reinterpret_cast<const uint4*>(p.q + (seq.q0 + r / G) * p.q_stride +
                                              static_cast<long long>(cur.h * G + r % G) * kDh + j * 8);
        st_shared_v4(q_base + (j >> 3) * (kRows * 128) + r * 128 + (((j & 7) ^ (r & 7)) << 4), v.x, v.y, v.z, v.w);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(w.bar(kQFull));
      float m[kRows], l[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
      }
      for (int c = c0; c < c1; ++c, ++i) {
        const int buf = i % kBufs, key = c * kKeys + tid;
        w.warp(kSFull + buf, (i / kBufs) & 1, kStatusTimeout);
        tc_fence_after();
        uint32_t x[kRows];
        tmem_ld_32x32b_x16(my_tmem + buf * kRows, x);
        tmem_ld_wait();
        const uint32_t bad = *const_cast<volatile uint32_t*>(&sm->bad[i & 31]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(w.bar(kSFree + buf));
        const bool gone = (bad >> (tid >> 4) & 1u) != 0 || key >= shape.cap;
        const bool edge = (c + 1) * kKeys > see_all;
        float* to = kept ? p.scores + static_cast<size_t>(cur.first + c) * p.rule.max_rows * kKeys + tid : nullptr;
        const int hidden = gone ? kRows : edge ? min(max(key - (seq.kv - seq.n), 0), kRows) * G : 0;
        float s[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) s[r] = __uint_as_float(x[r]);
        few_take(s, rows, hidden, p.qscale, to, m, l);
      }
      few_finish(&sm->few, m, l, rows, cur, range, c0, c1, w.ok, p.part, p.counters, refs_of(p, seq, cur.h));
      if (end >= range.g1) break;
      work_next(bt, shape, p.Hkv, &cur);
      asm volatile("bar.sync 1, 128;" ::: "memory");
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace few

// ============================================================================ many rows: references
namespace many {

constexpr int kTiles = 2;
constexpr int kThreads = 10 * 32, kMmaWarp = 8, kTmaWarp = 9;
template <int kDh>
struct Cfg {
  static constexpr int units = kDh / 64;                     // of a step's keys, and of a tile's query rows
  static constexpr int q_bytes = kTiles * units * kUnitBytes;
  static constexpr int ring = (kSmemBytes - kSmallBytes - q_bytes) / kUnitBytes / units * units;
};
constexpr int kMaxRing = 12;
enum Bars { kQFull = 0, kQEmpty = 1, kSFull = 2, kSFree = kSFull + 4, kUFull = kSFree + 4, kUEmpty = kUFull + kMaxRing, kBars = kUEmpty + kMaxRing };
struct Small {
  uint64_t bars[kBars];
  WorkScratch work;
  uint32_t bad[32];           // (copies run up to 16 steps ahead of who reads it)
  volatile int abort;
  int tmem, last;
};
static_assert(sizeof(Small) <= kSmallBytes, "the small arrays fit");

template <int kDh>
__global__ void __launch_bounds__(kThreads, 1)
    weights_ref_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ WeightsParams p) {
  using C = Cfg<kDh>;
  static_assert(C::ring <= kMaxRing, "barriers");
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t q_base = smem_u32(smem), u_base = q_base + C::q_bytes;
  Small* sm = reinterpret_cast<Small*>(smem + kSmemBytes - kSmallBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedBatch& bt = p.batch;
  const int G = p.shape.G, tile_rows = p.shape.rows / kTiles;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  WorkRange range;
  WorkCursor cur;
  WorkShape shape = p.shape;
  if (!scores_kept(p.rule)) shape.min_rows = 0;      // those of few rows too
  if (!work_locate<kThreads, false>(bt, shape, p.Hkv, &sm->work, &range, &cur, p.status)) return;
  Waits w = {smem_u32(sm->bars), &sm->abort, p.status, true};
  if (tid == 0) {
    for (int i = 0; i < kBars; ++i) mbar_init(w.bar(i), i >= kSFree && i < kUFull ? 4 : 1);
    fence_mbar_init();
    sm->abort = 0;
  }
  if (warp == kTmaWarp && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&sm->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = same_in_all(static_cast<uint32_t>(sm->tmem));
  const int n_chunks = range.g1 - range.g0;
  auto tiles_of = [&](const WorkCursor& c) { return work_rows(c.seq, shape) - c.rt * shape.rows > tile_rows ? 2 : 1; };

  if (warp == kTmaWarp) {
    fence_proxy_async_global();
    KeyCopies<C::units> kc = {0, 0u, 0u, 0u, kUFull, kUEmpty, C::ring, u_base};
    int c = cur.c, item = 0;
    bool fresh = true, q_sent = false;
    for (int i = 0; i < n_chunks; ++i) {
      if (fresh) {
        if (!w.warp(kQEmpty, (item & 1) ^ 1, kStatusTimeout)) break;
        const int boxes = tiles_of(cur) * C::units;
        if (lane == 0) mbar_arrive_expect_tx(w.bar(kQFull), static_cast<uint32_t>(boxes * tile_rows * 128));
        __syncwarp();
        if (lane < boxes)
          tma_load_3d(q_base + lane * kUnitBytes, &tmQ, w.bar(kQFull), (lane % C::units) * 64, cur.h * G,
                      cur.seq.q0 + (cur.rt * kTiles + lane / C::units) * (tile_rows / G));
        q_sent = true;
        fresh = false;
      }
      if (!kc.step(p, &tmK, w, cur.b, cur.h, c * kKeys, tile_keys(cur.seq, shape, cur.rt), &sm->bad[i & 31])) break;
      if (++c == cur.nc && i + 1 < n_chunks) {
        work_next(bt, shape, p.Hkv, &cur);
        c = 0;
        ++item;
        fresh = true;
      }
    }
    if (!w.ok) {
      if (q_sent) mbar_wait(w.bar(kQFull), static_cast<uint32_t>((fresh ? item - 1 : item) & 1));
      kc.drain(w);
    }
  } else if (warp == kMmaWarp) {
    constexpr uint32_t idesc = make_idesc(1u, kTileRows, kKeys);
    constexpr uint64_t hi = desc_high(1024);
    const uint32_t ub = same_in_all(u_base), qb = same_in_all(q_base);
    int pos = 0, item = 0, c = cur.c, used[kTiles] = {0, 0}, tiles = tiles_of(cur);
    uint32_t round = 0;
    bool fresh = true;
    for (int i = 0; i < n_chunks && w.ok; ++i) {
      if (fresh && !w.warp(kQFull, item & 1, kStatusTimeout)) break;
      fresh = false;
      const bool last = c + 1 == cur.nc || i + 1 == n_chunks;
      for (int t = 0; t < tiles; ++t) {
        const int buf = t * 2 + (used[t] & 1);
        if (!w.warp(kSFree + buf, ((used[t] >> 1) & 1) ^ 1, kStatusTimeout)) break;
        ++used[t];
        int at = pos;
        uint32_t rd = round;
#pragma unroll
        for (int u = 0; u < C::units; ++u) {
          if (!w.warp(kUFull + at, rd & 1, kStatusTimeout)) break;
          tc_fence_after();
          const uint32_t all = same_in_all(static_cast<uint32_t>(at | buf << 8 | t << 16));
          const uint32_t al = desc_low(qb + ((all >> 16) * C::units + u) * kUnitBytes, 16);
          const uint32_t bl = desc_low(ub + (all & 255) * kUnitBytes, 16), d = tmem + (all >> 8 & 255) * kKeys;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_bf16(d, hi | (al + 2 * k), hi | (bl + 2 * k), idesc, u + k != 0 ? 1u : 0u);
            if (t + 1 == tiles) tc_commit(w.bar(kUEmpty + at));
            if (u + 1 == C::units) {
              tc_commit(w.bar(kSFull + buf));
              if (t + 1 == tiles && last) tc_commit(w.bar(kQEmpty));
            }
          }
          __syncwarp();
          if (++at == C::ring) {
            at = 0;
            ++rd;
          }
        }
        if (t + 1 == tiles) {
          pos = at;
          round = rd;
        }
      }
      if (++c == cur.nc && i + 1 < n_chunks) {
        work_next(bt, shape, p.Hkv, &cur);
        c = 0;
        ++item;
        fresh = true;
        tiles = tiles_of(cur);
      }
    }
    __syncwarp();
  } else {
    // a query row a thread
    const int t = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t my_tmem = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const float2 qs2 = make_float2(p.qscale, p.qscale);
    int i = 0, used = 0;
    for (;;) {
      const int end = min(range.g1, cur.first + cur.nc), c0 = cur.c, c1 = end - cur.first;
      const PagedSeq seq = cur.seq;
      const int row0 = cur.rt * shape.rows + t * tile_rows;
      const int rows = max(0, min(tile_rows, work_rows(seq, shape) - row0));
      const bool real = r < rows;
      float m = -INFINITY, l = 0.f;
      if (rows > 0 && (warp & 3) * 32 >= rows) {      // (none of this warp's rows is a token's)
        for (int c = c0; c < c1; ++c, ++used) {
          w.warp(kSFull + t * 2 + (used & 1), (used >> 1) & 1, kStatusTimeout);
          __syncwarp();
          if (lane == 0) mbar_arrive(w.bar(kSFree + t * 2 + (used & 1)));
        }
      } else if (rows > 0) {
        // (rows of no token go without masks: nothing of theirs is written)
        const int see = real ? visible_keys(seq, (row0 + r) / G, shape.cap) : 0x7FFFFFFF;
        const int see_all = visible_keys(seq, row0 / G, shape.cap);
        for (int c = c0; c < c1; ++c, ++used) {
          const int buf = t * 2 + (used & 1), key0 = c * kKeys;
          w.warp(kSFull + buf, (used >> 1) & 1, kStatusTimeout);
          tc_fence_after();
          const uint32_t bad = *const_cast<volatile uint32_t*>(&sm->bad[(i + c - c0) & 31]);
          const bool edge = key0 + kKeys > see_all || bad != 0;
          uint32_t x[4][32];
#pragma unroll
          for (int q = 0; q < 4; ++q) tmem_ld_32x32b_x32(my_tmem + buf * kKeys + q * 32, x[q]);
          tmem_ld_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(w.bar(kSFree + buf));
          if (__builtin_expect(edge, 0)) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const int k = q * 32 + e;
                if (key0 + k >= see || (bad >> (k >> 4) & 1u) != 0) x[q][e] = 0xFF800000u;      // -inf
              }
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              mx[(e / 2) & 3] = max_of_3(mx[(e / 2) & 3], __uint_as_float(x[q][e]), __uint_as_float(x[q][e + 1]));
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.qscale;
          const float up = fmaxf(m, top);
          l *= few_rescale(m, up);
          m = up;
          const float ref = m == -INFINITY ? 0.f : -m;
          const float2 ref2 = make_float2(ref, ref);
          float2 sum[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[e] = make_float2(0.f, 0.f);
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float2 v = fma_pair(make_float2(__uint_as_float(x[q][e]), __uint_as_float(x[q][e + 1])), qs2, ref2);
              v.x = ex2(v.x);
              v.y = ex2(v.y);
              sum[(e >> 1) & 3] = add_pair(sum[(e >> 1) & 3], v);
            }
          sum[0] = add_pair(add_pair(sum[0], sum[1]), add_pair(sum[2], sum[3]));
          l += sum[0].x + sum[0].y;
        }
      }
      i += c1 - c0;
      // ---- the part in this range
      float* refs = refs_of(p, seq, cur.h);
      if (c0 == 0 && c1 == cur.nc) {
        if (real && w.ok) refs[row0 + r] = log_sum(m, l);
      } else {
        constexpr int kSlot = kTiles * kTileRows * 2;
        float* slot = p.part + (2 * static_cast<size_t>(blockIdx.x) + (c0 == 0 ? 1 : 0)) * kSlot;
        slot[t * kTileRows + r] = m;
        slot[kTiles * kTileRows + t * kTileRows + r] = l;
        const int owner = cur.first / range.per, parts = (cur.first + cur.nc - 1) / range.per - owner + 1;
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (tid == 0) {
          bool last = false;
          if (w.ok) {
            last = atomic_add_acq_rel_gpu(p.counters + owner, 1u) == static_cast<unsigned int>(parts - 1);
            if (last) p.counters[owner] = 0u;
          }
          sm->last = last;
        }
        asm volatile("bar.sync 1, 256;" ::: "memory");
        if (sm->last != 0 && real) {
          auto part = [&](int k) {
            return p.part + (2 * static_cast<size_t>(owner + k) + (k == 0 ? 1 : 0)) * kSlot + t * kTileRows + r;
          };
          float M = -INFINITY, L = 0.f;
#pragma unroll 4
          for (int k = 0; k < parts; ++k) M = fmaxf(M, __ldcg(part(k)));
#pragma unroll 4
          for (int k = 0; k < parts; ++k) L += __ldcg(part(k) + kTiles * kTileRows) * few_rescale(__ldcg(part(k)), M);
          refs[row0 + r] = log_sum(M, L);
        }
      }
      if (end >= range.g1) break;
      work_next(bt, shape, p.Hkv, &cur);
      __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

}  // namespace many

// ============================================================================ many rows: sums
namespace sum {

constexpr int kThreads = 10 * 32, kMmaWarp = 8, kTmaWarp = 9;
constexpr int kBufs = 4;
template <int kDh>
struct Cfg {
  static constexpr int units = kDh / 64;
  static constexpr int k_ring = 2 * units;                        // two tiles of keys
  static constexpr int q_ring = (kSmemBytes - kSmallBytes) / kUnitBytes / units - 2;     // tiles of query rows
};
constexpr int kMaxK = 4, kMaxQ = 12;
enum Bars {
  kKFull = 0,
  kKEmpty = kKFull + kMaxK,
  kQFull = kKEmpty + kMaxK,
  kQEmpty = kQFull + kMaxQ,
  kSFull = kQEmpty + kMaxQ,
  kSFree = kSFull + kBufs,
  kBars = kSFree + kBufs
};
struct Small {
  uint64_t bars[kBars];
  SpanScratch span;
  volatile int abort;
  int tmem;
  __align__(16) float ref[2][2][kTileRows];      // minus the references, of a group's tile, two of them
  float sums[2][kKeys];
  int odd[2];              // of two units: n + 1 if a reference of the n-th is NaN
};
static_assert(sizeof(Small) <= kSmallBytes, "the small arrays fit");

// One K/V head and 128 keys of a sequence, and the tiles of query rows that see some of them.
struct Unit {
  PagedSeq seq;
  int b, h, key0, keys;
  int t0, t1;              // tiles
};

// kAsk: whether the scores of few rows were kept is for the first kernel to say. (In one kernel with the other case,
// the products' loop was laid out worse: 148 us in place of 145.)
template <int kDh, bool kAsk>
__global__ void __launch_bounds__(kThreads, 1)
    weights_sum_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ WeightsParams p) {
  using C = Cfg<kDh>;
  static_assert(C::q_ring <= kMaxQ && C::k_ring <= kMaxK, "barriers");
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t k_base = smem_u32(smem), q_base = k_base + C::k_ring * kUnitBytes;
  Small* sm = reinterpret_cast<Small*>(smem + kSmemBytes - kSmallBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedBatch& bt = p.batch;
  const int G = p.shape.G, cap = p.shape.cap, tile_rows = kTileRows / G * G;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // All units are numbered by (sequence, keys, head), and block c takes every grid-th of them: keys that few
  // rows see stand behind those that many do, so that all blocks get some of both.
  WorkShape shape = p.shape;
  if (kAsk && !scores_kept(p.rule)) shape.min_rows = 0;      // those of few rows too
  auto key_tiles = [&](int b) {
    const PagedSeq s = paged_seq(bt.q_start, bt.kv_len, b, bt.n_tokens);
    return work_rows(s, kAsk ? shape : p.shape) == 0 ? 0 : (min(s.kv, cap) + kKeys - 1) / kKeys;
  };
  auto units_of = [&](int b) {
    const long long u = static_cast<long long>(key_tiles(b)) * p.Hkv;
    return static_cast<int>(min(u, static_cast<long long>(kCountLimit)));
  };
  int total = 0;
  {
    // (the sum of all sequences' units)
    int mine = 0;
    for (int b = tid; b < bt.B; b += kThreads) mine = count_add(mine, units_of(b));
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) mine = count_add(mine, __shfl_xor_sync(0xffffffffu, mine, off));
    if (lane == 0) sm->span.scan[warp] = mine;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) total = count_add(total, sm->span.scan[i]);
  }
  if (total == kCountLimit || static_cast<int>(blockIdx.x) >= total) return;
  Waits w = {smem_u32(sm->bars), &sm->abort, p.status, true};
  // rows of a tile that no copy fills (heads that do not divide 128)
  for (int e = tid; e < C::q_ring * C::units * (kTileRows - tile_rows) * 8; e += kThreads) {
    const int u = e / ((kTileRows - tile_rows) * 8), o = e % ((kTileRows - tile_rows) * 8);
    st_shared_v4(q_base + u * kUnitBytes + tile_rows * 128 + o * 16, 0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  if (tid == 0) {
    for (int i = 0; i < kBars; ++i) mbar_init(w.bar(i), i >= kSFree ? 4 : 1);
    fence_mbar_init();
    sm->abort = 0;
    sm->odd[0] = sm->odd[1] = 0;
  }
  if (warp == kTmaWarp && lane == 0) {
    prefetch_tmap(&tmQ);
    prefetch_tmap(&tmK);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&sm->tmem), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = same_in_all(static_cast<uint32_t>(sm->tmem));

  // this block's units, in order; each role walks them by itself
  int u = static_cast<int>(blockIdx.x), b = 0, first = 0;
  auto next_unit = [&](Unit* out) {
    if (u >= total) return false;
    for (int n = units_of(b); u - first >= n; n = units_of(b)) {
      first += n;
      ++b;
    }
    out->seq = paged_seq(bt.q_start, bt.kv_len, b, bt.n_tokens);
    out->b = b;
    out->h = (u - first) % p.Hkv;
    out->key0 = (u - first) / p.Hkv * kKeys;
    out->keys = min(out->seq.kv, cap);
    const int i0 = min(max(0, out->key0 - (out->seq.kv - out->seq.n)), out->seq.n - 1);   // first token that sees a key
    out->t0 = static_cast<int>(static_cast<long long>(i0) * G / tile_rows);
    out->t1 = static_cast<int>((static_cast<long long>(out->seq.n) * G + tile_rows - 1) / tile_rows);
    u += static_cast<int>(gridDim.x);
    return true;
  };
  Unit un;

  if (warp == kTmaWarp) {
    fence_proxy_async_global();
    KeyCopies<C::units> kc = {0, 0u, 0u, 0u, kKFull, kKEmpty, C::k_ring, k_base};
    int pos = 0;
    uint32_t round = 0, armed = 0, parity = 0;
    while (w.ok && next_unit(&un)) {
      if (!kc.step(p, &tmK, w, un.b, un.h, un.key0, un.keys, nullptr)) break;
      for (int t = un.t0; t < un.t1; ++t) {
        if (!w.warp(kQEmpty + pos, (round & 1) ^ 1, kStatusTimeout)) break;
        if (lane == 0) mbar_arrive_expect_tx(w.bar(kQFull + pos), static_cast<uint32_t>(C::units * tile_rows * 128));
        __syncwarp();
        if (lane < C::units)
          tma_load_3d(q_base + (pos * C::units + lane) * kUnitBytes, &tmQ, w.bar(kQFull + pos), lane * 64, un.h * G,
                      un.seq.q0 + t * (tile_rows / G));
        armed |= 1u << pos;
        parity = (parity & ~(1u << pos)) | (round & 1u) << pos;
        if (++pos == C::q_ring) {
          pos = 0;
          ++round;
        }
      }
    }
    if (!w.ok) {
      kc.drain(w);
      for (int i = 0; i < C::q_ring; ++i)
        if (armed & (1u << i)) mbar_wait(w.bar(kQFull + i), (parity >> i) & 1u);
    }
  } else if (warp == kMmaWarp) {
    constexpr uint32_t idesc = make_idesc(1u, kKeys, kTileRows);
    constexpr uint64_t hi = desc_high(1024);
    const uint32_t kbase = same_in_all(k_base), qb = same_in_all(q_base);
    int pos = 0, kb = 0, j = 0;
    uint32_t round = 0, k_round = 0;
    while (w.ok && next_unit(&un)) {
      for (int i = 0; i < C::units; ++i)
        if (!w.warp(kKFull + kb * C::units + i, k_round & 1, kStatusTimeout)) break;
      for (int t = un.t0; t < un.t1 && w.ok; ++t, ++j) {
        const int buf = j % kBufs;
        if (!w.warp(kSFree + buf, ((j / kBufs) & 1) ^ 1, kStatusTimeout) || !w.warp(kQFull + pos, round & 1, kStatusTimeout))
          break;
        tc_fence_after();
        const uint32_t all = same_in_all(static_cast<uint32_t>(pos | buf << 8 | kb << 16));
        const uint32_t al = desc_low(kbase + (all >> 16) * C::units * kUnitBytes, 16);
        const uint32_t bl = desc_low(qb + (all & 255) * C::units * kUnitBytes, 16), d = tmem + (all >> 8 & 255) * kTileRows;
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < C::units; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_bf16(d, hi | (al + (i * kUnitBytes >> 4) + 2 * k), hi | (bl + (i * kUnitBytes >> 4) + 2 * k), idesc,
                       i + k != 0 ? 1u : 0u);
          tc_commit(w.bar(kQEmpty + pos));
          if (t + 1 == un.t1)
            for (int i = 0; i < C::units; ++i) tc_commit(w.bar(kKEmpty + kb * C::units + i));
          tc_commit(w.bar(kSFull + buf));
        }
        __syncwarp();
        if (++pos == C::q_ring) {
          pos = 0;
          ++round;
        }
      }
      if (++kb == 2) {
        kb = 0;
        ++k_round;
      }
    }
    __syncwarp();
  } else {
    // a key a thread; a group of four warps takes every other tile
    const int grp = warp >> 2, k = (warp & 3) * 32 + lane;
    const uint32_t my_tmem = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const float2 qs2 = make_float2(p.qscale, p.qscale);
    int j = 0, mine = 0, unit = 0;
    while (next_unit(&un)) {
      const float* refs = refs_of(p, un.seq, un.h);
      const int all = un.seq.n * G, key = un.key0 + k, past = un.seq.kv - un.seq.n;
      // the key's place and old weight, on their way under the products
      float* W = nullptr;
      float old = 0.f;
      if (grp == 0 && key < un.keys) {
        const int page = lookup(p, un.b, key);
        if (page >= 0) {
          W = p.W + ((static_cast<size_t>(page) * p.Hkv + un.h) << p.page_shift) + (key & ((1 << p.page_shift) - 1));
          if (key < past && p.decay != 0.f) old = *W;
        }
      }
      float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      int t = un.t0 + ((j + grp) & 1);
      auto fetch = [&](int tile) {
        const int at = tile * tile_rows + k;
        return tile < un.t1 && k < tile_rows && at < all ? -__ldcg(refs + at) : -INFINITY;
      };
      float nref = fetch(t);
      uint32_t odd = 0;        // above infinity's bits: a reference of the unit is NaN
      for (; t < un.t1; t += 2, ++mine) {
        const int at = j + (t - un.t0), buf = at % kBufs;
        float* rs = sm->ref[grp][mine & 1];
        // (a reference that is NaN as infinity, weights of 0: it must not reach keys that its row does not see. A store to
        // sm->odd from here took 3 us of 145.)
        rs[k] = fmaxf(nref, -INFINITY);
        odd = max(odd, __float_as_uint(nref) & 0x7FFFFFFFu);
        asm volatile("bar.sync %0, 128;" ::"r"(1 + grp) : "memory");
        nref = fetch(t + 2);
        const int row0 = t * tile_rows;
        const bool edge = un.key0 + kKeys - 1 > past + row0 / G || row0 + tile_rows > all || tile_rows < kTileRows;
        // columns that see the key
        const int lo = static_cast<int>(min(max(static_cast<long long>(key - past) * G - row0, 0LL), 256LL));
        const int hi_ = min(tile_rows, all - row0);
        w.warp(kSFull + buf, (at / kBufs) & 1, kStatusTimeout);
        tc_fence_after();
        uint32_t x[4][32];
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_ld_32x32b_x32(my_tmem + buf * kTileRows + q * 32, x[q]);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(w.bar(kSFree + buf));
        if (__builtin_expect(edge, 0)) {
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (q * 32 + e < lo || q * 32 + e >= hi_) x[q][e] = 0xFF800000u;       // -inf
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 r4 = *reinterpret_cast<const float4*>(&rs[q * 32 + e]);
            float2 v = fma_pair(make_float2(__uint_as_float(x[q][e]), __uint_as_float(x[q][e + 1])), qs2,
                                make_float2(r4.x, r4.y));
            float2 z = fma_pair(make_float2(__uint_as_float(x[q][e + 2]), __uint_as_float(x[q][e + 3])), qs2,
                                make_float2(r4.z, r4.w));
            v.x = ex2(v.x);
            v.y = ex2(v.y);
            z.x = ex2(z.x);
            z.y = ex2(z.y);
            acc[0] = add_pair(acc[0], v);
            acc[1] = add_pair(acc[1], z);
          }
      }
      j += un.t1 - un.t0;
      acc[0] = add_pair(acc[0], acc[1]);
      float add = acc[0].x + acc[0].y;
      if (odd > 0x7F800000u) sm->odd[unit & 1] = unit + 1;
      if (grp == 1) sm->sums[unit & 1][k] = add;
      asm volatile("bar.sync 3, 256;" ::: "memory");
      if (__builtin_expect(sm->odd[unit & 1] == unit + 1, 0))      // and the keys that such a row does see
#pragma unroll 1
        for (int r = static_cast<int>(max(static_cast<long long>(key - past) * G, 0LL)); r < all; ++r) {
          const float ref = __ldcg(refs + r);
          if (ref != ref) add = ref;
        }
      if (W != nullptr && w.ok) *W = p.decay * old + (add + sm->sums[unit & 1][k]);
      ++unit;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, 512);
}

}  // namespace sum

template <int kDh>
cudaError_t launch(const WeightsLaunch& a, const DeviceInfo& dev, cudaStream_t stream, std::string* msg) {
  const int G = a.Hq / a.layer.Hkv, page_size = 1 << a.layer.page_shift;
  CUtensorMap q, k;
  const cuuint64_t slabs = static_cast<cuuint64_t>(a.layer.num_pages) * a.layer.Hkv;
  if (!encode_tiles(&q, a.q, kDh, a.Hq, a.batch.n_tokens, kDh * 2, static_cast<cuuint64_t>(a.q_stride) * 2, G,
                    kTileRows / G) ||
      !encode_tiles(&k, a.layer.K, kDh, page_size, slabs, kDh * 2, static_cast<cuuint64_t>(page_size) * kDh * 2,
                    page_size < kKeys ? page_size : kKeys, 1)) {
    *msg = "(the tensor maps of q and the pool cannot be encoded)";
    return cudaErrorInvalidValue;
  }
  WeightsParams p;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.q_stride = a.q_stride;
  p.W = a.weights;
  p.decay = a.decay;
  p.qscale = a.scale * 1.4426950408889634f;
  const WeightsPlaces at = weights_places(a);
  p.counters = at.counters;
  p.ref = at.ref;
  p.part = at.part;
  p.scores = at.scores;
  WeightsSplit split = weights_split(a.batch.B, a.batch.width, a.layer.page_shift, a.layer.num_pages, a.layer.Hkv, G, a.max_new);
  p.rule = score_rule(split, at);
  if (split.many && !p.rule.kept && !p.rule.ask) split.few_rows = 0;      // (no room at all)
  p.status = dev.status_word;
  p.batch = a.batch;
  p.num_pages = a.layer.num_pages;
  p.Hkv = a.layer.Hkv;
  p.page_shift = a.layer.page_shift;
  p.shape.G = G;
  p.shape.chunk_shift = kChunkShift;
  p.shape.coarse = false;
  p.shape.cap = a.batch.width << a.layer.page_shift;
  WeightsParams few = p;
  few.shape.rows = few::kRows;
  few.shape.min_rows = 0;
  few.shape.max_rows = split.few_rows;      // (the room for scores holds no more)
  few.shape.alone = !split.many;
  p.shape.rows = many::kTiles * (kTileRows / G * G);
  p.shape.min_rows = split.few_rows + 1;
  p.shape.max_rows = 0x7FFFFFFF;
  WeightsParams sums = p;
  if (!p.rule.kept && !p.rule.ask) sums.shape.min_rows = 0;      // without their scores, the few rows' weights too
  if (!split.many) sums.shape.max_rows = split.few_rows;
  static SmemOnce once[4];
  cudaError_t e = allow_smem(few::weights_few_kernel<kDh>, kSmemBytes, dev.device, &once[0]);
  if (e == cudaSuccess) e = allow_smem(many::weights_ref_kernel<kDh>, kSmemBytes, dev.device, &once[1]);
  if (e == cudaSuccess) e = allow_smem(sum::weights_sum_kernel<kDh, false>, kSmemBytes, dev.device, &once[2]);
  if (e == cudaSuccess) e = allow_smem(sum::weights_sum_kernel<kDh, true>, kSmemBytes, dev.device, &once[3]);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int grid = dev.num_sms < kWeightsMaxBlocks ? dev.num_sms : kWeightsMaxBlocks;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto launched = [&](cudaError_t r) {
    if (r == cudaSuccess) count_launches(1);
    e = r;
    return r == cudaSuccess;
  };
  if (split.few_rows > 0) {
    cfg.blockDim = dim3(few::kThreads);
    if (!launched(cudaLaunchKernelEx(&cfg, few::weights_few_kernel<kDh>, k, few))) return e;
  }
  if (split.many) {
    cfg.blockDim = dim3(many::kThreads);
    if (!launched(cudaLaunchKernelEx(&cfg, many::weights_ref_kernel<kDh>, q, k, p))) return e;
  }
  if (split.many || !p.rule.kept) {
    cfg.blockDim = dim3(sum::kThreads);
    if (!launched(p.rule.ask ? cudaLaunchKernelEx(&cfg, sum::weights_sum_kernel<kDh, true>, q, k, sums)
                             : cudaLaunchKernelEx(&cfg, sum::weights_sum_kernel<kDh, false>, q, k, sums)))
      return e;
  }
  if (split.few_rows > 0 && (p.rule.kept || p.rule.ask)) {
    WeightsAdd add = {p.rule, p.batch, few.shape, p.num_pages, p.Hkv, p.page_shift, p.scores, p.ref, p.W, p.decay};
    e = launch_weights_add(add, dev, stream);
  }
  return e;
}

}  // namespace

cudaError_t launch_weights_tile(const WeightsLaunch& a, const DeviceInfo& dev, cudaStream_t stream, std::string* msg) {
  return a.dh == 64 ? launch<64>(a, dev, stream, msg) : launch<128>(a, dev, stream, msg);
}

}  // namespace cxa
