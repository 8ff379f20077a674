// Attention of new tokens over a paged bf16 K/V cache, for sequences with many query rows
// a K/V head (prompts and chunks of them): tcgen05 products over 128-row tiles.
//
//   S = Q K^T (128 rows x a chunk of keys), P = 2^(scale log2(e) S - m), O += P V
//
// A work item is a pair of 128-row tiles (a tile: 128 / G tokens times the G query heads of
// one K/V head), dealt out by paged_work.cuh in chunks of 16 KB of K and of V (128 keys of
// 64 channels, 64 keys of 128). One block runs on an SM and works on both tiles of its item,
// which share each K and V tile read (a block a tile, two blocks an SM, read twice as much:
// 418 us against 401 us, where the change was made, for 2048 tokens over 32768 keys of 20
// heads, its K and V coming 11 times from DRAM); one tile's products run under the other's
// exponentials:
//
//  * warp 18 streams by TMA: the item's Q (a box of 128 / G tokens x G heads a tile, which
//    lands token by token, the row order of a tile), and K and V page by page into rings of
//    five tiles each; the boxes of a chunk are issued by a lane each. A K tile comes back as
//    soon as both tiles' scores are done, a V tile after both P.V.
//  * warps 16 and 17 issue the products of a tile each: scores of chunk i + 1 once the
//    softmax warps have read those of chunk i, then P.V of chunk i. P is read from tensor
//    memory, V as it lies in shared memory (rows of keys: an MN-major operand).
//  * warps 0..7 and 8..15 do the softmax of a tile each, two threads a row: a warp has 32 rows
//    and one half of a chunk's keys, its partner the other half (one thread a row: 352 us
//    against 345, the mixed batch below 197 against 180). They take their scores into
//    registers at once, which lets the next chunk's scores start while the exponentials run.
//    A row's reference m moves, and O is rescaled, only when a score passes it by more than
//    2^8 (decided for the sequence's rows among the 32 of two partners together, so that the
//    common chunk costs them one barrier and no exchange); the sums of the halves meet at an
//    item's end.
//
// A tile whose last token sees fewer keys than its neighbour's leaves the item's last chunks
// out (its softmax warps then hand the K and V tiles back).
//
// Measured: 2048 tokens over 32768 keys of 20 heads of 64 channels 319 us, 1040 TFLOP/s, with
// 128 channels 505 to 520 us, 1290 to 1320 TFLOP/s. Bound by the chain of a tile's steps, some 2250 clocks a
// chunk of 128 keys for the two tiles: scores, read, exponentials (1024 clocks of the SM's
// units for the two tiles), conversion, P.V (the products of both: 1045 clocks), each handing
// over through a barrier (some 250 clocks there and back). Tensor pipe 43 %, exponentials
// 45 %, issue 62 % busy. A barrier order that sends the tiles in turns, and a start of one half
// a chunk behind the other, gained nothing. Tensor memory: S, P and O side by side in 256
// columns a tile.
//
// P is rounded to one bf16 value (an error of up to 2^-8 of each weight, of either sign, as
// the bf16 output has itself: 2.3e-3 of a result in all, against 1.7e-3 with exact weights);
// sums, references and O are fp32, the sums of the values before rounding.
//
// Keys behind an item's last visible one weigh 0 and their V rows, which may hold anything,
// are zeroed in shared memory before P.V, as are those of a page outside the pool, which the
// copy warp leaves out. Keys that some rows see and others do not weigh
// 0 in the others; if one of them has a V that is not finite (0 * inf), those keys are
// added row by row on the CUDA cores instead. Both tiles' softmax warps meet in such chunks.
#include <cuda.h>
#include <cuda_bf16.h>

#include <cmath>

#include "paged.cuh"
#include "paged_work.cuh"
#include "ptx.cuh"
#include "tc_util.cuh"

namespace cxa {
namespace {

constexpr int kTiles = 2;                    // of an item
constexpr int kSoftWarps = 8;                // a tile: two to 32 rows, each with half of a chunk's keys
constexpr int kMmaWarp = kTiles * kSoftWarps, kTmaWarp = kMmaWarp + kTiles;
constexpr int kThreads = (kTmaWarp + 1) * 32;
constexpr int kTileRows = 128;
constexpr int kTileBytes = 16384;            // K or V of a chunk
constexpr int kStages = 5;                   // of K and of V
constexpr int kQBytes = 65536;               // the Q tiles of two items of 64 channels, of one of 128
constexpr int kMaxBlocks = kTileMaxBlocks;
constexpr uint32_t kTmemTile = 256;          // columns of a tile
constexpr float kMoveLog2 = 8.f;
constexpr int kGroup = 8;                    // parts of an item that are merged at once, and then of those

// Barriers; the last four one a tile.
enum Bars {
  kQFull = 0,
  kQEmpty = kQFull + 2,
  kKFull = kQEmpty + 2,
  kKEmpty = kKFull + kStages,
  kVFull = kKEmpty + kStages,
  kVEmpty = kVFull + kStages,
  kSFull = kVEmpty + kStages,
  kSFree = kSFull + kTiles,
  kPFull = kSFree + kTiles,
  kPvDone = kPFull + kTiles,
  kBars = kPvDone + kTiles
};
static_assert(kSFull <= 32, "a bit mask holds the barriers that copies complete");
struct Small {
  uint64_t bars[kBars];
  WorkScratch work;
  WorkCursor at[kTiles * kSoftWarps];   // the softmax warps' items: registers hold scores
  uint32_t bad[8];          // boxes of chunk i whose page is outside the pool, at i % 8
  volatile int abort;
  int tmem;
  int last[kTiles];
  volatile int acc[kTiles]; // the segment's first P.V adds to O
  float swap[kTiles][kTileRows];   // between the two threads of a row
};

constexpr int kSmemBytes = kQBytes + 2 * kStages * kTileBytes + 3072;
static_assert(sizeof(Small) <= 3072, "the small arrays fit behind the tiles");

template <int kDh>
struct Tile {
  static constexpr int chunk = 8192 / kDh;        // keys
  static constexpr int chunk_shift = kDh == 64 ? 7 : 6;
  static constexpr int halves = kDh / 64;         // 128-byte columns of a row
  static constexpr int q_bufs = 128 / kDh;
  static constexpr int half_bytes = chunk * 128;  // of K or V
  static constexpr uint32_t p_col = chunk;        // tensor memory: S, P, O
  static constexpr uint32_t o_col = 256 - kDh;
};

struct TileParams {
  void* out;
  long long o_stride;
  float qscale;
  unsigned int* counters;    // [grid][kTiles][3]
  float* part;               // [2 * grid][kTiles][kDh + 2][128]
  unsigned int* status;
  PagedBatch batch;
  int num_pages, Hkv, page_shift;
  WorkShape shape;
};

// The softmax warps of a tile, of both, and the two of 32 rows.
__device__ __forceinline__ void tile_sync(int tile) {
  asm volatile("bar.sync %0, 256;" ::"r"(1 + tile) : "memory");
}
__device__ __forceinline__ void item_sync() { asm volatile("bar.sync 3, 512;" ::: "memory"); }
__device__ __forceinline__ bool item_or(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 3, 512, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v))
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void pair_sync(int pair) { asm volatile("bar.sync %0, 64;" ::"r"(4 + pair) : "memory"); }
__device__ __forceinline__ bool pair_or(int pair, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "r"(4 + pair)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// a * b + c and a + b on pairs.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
__device__ __forceinline__ uint32_t tmem_ld_1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
  return r;
}
__device__ __forceinline__ void tmem_st_1(uint32_t taddr, uint32_t r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(r) : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]: one thread issues.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Zeroes `bytes` of shared memory from each address that a lane gives (0: none), by the warp, for
// the products that read it next. (Rare, and apart: in line it moves the other warps' registers
// about, 2048 tokens over 32768 keys of 20 heads on 4 331 us against 329.)
__device__ __noinline__ void zero_rows(uint32_t to, int bytes, int lane) {
  for (uint32_t m = __ballot_sync(0xffffffffu, to != 0u); m != 0; m &= m - 1) {
    const uint32_t at = __shfl_sync(0xffffffffu, to, __ffs(m) - 1);
    for (int o = lane * 16; o < bytes; o += 512) st_shared_v4(at + o, 0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  __syncwarp();
}

template <int kDh>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tile_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TileParams p) {
  using T = Tile<kDh>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  const uint32_t q_base = base, k_base = base + kQBytes, v_base = k_base + kStages * kTileBytes;
  Small* sm = reinterpret_cast<Small*>(smem + kQBytes + 2 * kStages * kTileBytes);
  auto bar = [&](int i) { return smem_u32(&sm->bars[i]); };
  // tile t of Q buffer qb
  auto q_tile = [&](int qb, int t) {
    return q_base + static_cast<uint32_t>((qb * kTiles + t) * (kTileRows * kDh * 2));
  };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedBatch& bt = p.batch;
  const int G = p.shape.G, tile_rows = p.shape.rows / kTiles;
  // rows, keys and chunks of tile t of an item
  auto rows_of = [&](const WorkCursor& w, int t) {
    return max(0, min(tile_rows, work_rows(w.seq, p.shape) - w.rt * p.shape.rows - t * tile_rows));
  };
  auto chunks_of = [&](const WorkCursor& w, int t) {
    if (rows_of(w, t) == 0) return 0;
    const int last = min(w.seq.n - 1, (w.rt * p.shape.rows + (t + 1) * tile_rows - 1) / G);
    return max(1, (visible_keys(w.seq, last, p.shape.cap) + T::chunk - 1) >> T::chunk_shift);
  };

  // Launched early behind paged_rows_kernel of the same call, and nothing of another call
  // between the two (cxa_paged_attention sees to it). Every thread of that grid waits for all
  // grids before it, and for what they wrote to be performed, before it lets this one start. So
  // the batch, Q, the pool and the scratch lie in memory as those grids left them when this
  // one's first block starts, and what it reads before its own wait, at its end, is of theirs
  // alone: the few-rows grid writes other rows and other scratch. What is left to do here is to
  // drop what this SM's L1 may hold from before (the fence below) and, for the copies, which
  // read past the generic proxy, to order them behind it (the proxy fence of the copy warp).
  // With a wait here instead the mixed batch takes 188 us against 178: its blocks start as the
  // few-rows grid's leave, which they do over some 10 us.
  __threadfence();
  WorkRange range;
  WorkCursor cur;
  WorkShape shape = p.shape;
  const bool active = work_locate<kThreads, false>(bt, shape, p.Hkv, &sm->work, &range, &cur);
  if (active) {
    if (tid == 0) {
      for (int i = 0; i < kBars; ++i) {
        const bool by_tiles = (i >= kQEmpty && i < kKFull) || (i >= kKEmpty && i < kVFull) || (i >= kVEmpty && i < kSFull);
        mbar_init(bar(i), by_tiles ? kTiles : i >= kSFree && i < kPvDone ? kSoftWarps : 1);
      }
      fence_mbar_init();
      sm->abort = 0;
    }
    if (tid < 8) sm->bad[tid] = 0;
    if (warp == kTmaWarp && lane == 0) {
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
    }
    if (warp == kMmaWarp) {
      tmem_alloc(smem_u32(&sm->tmem), kTiles * kTmemTile);
      tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = static_cast<uint32_t>(sm->tmem);
    // A wait that runs out, or that another warp's has cut short, leaves ok false: the copy
    // and product warps then stop; the softmax warps go on through their loop, barriers
    // included, without waiting for anything or writing results.
    bool ok = true;
    auto wait = [&](int i, uint32_t parity) {      // by one thread
      // (the code after the first attempt is short: it stands in the softmax warps' loop)
      uint64_t t0 = 0;
      while (ok && __builtin_expect(!mbar_try_wait_1ms(bar(i), parity), 0)) {
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        if (sm->abort != 0 || now - t0 > kWaitLimitNs) {
          ok = false;
          sm->abort = 1;
          atomicOr(p.status, kStatusTimeout);
        }
      }
      return ok;
    };
    auto wait_warp = [&](int i, uint32_t parity) { // by a whole warp, with one answer
      if (__all_sync(0xffffffffu, mbar_test_wait(bar(i), parity))) return ok;   // far quicker, if it is so
      wait(i, parity);
      ok = __all_sync(0xffffffffu, ok);
      return ok;
    };
    auto wait_both = [&](int i, uint32_t pi, int k, uint32_t pk) {   // for two barriers, as wait_warp
      if (__all_sync(0xffffffffu, mbar_test_wait(bar(i), pi) && mbar_test_wait(bar(k), pk))) return ok;
      wait(i, pi);
      wait(k, pk);
      ok = __all_sync(0xffffffffu, ok);
      return ok;
    };
    const int n_chunks = range.g1 - range.g0;

    if (warp == kTmaWarp) {
      // ---------------------------------------------------------------- copies
      fence_proxy_async_global();
      const int ps_shift = min(p.page_shift, T::chunk_shift);
      const int box_rows = 1 << ps_shift;                // keys a box
      const int box = lane / T::halves, half = lane % T::halves;
      const bool mine = box < (T::chunk >> ps_shift);
      int c = cur.c, item = 0;
      bool fresh = true;
      uint32_t armed = 0, parity = 0;                    // barriers copies were sent to, and the phase
      auto sent = [&](int b, int round) {
        armed |= 1u << b;
        parity = (parity & ~(1u << b)) | (static_cast<uint32_t>(round & 1) << b);
      };
      for (int i = 0; i < n_chunks; ++i) {
        if (fresh) {
          const int qb = item % T::q_bufs;
          if (!wait_warp(kQEmpty + qb, ((item / T::q_bufs) & 1) ^ 1)) break;
          const int tiles = rows_of(cur, 1) > 0 ? 2 : 1;
          if (lane == 0)
            mbar_arrive_expect_tx(bar(kQFull + qb), static_cast<uint32_t>(tiles * T::halves * tile_rows * 128));
          __syncwarp();
          if (lane < tiles * T::halves)
            tma_load_3d(q_tile(qb, lane / T::halves) + (lane % T::halves) * (kTileRows * 128), &tmQ, bar(kQFull + qb),
                        (lane % T::halves) * 64, cur.h * G,
                        cur.seq.q0 + (cur.rt * kTiles + lane / T::halves) * (tile_rows / G));
          sent(kQFull + qb, item / T::q_bufs);
          fresh = false;
        }
        const int key0 = c << T::chunk_shift;
        const int need = min(T::chunk, tile_keys(cur.seq, p.shape, cur.rt) - key0);   // keys of the chunk
        const int at = key0 + box * box_rows;
        const bool want = mine && box * box_rows < need;
        int page = 0;
        if (want)
          page = paged_lookup(bt.table + static_cast<size_t>(cur.b) * bt.width, bt.width, p.page_shift, p.num_pages, at);
        const bool load = want && page >= 0;
        const uint32_t bad = __ballot_sync(0xffffffffu, want && page < 0);
        const uint32_t bytes = static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, load)) * box_rows * 128);
        const int x = half * 64, y = at & ((1 << p.page_shift) - 1), z = page * p.Hkv + cur.h;
        const uint32_t dst = static_cast<uint32_t>(half * T::half_bytes + box * box_rows * 128);
        const int st = i % kStages, round = i / kStages;
        if (!wait_warp(kKEmpty + st, (round & 1) ^ 1)) break;
        if (lane == 0) {
          uint32_t boxes = 0;    // a bit a box, whose scores are left out
          for (uint32_t m = bad; m != 0; m &= m - 1) boxes |= 1u << ((__ffs(m) - 1) / T::halves);
          sm->bad[i & 7] = boxes;
          if (bad != 0) atomicOr(p.status, kStatusBadPage);
          mbar_arrive_expect_tx(bar(kKFull + st), bytes);
        }
        __syncwarp();
        if (load) tma_load_3d(k_base + st * kTileBytes + dst, &tmK, bar(kKFull + st), x, y, z);
        sent(kKFull + st, round);
        if (!wait_warp(kVEmpty + st, (round & 1) ^ 1)) break;
        if (bad != 0)            // no copy fills the V rows of a bad page, and 0 * inf is not 0
          zero_rows(want && page < 0 ? v_base + st * kTileBytes + dst : 0u, box_rows * 128, lane);
        if (lane == 0) mbar_arrive_expect_tx(bar(kVFull + st), bytes);
        __syncwarp();
        if (load) tma_load_3d(v_base + st * kTileBytes + dst, &tmV, bar(kVFull + st), x, y, z);
        sent(kVFull + st, round);
        if (++c == cur.nc && i + 1 < n_chunks) {
          work_next(bt, p.shape, p.Hkv, &cur);
          c = 0;
          ++item;
          fresh = true;
        }
      }
      if (!ok)      // the copies under way land before the block ends
        for (int b = 0; b < kSFull; ++b)
          if (armed & (1u << b)) mbar_wait(bar(b), (parity >> b) & 1u);
    } else if (warp >= kMmaWarp) {
      // ---------------------------------------------------------------- products of a tile
      // The whole warp walks the chunks, with one lane issuing, and the operands' addresses are
      // known to be the same in every lane: a product of 32 or 64 clocks leaves no time to
      // carry them over from a lane's registers one by one.
      constexpr uint32_t idesc_s = make_idesc(1u, kTileRows, T::chunk);
      constexpr uint32_t idesc_o = make_idesc(1u, kTileRows, 64) | (1u << 16);   // V MN-major
      const int t = __shfl_sync(0xffffffffu, warp, 0) - kMmaWarp;
      const uint32_t my = __shfl_sync(0xffffffffu, tmem + t * kTmemTile, 0);
      constexpr uint64_t k_hi = desc_high(1024), mn_hi = desc_high(1024);
      // the scores' cursor: chunk i of the range, chunk c of the item, j of the tile's own
      int i = -1, c = cur.c - 1, item = 0, j = 0, nc = chunks_of(cur, t);
      bool fresh = true;      // the item's Q has not been waited for
      // To the tile's next chunk; false at the end of the range.
      auto next = [&]() {
        for (;;) {
          if (++i == n_chunks) return false;
          if (++c == cur.nc) {
            // a Q that this tile has no (more) scores of goes back at once, or behind them
            if (fresh) {
              if (!wait_warp(kQFull + item % T::q_bufs, (item / T::q_bufs) & 1)) return false;
              if (lane == 0) mbar_arrive(bar(kQEmpty + item % T::q_bufs));
            } else if (elect_one()) {
              tc_commit(bar(kQEmpty + item % T::q_bufs));
            }
            __syncwarp();
            work_next(bt, p.shape, p.Hkv, &cur);
            c = 0;
            ++item;
            fresh = true;
            nc = chunks_of(cur, t);
          }
          if (c < nc) return true;
        }
      };
      auto scores = [&]() {
        const int qb = item % T::q_bufs, st = i % kStages;
        if (fresh && !wait_warp(kQFull + qb, (item / T::q_bufs) & 1)) return;
        fresh = false;
        // (a barrier that nothing has completed yet passes for the phase before its first)
        if (!wait_both(kKFull + st, (i / kStages) & 1, kSFree + t, (j & 1) ^ 1)) return;
        tc_fence_after();
        const int at = __shfl_sync(0xffffffffu, st | qb << 8, 0), k_at = at & 255;
        const uint32_t ql = desc_low(q_tile(at >> 8, t), 16), kl = desc_low(k_base + k_at * kTileBytes, 16);
        const uint32_t k_empty = bar(kKEmpty + k_at);
        if (elect_one()) {
#pragma unroll
          for (int h = 0; h < T::halves; ++h)
#pragma unroll
            for (int k = 0; k < 4; ++k)      // 16 channels: 32 bytes
              mma_bf16(my, k_hi | (ql + (h * (kTileRows * 128) >> 4) + 2 * k),
                       k_hi | (kl + (h * T::half_bytes >> 4) + 2 * k), idesc_s, h + k != 0 ? 1u : 0u);
          tc_commit(bar(kSFull + t));
          tc_commit(k_empty);
        }
        __syncwarp();
        ++j;
      };
      bool more = next(), starts = true;
      if (more) scores();
      for (int pj = 0; more && ok; ++pj) {     // P.V of the tile's chunk pj
        const int st = i % kStages, round = i / kStages;
        // The next scores go first, so that the softmax warps find them; but not those of
        // another item, whose copies may wait for this P.V.
        const bool same = c + 1 < nc && i + 1 < n_chunks;
        if (same) {
          ++i;
          ++c;
          scores();
        }
        if (!ok || !wait_both(kVFull + st, round & 1, kPFull + t, pj & 1)) break;
        tc_fence_after();
        const uint32_t acc0 = !starts || sm->acc[t] != 0 ? 1u : 0u;
        const uint32_t at = __shfl_sync(0xffffffffu, st | acc0 << 8, 0), acc = at >> 8;
        const uint32_t vl = desc_low(v_base + (at & 255) * kTileBytes, 1024), v_empty = bar(kVEmpty + (at & 255));
        if (elect_one()) {
#pragma unroll
          for (int kb = 0; kb < T::chunk / 16; ++kb)     // 16 keys: 2048 bytes
#pragma unroll
            for (int h = 0; h < T::halves; ++h)
              mma_bf16_ts(my + T::o_col + h * 64, my + T::p_col + kb * 8,
                          mn_hi | (vl + ((h * T::half_bytes + kb * 2048) >> 4)), idesc_o, kb != 0 ? 1u : acc);
          tc_commit(bar(kPvDone + t));
          tc_commit(v_empty);
        }
        __syncwarp();
        starts = !same;
        if (!same) {
          more = next();
          if (more) scores();
        }
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------------- softmax, two threads a row
      const int t = warp / kSoftWarps, hf = (warp >> 2) & 1, r = (warp & 3) * 32 + lane, pair = t * 4 + (warp & 3);
      const uint32_t my_tmem = tmem + t * kTmemTile + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      constexpr int XC = T::chunk / 2, OC = kDh / 2;      // this thread's columns of S and of O
      const uint32_t my_s = my_tmem + hf * XC, my_p = my_tmem + T::p_col + hf * (XC / 2), my_o = my_tmem + T::o_col + hf * OC;
      const int box_shift = min(p.page_shift, T::chunk_shift);
      const float2 qs2 = make_float2(p.qscale, p.qscale);
      WorkCursor& at = sm->at[warp];
      if (lane == 0) at = cur;
      __syncwarp();
      int c = cur.c, c0 = cur.c, nc = 0, j = 0;       // j: chunks of this tile so far
      float m = -INFINITY, l = 0.f;
      bool fresh = true;
      constexpr int XB = XC / 32;
      // The row's scores, all in registers, so that the next chunk's products can start.
      auto load_scores = [&](uint32_t (&x)[XB][32]) {
#pragma unroll
        for (int b = 0; b < XB; ++b) tmem_ld_32x32b_x32(my_s + 32 * b, x[b]);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kSFree + t));
      };
      // Scores -> probabilities, which go to tensor memory; m, l and O follow.
      auto softmax = [&](uint32_t (&x)[XB][32]) {
        float mx[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) mx[q] = -INFINITY;
#pragma unroll
        for (int b = 0; b < XB; ++b)
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            mx[(e / 2) & 3] = max3(mx[(e / 2) & 3], __uint_as_float(x[b][e]), __uint_as_float(x[b][e + 1]));
        float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.qscale;
        const bool pv = j == 0 || mbar_test_wait(bar(kPvDone + t), (j - 1) & 1);
        // the references of 32 rows move together, to the largest score so far
        float corr = 1.f;
        const bool moved = pair_or(pair, top > m + kMoveLog2);
        if (__builtin_expect(moved, 0)) {
          if (hf == 1) sm->swap[t][r] = top;
          pair_sync(pair);
          if (hf == 0) {
            top = fmaxf(top, sm->swap[t][r]);
            sm->swap[t][r] = top;
          }
          pair_sync(pair);
          top = sm->swap[t][r];
          const float to = fmaxf(m, top);
          corr = m == -INFINITY ? 0.f : ex2(m - to);
          m = to;
          l *= corr;
        }
        const float ref = m == -INFINITY ? 0.f : -m;
        const float2 ref2 = make_float2(ref, ref);
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
        for (int b = 0; b < XB; ++b)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float2 v = make_float2(__uint_as_float(x[b][2 * e]), __uint_as_float(x[b][2 * e + 1]));
            v = fma2(v, qs2, ref2);
            v.x = ex2(v.x);
            v.y = ex2(v.y);
            x[b][2 * e] = __float_as_uint(v.x);
            x[b][2 * e + 1] = __float_as_uint(v.y);
          }
        // (apart: in one loop each sum and conversion stands behind its own exponential)
#pragma unroll
        for (int b = 0; b < XB; ++b)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float2 v = make_float2(__uint_as_float(x[b][2 * e]), __uint_as_float(x[b][2 * e + 1]));
            sum[e & 1] = add2(sum[e & 1], v);
            x[0][16 * b + e] = pack_bf16(v.x, v.y);     // behind what is still to be read
          }
        sum[0] = add2(sum[0], sum[1]);
        l += sum[0].x + sum[0].y;

        // P's place and O are free once the previous P.V has run
        if (!__all_sync(0xffffffffu, pv)) wait_warp(kPvDone + t, (j - 1) & 1);
        tc_fence_after();
        if (__builtin_expect(moved && c != c0, 0)) {
#pragma unroll 1
          for (int b = 0; b < OC / 16; ++b) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(my_o + 16 * b, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
            tmem_st_32x32b_x16(my_o + 16 * b, o);
          }
        }
        if constexpr (XB == 2) {
          tmem_st_32x32b_x32(my_p, x[0]);
        } else {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = x[0][e];
          tmem_st_32x32b_x16(my_p, w);
        }
        tmem_st_wait();
      };
      auto give_p = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kPFull + t));
      };
      for (int i = 0; i < n_chunks; ++i) {
        if (fresh) {
          fresh = false;
          nc = chunks_of(at, t);
          // A row that is no token's of the sequence (it holds padding, the next sequence's
          // tokens, or what no copy has filled) starts with a reference that no score passes:
          // it has no say in when the references of its 32 rows move.
          m = r < rows_of(at, t) ? -INFINITY : INFINITY;
          l = 0.f;
          c0 = c;
          if (r == 0 && hf == 0) sm->acc[t] = 0;
          __syncwarp();       // (without it 323 us against 319 for 2048 tokens over 32768 keys)
        }
        // The chunks that every row of the item sees, but for the tile's last, in a loop of
        // their own: the code between two of them is fetched anew for each by every warp.
        const int plain =
            min(min(visible_keys(at.seq, at.rt * p.shape.rows / G, p.shape.cap) >> T::chunk_shift, nc - 1) - c,
                n_chunks - 1 - i);
        for (int e = i + plain; i < e; ++i) {
          wait_warp(kSFull + t, j & 1);
          tc_fence_after();
          const uint32_t bad = *const_cast<volatile uint32_t*>(&sm->bad[i & 7]);
          uint32_t x[XB][32];        // (load_scores, with the look at `bad` under its latency)
#pragma unroll
          for (int b = 0; b < XB; ++b) tmem_ld_32x32b_x32(my_s + 32 * b, x[b]);
          tmem_ld_wait();
          if (__builtin_expect(bad != 0, 0)) break;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(kSFree + t));
          softmax(x);
          give_p();
          ++j;
          ++c;
        }
        const int row0 = at.rt * p.shape.rows + t * tile_rows, rows = rows_of(at, t);
        const int see = r < rows ? visible_keys(at.seq, (row0 + r) / G, p.shape.cap) : 0;
        const int see_all = visible_keys(at.seq, row0 / G, p.shape.cap);                       // all of the tile's rows
        const int see_item = visible_keys(at.seq, at.rt * p.shape.rows / G, p.shape.cap);      // and of the item's
        const int keys = tile_keys(at.seq, p.shape, at.rt);                                    // some of the item's
        const int key0 = c << T::chunk_shift;
        const int st = i % kStages, round = i / kStages;
        const bool here = c < nc;                          // the tile sees some of the chunk
        const bool starts = c == c0, ends = here && (c + 1 == nc || i + 1 == n_chunks);
        const int lim = see - key0;
        if (here) {
          wait_warp(kSFull + t, j & 1);
          tc_fence_after();
        } else {
          wait_warp(kKFull + st, round & 1);
        }
        const uint32_t bad = *const_cast<volatile uint32_t*>(&sm->bad[i & 7]);
        // Some row of the item misses a key. Both tiles' warps meet at barriers then: this goes by
        // positions alone, so that they agree on it also after a wait that ran out, when what
        // they read in shared memory (`bad`) may differ.
        const bool special = key0 + T::chunk > see_item;
        if (!here) {
          tile_sync(t);         // every warp of the tile has seen the chunk come
          if (warp % kSoftWarps == 0 && lane == 0) mbar_arrive(bar(kKEmpty + st));
          __syncwarp();
        }
        if (here) {
          uint32_t x[XB][32];
          load_scores(x);
          if (key0 + T::chunk > see_all || bad != 0) {
#pragma unroll
            for (int b = 0; b < XB; ++b)
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const int k = hf * XC + 32 * b + e;
                if (k >= lim || ((bad >> (k >> box_shift)) & 1u) != 0) x[b][e] = 0xFF800000u;   // -inf
              }
          }
          softmax(x);
        }

        if (special) {
          // keys [lo, hi) of the chunk are seen by some rows of the item and not by others,
          // keys from hi on by none
          const int lo = max(0, see_item - key0), hi = min(T::chunk, keys - key0);
          wait_warp(kVFull + st, round & 1);
          const int key = r & (T::chunk - 1), half = r >> T::chunk_shift;   // this thread's part of V: 64 bytes
          const bool has = T::chunk * T::halves > r;
          const uint32_t vt = v_base + st * kTileBytes;
          const uint32_t vrow = vt + half * T::half_bytes + key * 128 + hf * 64;
          bool wild = false;
          if (has && key >= lo && key < hi)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint4 u = ld_shared_v4(vrow + 16 * q);
              const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) wild |= (w[e] & 0x7F80u) == 0x7F80u || (w[e] & 0x7F800000u) == 0x7F800000u;
            }
          tc_fence_before();     // (the other thread's half of P)
          wild = item_or(wild);
          tc_fence_after();
          if (wild) {
            if (here) {
#pragma unroll 1
              for (int b = 0; b < OC / 32; ++b) {
                const int ch = hf * OC + 32 * b;         // first of 32 channels
                uint32_t o[32];
                tmem_ld_32x32b_x32(my_o + 32 * b, o);
                tmem_ld_wait();
                if (starts)
#pragma unroll
                  for (int e = 0; e < 32; ++e) o[e] = 0u;
#pragma unroll 1
                for (int k = lo; k < hi; ++k) {
                  const uint32_t w = tmem_ld_1(my_tmem + T::p_col + (k >> 1));
                  tmem_ld_wait();
                  // (a bad page's keys, P and V of which are 0 anyway, are passed over: without the
                  // second condition the compiler spills 276 bytes instead of 56)
                  if (k < lim && ((bad >> (k >> box_shift)) & 1u) == 0) {
                    const float pk = __uint_as_float((k & 1) ? w & 0xFFFF0000u : w << 16);
                    const uint32_t vr = vt + (ch / 64) * T::half_bytes + k * 128;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                      const uint4 u = ld_shared_v4(vr + (((ch % 64 / 8 + q) ^ (k & 7)) << 4));
                      const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                      for (int e = 0; e < 4; ++e) {
                        float a0 = __uint_as_float(o[8 * q + 2 * e]), a1 = __uint_as_float(o[8 * q + 2 * e + 1]);
                        a0 = fmaf(pk, __uint_as_float(v[e] << 16), a0);
                        a1 = fmaf(pk, __uint_as_float(v[e] & 0xFFFF0000u), a1);
                        o[8 * q + 2 * e] = __float_as_uint(a0);
                        o[8 * q + 2 * e + 1] = __float_as_uint(a1);
                      }
                    }
                  }
                  __syncwarp();    // the next load is the whole warp's
                }
                tmem_st_32x32b_x32(my_o + 32 * b, o);
                tmem_st_wait();
              }
            }
            tc_fence_before();
            item_sync();      // V and P have been read
            tc_fence_after();
            if (here && hf == 0) {
              for (int k = lo >> 1; 2 * k < hi; ++k) {    // P.V leaves these keys out
                uint32_t w = tmem_ld_1(my_tmem + T::p_col + k);
                tmem_ld_wait();
                w &= 2 * k >= lo ? 0u : 0x0000FFFFu;
                tmem_st_1(my_tmem + T::p_col + k, w);
              }
              tmem_st_wait();
            }
          }
          if (here && starts && wild && r == 0 && hf == 0) sm->acc[t] = 1;
          if (has && key >= (wild ? lo : hi))
#pragma unroll
            for (int q = 0; q < 4; ++q) st_shared_v4(vrow + 16 * q, 0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
        }
        if (here) {
          give_p();
        } else {
          wait_warp(kVFull + st, round & 1);
          tile_sync(t);         // every warp of the tile has left V
          if (warp % kSoftWarps == 0 && lane == 0) mbar_arrive(bar(kVEmpty + st));
          __syncwarp();
        }

        if (ends) {
          // ---- the tile's part in this range: written out, or left for the merge
          wait_warp(kPvDone + t, j & 1);
          tc_fence_after();
          const bool whole = c0 == 0 && c + 1 == nc;
          const int tok = (row0 + r) / G, hd = at.h * G + (row0 + r) % G;
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) +
                               (r < rows ? (at.seq.q0 + tok) * p.o_stride + static_cast<long long>(hd) * kDh : 0);
          constexpr size_t kSlot = static_cast<size_t>(kTileRows) * (kDh + 2);
          float* slot = p.part + ((2 * static_cast<size_t>(blockIdx.x) + (c0 == 0 ? 1 : 0)) * kTiles + t) * kSlot;
          // the two threads of a row add their sums up
          if (hf == 1) sm->swap[t][r] = l;
          pair_sync(pair);
          if (hf == 0) {
            l += sm->swap[t][r];
            sm->swap[t][r] = l;
          }
          pair_sync(pair);
          l = sm->swap[t][r];
          // 32 channels, from hf * OC + 32 * b on
          auto put = [&](int b, const float (&o)[32], float inv) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint4 u;
              u.x = pack_bf16(o[8 * q] * inv, o[8 * q + 1] * inv);
              u.y = pack_bf16(o[8 * q + 2] * inv, o[8 * q + 3] * inv);
              u.z = pack_bf16(o[8 * q + 4] * inv, o[8 * q + 5] * inv);
              u.w = pack_bf16(o[8 * q + 6] * inv, o[8 * q + 7] * inv);
              *reinterpret_cast<uint4*>(dst + hf * OC + 32 * b + 8 * q) = u;
            }
          };
          const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll 1
          for (int b = 0; b < OC / 32; ++b) {
            uint32_t w[32];
            tmem_ld_32x32b_x32(my_o + 32 * b, w);
            tmem_ld_wait();
            if (r < rows && ok) {
              float o[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(w[e]);
              if (whole) {
                put(b, o, inv);
              } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) slot[(hf * OC + 32 * b + e) * kTileRows + r] = o[e];
              }
            }
            __syncwarp();
          }
          tc_fence_before();
          if (!whole) {
            if (r < rows && ok && hf == 0) {
              slot[kDh * kTileRows + r] = m;
              slot[(kDh + 1) * kTileRows + r] = l;
            }
            // merged in groups of kGroup parts first, then the groups, each by its last arriver
            const int owner0 = at.first / range.per;
            const int parts = (at.first + nc - 1) / range.per - owner0 + 1;
            auto part = [&](int k) {
              return p.part + ((2 * static_cast<size_t>(owner0 + k) + (k == 0 ? 1 : 0)) * kTiles + t) * kSlot + r;
            };
            auto last_of = [&](int counter, int n) {
              tile_sync(t);      // what the tile's warps have to show is written
              if (r == 0 && hf == 0) {
                bool last = false;
                if (ok) {
                  unsigned int* const at_counter = p.counters + counter;
                  last = atomic_add_acq_rel_gpu(at_counter, 1u) == static_cast<unsigned int>(n - 1);
                  if (last) *at_counter = 0u;
                }
                sm->last[t] = last;
              }
              tile_sync(t);
              return sm->last[t] != 0;
            };
            // parts first, first + step, ... (n of them) into the result, or into part `first`
            auto merge = [&](int first, int step, int n, bool final) {
              const int m_n = r < rows ? n : 0;
              float M = -INFINITY, L = 0.f;
#pragma unroll 4
              for (int k = 0; k < m_n; ++k) M = fmaxf(M, __ldcg(part(first + k * step) + kDh * kTileRows));
              const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll 4
              for (int k = 0; k < m_n; ++k) {
                const float* src = part(first + k * step) + kDh * kTileRows;
                L += __ldcg(src + kTileRows) * ex2(__ldcg(src) - ref);
              }
              const float linv = L > 0.f || L != L ? 1.f / L : 0.f;
#pragma unroll 1
              for (int b = 0; b < OC / 32; ++b) {
                float o[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0.f;
#pragma unroll 1
                for (int k = 0; k < m_n; ++k) {
                  const float* src = part(first + k * step);
                  const float f = ex2(__ldcg(src + kDh * kTileRows) - ref);
                  float w[32];
#pragma unroll
                  for (int e = 0; e < 32; ++e) w[e] = __ldcg(src + (hf * OC + 32 * b + e) * kTileRows);
#pragma unroll
                  for (int e = 0; e < 32; ++e) o[e] = fmaf(f, w[e], o[e]);
                }
                if (m_n == 0) continue;
                if (final) {
                  put(b, o, linv);
                } else {
                  float* to = const_cast<float*>(part(first));
#pragma unroll
                  for (int e = 0; e < 32; ++e) to[(hf * OC + 32 * b + e) * kTileRows] = o[e];
                }
              }
              if (!final) {
                __syncwarp();
                pair_sync(pair);      // both threads of a row have read the old values
                if (hf == 0 && m_n != 0) {
                  float* to = const_cast<float*>(part(first)) + kDh * kTileRows;
                  to[0] = M;
                  to[kTileRows] = L;
                }
              }
            };
            const int group = (static_cast<int>(blockIdx.x) - owner0) / kGroup, leader = group * kGroup;
            const int groups = (parts + kGroup - 1) / kGroup, n = min(kGroup, parts - leader);
            // a block may lead a group of the item that ends in it and one of the item that begins in it
            const int counter = ((owner0 + leader) * kTiles + t) * 3;
            if (last_of(counter + (group == 0 ? 0 : 1), n)) {
              merge(leader, 1, n, groups == 1);
              if (groups > 1 && last_of((owner0 * kTiles + t) * 3 + 2, groups)) merge(0, kGroup, groups, true);
            }
          }
        }
        if (here) ++j;
        if (++c == at.nc && i + 1 < n_chunks) {
          __syncwarp();
          if (lane == 0) work_next(bt, p.shape, p.Hkv, &at);
          __syncwarp();
          c = 0;
          fresh = true;
        }
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTiles * kTmemTile);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

static_assert(kTileCounters == kMaxBlocks * kTiles * 3, "three counters a tile of a block");

// Query rows of an item: whole tokens in each tile.
int item_rows(int G) { return kTiles * (kTileRows / G * G); }

template <int kDh>
cudaError_t prepare(const PagedAttnLaunch& a, const DeviceInfo& dev, PagedTileMaps* maps, std::string* msg) {
  using T = Tile<kDh>;
  const int G = a.Hq / a.layer.Hkv;
  const int page_size = 1 << a.layer.page_shift;
  const int box_rows = page_size < T::chunk ? page_size : T::chunk;
  const cuuint64_t slabs = static_cast<cuuint64_t>(a.layer.num_pages) * a.layer.Hkv;
  if (!encode_tiles(&maps->q, a.q, kDh, a.Hq, a.batch.n_tokens, kDh * 2, static_cast<cuuint64_t>(a.q_stride) * 2, G,
              kTileRows / G) ||
      !encode_tiles(&maps->k, a.layer.K, kDh, page_size, slabs, kDh * 2, static_cast<cuuint64_t>(page_size) * kDh * 2,
              box_rows, 1) ||
      !encode_tiles(&maps->v, a.layer.V, kDh, page_size, slabs, kDh * 2, static_cast<cuuint64_t>(page_size) * kDh * 2,
              box_rows, 1)) {
    *msg = "the tensor maps of q and the pool cannot be encoded";
    return cudaErrorInvalidValue;
  }
  static SmemOnce once;
  const cudaError_t e = allow_smem(paged_tile_kernel<kDh>, kSmemBytes, dev.device, &once);
  if (e != cudaSuccess) *msg = "shared memory of the tile kernel";
  return e;
}

template <int kDh>
cudaError_t launch(const PagedAttnLaunch& a, const PagedTileMaps& maps, const DeviceInfo& dev, cudaStream_t stream) {
  using T = Tile<kDh>;
  TileParams prm;
  prm.out = a.out;
  prm.o_stride = a.o_stride;
  prm.qscale = a.scale * 1.4426950408889634f;
  prm.counters = static_cast<unsigned int*>(a.workspace) + kRowsCounters;
  prm.part = reinterpret_cast<float*>(static_cast<uint8_t*>(a.workspace) + kPagedCounterBytes +
                                      paged_rows_part_bytes(kDh));
  prm.status = dev.status_word;
  prm.batch = a.batch;
  prm.num_pages = a.layer.num_pages;
  prm.Hkv = a.layer.Hkv;
  prm.page_shift = a.layer.page_shift;
  prm.shape.G = a.Hq / a.layer.Hkv;
  prm.shape.rows = item_rows(prm.shape.G);
  prm.shape.chunk_shift = T::chunk_shift;
  prm.shape.coarse = false;
  prm.shape.cap = a.batch.width << a.layer.page_shift;
  prm.shape.min_rows = kFewRows + 1;
  prm.shape.max_rows = 0x7FFFFFFF;

  cudaLaunchConfig_t cfg = {};
  int grid = dev.num_sms;
  if (grid > kMaxBlocks) grid = kMaxBlocks;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, paged_tile_kernel<kDh>, maps.q, maps.k, maps.v, prm);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace

bool paged_tile_takes(int G, bool act_bf16, int max_new) {
  // A tile holds whole tokens, so G query heads have to fit into it.
  return act_bf16 && G <= kTileRows && static_cast<long long>(max_new) * G > kFewRows;
}

bool paged_tile_countable(const PagedAttnLaunch& a) {
  const int G = a.Hq / a.layer.Hkv;
  return work_bound(a.batch, a.layer.page_shift, a.layer.Hkv, G, item_rows(G),
                    a.dh == 64 ? Tile<64>::chunk_shift : Tile<128>::chunk_shift) < kCountLimit;
}

size_t paged_tile_part_bytes(int dh) {
  return static_cast<size_t>(2 * kMaxBlocks) * kTiles * kTileRows * (dh + 2) * 4;
}

cudaError_t prepare_paged_tile(const PagedAttnLaunch& a, const DeviceInfo& dev, PagedTileMaps* maps, std::string* msg) {
  return a.dh == 64 ? prepare<64>(a, dev, maps, msg) : prepare<128>(a, dev, maps, msg);
}

cudaError_t launch_paged_tile(const PagedAttnLaunch& a, const PagedTileMaps& maps, const DeviceInfo& dev,
                              cudaStream_t stream) {
  return a.dh == 64 ? launch<64>(a, maps, dev, stream) : launch<128>(a, maps, dev, stream);
}

}  // namespace cxa
