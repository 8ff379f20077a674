// Attention over a latent cache's bf16 pages: every key's row [c | r], latent + rope channels, is the key
// of all heads and, in its first `latent` channels, their value. tcgen05 products over steps of 64 keys:
//
//   S^T = [C | R] Q^T  (64 keys x kR query rows),  P = 2^(scale log2(e) S - m),  O^T += C^T P
//
// The rows of a tile are a sequence's new tokens times all heads, 16, 32 or 64 of them: few against the
// 512 channels of a result, so both products are taken transposed. Keys are the rows of the first, channels
// those of the second, and query rows the columns of both: O^T lies in tensor memory as latent / 128 tiles
// of 128 channels by kR columns, where O would not leave room for S. The keys' rows are read by both products
// from the one copy in shared memory, along the channels in the first and across them in the second.
//
//  * warp 6 streams the keys' rows by TMA into two rings: 128 latent channels of 64 keys, 16 KB, a unit, which comes
//    back as soon as P.V has read it, and the rotated part's 8 KB, which the scores alone need. (One ring, where the
//    rotated part took a unit: 84 us for 64 heads over 262,144 keys, 72 so.) It also copies an item's
//    queries, where tokens' rows stand one behind the other (the softmax warps do, otherwise).
//  * warps 4 and 5 issue the products, one the scores, as units come, the other P.V: each waits for what it
//    needs alone (one warp for both, scores first: 112 us for 64 single tokens over 276,698 keys of 20 heads).
//  * warps 0 to 3 do the softmax, 16 keys each; a thread has two keys and a quarter of the rows. A row's
//    reference m moves, and O^T is rescaled, only when a score passes it by more than 2^8 (agreed on by one barrier a
//    step). Sums stay in each thread and meet at an item's end.
//
// Work is dealt out in steps of 64 keys (paged_work.cuh); items that a block boundary cuts are merged
// by latent_merge.cu. Bound by memory: a row of 1152 bytes is read once for the tile's rows. Measured, both
// kernels: 64 single tokens over 276,698 keys of 20 heads, 512 + 64 channels, 72 us (4.5 TB/s: the merge is 5 to 8 of
// them, the start 3, and an item's beginning and end are not covered by copies of the next); one token of 64 heads
// over 262,144 keys 72 us (4.2 TB/s: 64 rows leave rings of two steps, so that copies wait for P.V); one token over
// 448 keys of 256 channels, 8 heads, 12 us, latency.
//
// P is taken as two bf16 values (an error of up to 2^-16 of each weight), so that the output's own rounding is
// the only one that shows: with one, the error of single tokens' outputs was 1.9e-3 to 2.0e-3 in place of 1.7e-3. P.V
// then takes twice the products, which the reading of keys covers: 64 tokens over 276,698 keys 71.3 -> 72.3 us. Sums,
// references and O are fp32.
//
// Rows of keys behind an item's last visible one, and those of a page outside the pool, weigh 0 and are
// zeroed in shared memory before P.V, as they may hold anything. If a key that some rows see and others do
// not has a value that is not finite, its row is zeroed too and the rows that see it become NaN.
#include <cuda.h>
#include <cuda_bf16.h>

#include <cmath>

#include "latent_parts.cuh"
#include "paged_work.cuh"
#include "ptx.cuh"
#include "tc_util.cuh"

namespace cxa {
namespace {

constexpr int kSoftWarps = 4;
constexpr int kSWarp = kSoftWarps, kPvWarp = kSWarp + 1, kTmaWarp = kPvWarp + 1;
constexpr int kThreads = (kTmaWarp + 1) * 32;
constexpr int kKeys = 64, kChunkShift = 6;
constexpr int kUnitBytes = 16384;            // 128 channels of 64 keys
constexpr int kHalf = kUnitBytes / 2;        // 64 channels
constexpr int kMaxUnits = 12, kMaxRopes = 8;
constexpr int kSmemBytes = 232448;
constexpr float kMoveLog2 = 8.f;

enum Bars {
  kQFull = 0,
  kQEmpty = 1,
  kSFull = 2,
  kSFree = 4,
  kPFull = 6,
  kPvDone = 7,
  kUFull = 8,
  kUEmpty = kUFull + kMaxUnits,
  kRFull = kUEmpty + kMaxUnits,
  kREmpty = kRFull + kMaxRopes,
  kBars = kREmpty + kMaxRopes
};

struct Small {
  uint64_t bars[kBars];
  WorkScratch work;
  uint32_t bad[16];            // of step j, at j % 16: groups of 16 keys whose page is outside the pool
  volatile int abort;
  int tmem;
  float top[kSoftWarps][64];
  __align__(16) float corr[64];
  float m[64], inv[64];
  long long row[64];           // where the rows' results begin
};
constexpr int kSmallBytes = 3 << 10;
static_assert(sizeof(Small) <= kSmallBytes, "the small arrays fit behind the ring");

struct TileParams {
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  long long q_stride, o_stride;
  float qscale;
  LatentCut* cut;
  float* part;
  unsigned int* status;
  PagedBatch batch;
  int num_pages, page_shift, latent, rope;
  int units, ropes;            // of the rings: of 128 latent channels, and of the rotated part
  int q_packed;                // queries stand one behind the other: copied by their map
  WorkShape shape;
};

// Tensor memory: two buffers of S^T, then the tiles of O^T.
template <int kR>
struct Tm {
  static constexpr uint32_t o = 2 * kR;
  static constexpr uint32_t cols = kR == 16 ? 128 : kR == 32 ? 256 : 512;
};

__device__ __forceinline__ void soft_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool soft_or(bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v))
      : "memory");
  return r != 0;
}

// 16 lanes x 8 n columns: thread (g, t) has columns 8 i + 2 t, + 1 of lane g in r[4 i], r[4 i + 1] and of
// lane g + 8 in r[4 i + 2], r[4 i + 3].
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t a, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(a));
}
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t a, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(a));
}
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t a, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(a));
}

// Where P of a key's rows lies: one row of 2 kR bytes a key, its 16-byte pieces permuted as the products'
// swizzle of that width has them; and the high half of the products' descriptor.
template <int kR>
__device__ __forceinline__ uint32_t p_piece(int key, int piece) {
  const int x = kR == 64 ? key & 7 : kR == 32 ? key >> 1 & 3 : key >> 2 & 1;
  return static_cast<uint32_t>(key * (2 * kR) + ((piece ^ x) << 4));
}
template <int kR>
constexpr int kPartBytes = kKeys * kR * 2;      // the low part stands behind the high one
template <int kR>
constexpr uint64_t p_desc_high() {
  constexpr uint32_t layout = kR == 64 ? 2u : kR == 32 ? 4u : 6u;      // 128-, 64-, 32-byte swizzle
  return static_cast<uint64_t>((8u * 2 * kR) >> 4 | 1u << 14 | layout << 29) << 32;
}

template <int kR>
__global__ void __launch_bounds__(kThreads, 1)
    latent_tile_kernel(const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmQ,
                       const __grid_constant__ TileParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  const int quads = p.latent / 128, blocks = 2 * quads + (p.rope > 0 ? 1 : 0);      // of 64 channels
  const int NU = p.units, NR = p.ropes;
  const uint32_t u_base = base, r_base = u_base + NU * kUnitBytes, q_base = r_base + NR * kHalf;
  const uint32_t p_base = q_base + blocks * (kR * 128);
  Small* sm = reinterpret_cast<Small*>(smem + kSmemBytes - kSmallBytes);
  auto bar = [&](int i) { return smem_u32(&sm->bars[i]); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedBatch& bt = p.batch;
  const int H = p.shape.G;

  // what needs nothing of the kernels before: under their ends
  if (warp < kSoftWarps) {
    for (int i = tid; i < kBars; i += kSoftWarps * 32)
      mbar_init(bar(i), (i == kQFull && !p.q_packed) || (i >= kSFree && i <= kPFull) ? kSoftWarps : 1);
    fence_mbar_init();
    if (tid == 0) sm->abort = 0;
  } else if (warp == kSWarp) {
    tmem_alloc(smem_u32(&sm->tmem), Tm<kR>::cols);
    tmem_relinquish();
  } else if (warp == kTmaWarp && lane == 0) {
    prefetch_tmap(&tmC);
    prefetch_tmap(&tmQ);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  WorkRange range;
  WorkCursor cur;
  WorkShape shape = p.shape;
  LatentCut cut = {0, 0, 0, 0};
  const bool active = work_locate<kThreads, false, true>(bt, shape, 1, &sm->work, &range, &cur, p.status);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (!active) {
    if (tid == 0) p.cut[blockIdx.x] = cut;
    if (warp == kSWarp) tmem_dealloc(static_cast<uint32_t>(sm->tmem), Tm<kR>::cols);
    return;
  }
  const uint32_t tmem = __shfl_sync(0xffffffffu, static_cast<uint32_t>(sm->tmem), 0);
  // A wait that runs out, or that another warp's has cut short, leaves ok false: the copy and product
  // warps then stop; the softmax warps go on through their loop, barriers included, without waiting for
  // anything or writing results.
  bool ok = true;
  auto wait_warp = [&](int i, uint32_t parity) {      // by a whole warp, with one answer
    if (__all_sync(0xffffffffu, mbar_test_wait(bar(i), parity))) return ok;
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
    ok = __all_sync(0xffffffffu, ok);
    return ok;
  };
  // The steps [s0, s1) of the cursor's item in this block's range, and whether items follow.
  struct Part {
    int s0, s1, keys;
    bool begins, ends, last;
  };
  auto part_of = [&](const WorkCursor& c) {
    Part t;
    const int end = min(range.g1, c.first + c.nc), steps = tile_steps(c.seq, shape, c.rt);
    t.keys = tile_keys(c.seq, shape, c.rt);
    t.s0 = chunk_step(shape, c.c, c.nc, steps);
    t.s1 = chunk_step(shape, end - c.first, c.nc, steps);
    t.begins = c.c == 0;
    t.ends = end == c.first + c.nc;
    t.last = end >= range.g1;
    return t;
  };

  if (warp == kTmaWarp) {
    // ------------------------------------------------------------------ copies
    fence_proxy_async_global();
    const int box_shift = min(p.page_shift, kChunkShift), box_rows = 1 << box_shift;      // keys a box
    const int boxes = kKeys >> box_shift, box = lane % boxes, blk = lane / boxes;
    int pos = 0, r_pos = 0, step = 0, item = 0, q_sent = -1;
    uint32_t round = 0, armed = 0, parity = 0;      // units copies were sent to, and the phase
    uint32_t r_round = 0, r_armed = 0, r_parity = 0;
    for (bool more = true; more && ok; ++item) {
      const Part t = part_of(cur);
      if (p.q_packed) {
        if (!wait_warp(kQEmpty, (item & 1) ^ 1)) break;
        if (lane == 0) mbar_arrive_expect_tx(bar(kQFull), static_cast<uint32_t>(blocks * kR * 128));
        __syncwarp();
        if (lane < blocks)
          tma_load_3d(q_base + lane * (kR * 128), &tmQ, bar(kQFull), lane * 64, cur.seq.q0 * H + cur.rt * kR, 0);
        q_sent = item;
      }
      const int* row = bt.table + static_cast<size_t>(cur.b) * bt.width;
      auto page_of = [&](int s) {
        const int at = s * kKeys + box * box_rows;
        return s < t.s1 && at < t.keys ? paged_lookup(row, bt.width, p.page_shift, p.num_pages, at) : -2;
      };
      // Rows that copies will ask for a step later are fetched into L2, where a step takes half of the ring and
      // more (one token of 64 heads over 262144 rows: 82 us without, 74 a step ahead, 77 two; 20 heads
      // gain nothing).
      constexpr int kAhead = kR == 64 ? 1 : 0;
      int pages[kAhead + 1];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) pages[i + 1] = page_of(t.s0 + i);
      for (int s = t.s0; s < t.s1 && ok; ++s, ++step) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) pages[i] = pages[i + 1];
        pages[kAhead] = page_of(s + kAhead);
        const int page = pages[0], y = (s * kKeys + box * box_rows) & ((1 << p.page_shift) - 1);
        const int y_ahead = ((s + kAhead) * kKeys + box * box_rows) & ((1 << p.page_shift) - 1);
        const uint32_t lows = (1u << boxes) - 1u;                  // a lane a box
        const uint32_t good = __ballot_sync(0xffffffffu, page >= 0) & lows;
        const uint32_t bad = __ballot_sync(0xffffffffu, page == -1) & lows;
        for (int u = 0; u < quads; ++u) {
          if (!wait_warp(kUEmpty + pos, (round & 1) ^ 1)) break;
          if (lane == 0) {
            if (u == 0) {
              uint32_t groups = 0;       // of 16 keys
              for (uint32_t m = bad; m != 0; m &= m - 1)
                groups |= ((1u << (box_rows / 16)) - 1u) << ((__ffs(m) - 1) * (box_rows / 16));
              sm->bad[step & 15] = groups;
              if (bad != 0) atomicOr(p.status, kStatusBadPage);
            }
            mbar_arrive_expect_tx(bar(kUFull + pos), static_cast<uint32_t>(__popc(good) * 2 * box_rows * 128));
          }
          __syncwarp();
          if (blk < 2 && page >= 0)
            tma_load_3d(u_base + pos * kUnitBytes + blk * kHalf + box * box_rows * 128, &tmC, bar(kUFull + pos),
                        u * 128 + blk * 64, y, page);
          if (kAhead > 0 && blk < 2 && pages[kAhead] >= 0) tma_prefetch_3d(&tmC, u * 128 + blk * 64, y_ahead, pages[kAhead]);
          armed |= 1u << pos;
          parity = (parity & ~(1u << pos)) | (round & 1u) << pos;
          if (++pos == NU) {
            pos = 0;
            ++round;
          }
        }
        if (NR > 0 && ok && wait_warp(kREmpty + r_pos, (r_round & 1) ^ 1)) {
          if (lane == 0)
            mbar_arrive_expect_tx(bar(kRFull + r_pos), static_cast<uint32_t>(__popc(good) * box_rows * 128));
          __syncwarp();
          if (blk == 0 && page >= 0)
            tma_load_3d(r_base + r_pos * kHalf + box * box_rows * 128, &tmC, bar(kRFull + r_pos), p.latent, y, page);
          if (kAhead > 0 && blk == 0 && pages[kAhead] >= 0) tma_prefetch_3d(&tmC, p.latent, y_ahead, pages[kAhead]);
          r_armed |= 1u << r_pos;
          r_parity = (r_parity & ~(1u << r_pos)) | (r_round & 1u) << r_pos;
          if (++r_pos == NR) {
            r_pos = 0;
            ++r_round;
          }
        }
      }
      more = !t.last;
      if (more) work_next(bt, shape, 1, &cur);
    }
    if (!ok) {      // the copies under way land before the block ends
      for (int b = 0; b < NU; ++b)
        if (armed & (1u << b)) mbar_wait(bar(kUFull + b), (parity >> b) & 1u);
      for (int b = 0; b < NR; ++b)
        if (r_armed & (1u << b)) mbar_wait(bar(kRFull + b), (r_parity >> b) & 1u);
      if (q_sent >= 0) mbar_wait(bar(kQFull), static_cast<uint32_t>(q_sent) & 1u);
    }
  } else if (warp == kSWarp) {
    // ------------------------------------------------------------------ scores
    // (Addresses that are known to be the same in every lane need no carrying over from one: each product
    // of 32 clocks took 60 to issue otherwise.)
    constexpr uint32_t idesc = make_idesc(1u, kKeys, kR);
    constexpr uint64_t hi = desc_high(1024);
    const uint32_t ub = __shfl_sync(0xffffffffu, u_base, 0), qb = __shfl_sync(0xffffffffu, q_base, 0);
    const uint32_t rb = __shfl_sync(0xffffffffu, r_base, 0);
    int pos = 0, r_pos = 0, item = 0, step = 0;
    uint32_t round = 0, r_round = 0;
    for (bool more = true; more && ok; ++item) {
      const Part t = part_of(cur);
      if (!wait_warp(kQFull, item & 1)) break;
      for (int s = t.s0; s < t.s1 && ok; ++s, ++step) {
        if (!wait_warp(kSFree + (step & 1), ((step >> 1) & 1) ^ 1)) break;
        const uint32_t d = tmem + __shfl_sync(0xffffffffu, step & 1, 0) * kR;
        for (int u = 0; u < quads; ++u) {
          if (!wait_warp(kUFull + pos, round & 1)) break;
          tc_fence_after();
          const int at = __shfl_sync(0xffffffffu, pos, 0), un = __shfl_sync(0xffffffffu, u, 0);
          const uint32_t al = desc_low(ub + at * kUnitBytes, 16), bl = desc_low(qb + un * (2 * kR * 128), 16);
          const uint32_t acc = un != 0 ? 1u : 0u;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k)       // 16 channels: 32 bytes
              mma_bf16(d, hi | (al + 2 * k), hi | (bl + 2 * k), idesc, k != 0 ? 1u : acc);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_bf16(d, hi | (al + (kHalf >> 4) + 2 * k), hi | (bl + (kR * 128 >> 4) + 2 * k), idesc, 1u);
            if (NR == 0 && un + 1 == quads) {
              tc_commit(bar(kSFull + (step & 1)));
              if (s + 1 == t.s1) tc_commit(bar(kQEmpty));
            }
          }
          __syncwarp();
          if (++pos == NU) {
            pos = 0;
            ++round;
          }
        }
        if (NR > 0 && ok && wait_warp(kRFull + r_pos, r_round & 1)) {
          tc_fence_after();
          const int at = __shfl_sync(0xffffffffu, r_pos, 0);
          const uint32_t al = desc_low(rb + at * kHalf, 16), bl = desc_low(qb + quads * (2 * kR * 128), 16);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_bf16(d, hi | (al + 2 * k), hi | (bl + 2 * k), idesc, 1u);
            tc_commit(bar(kREmpty + at));      // P.V has no use for the rotated part
            tc_commit(bar(kSFull + (step & 1)));
            if (s + 1 == t.s1) tc_commit(bar(kQEmpty));
          }
          __syncwarp();
          if (++r_pos == NR) {
            r_pos = 0;
            ++r_round;
          }
        }
      }
      more = !t.last;
      if (more) work_next(bt, shape, 1, &cur);
    }
    __syncwarp();
  } else if (warp == kPvWarp) {
    // ------------------------------------------------------------------ P.V
    constexpr uint32_t idesc = make_idesc(1u, 128, kR) | 1u << 15 | 1u << 16;      // both operands MN-major
    constexpr uint64_t hi = desc_high(1024), p_hi = p_desc_high<kR>();
    const uint32_t ub = __shfl_sync(0xffffffffu, u_base, 0);
    const uint32_t pl = desc_low(__shfl_sync(0xffffffffu, p_base, 0), 1024);
    int pos = 0, step = 0;
    for (bool more = true; more && ok;) {
      const Part t = part_of(cur);
      for (int s = t.s0; s < t.s1 && ok; ++s, ++step) {
        if (!wait_warp(kPFull, step & 1)) break;
        tc_fence_after();
        const uint32_t acc = __shfl_sync(0xffffffffu, s != t.s0 ? 1u : 0u, 0);
        for (int u = 0; u < quads; ++u) {
          int next = pos + u;
          if (next >= NU) next -= NU;
          const int at = __shfl_sync(0xffffffffu, next, 0), un = __shfl_sync(0xffffffffu, u, 0);
          const uint32_t al = desc_low(ub + at * kUnitBytes, kHalf), d = tmem + Tm<kR>::o + un * kR;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 2 * (kKeys / 16); ++k)       // 16 keys: 2048 bytes of the rows, 32 kR of a part of P
              mma_bf16(d, hi | (al + k % (kKeys / 16) * (2048 >> 4)), p_hi | (pl + k * ((32 * kR) >> 4)), idesc,
                       k != 0 ? 1u : acc);
            tc_commit(bar(kUEmpty + at));
            if (un + 1 == quads) tc_commit(bar(kPvDone));
          }
          __syncwarp();
        }
        pos += quads;
        if (pos >= NU) pos -= NU;
      }
      more = !t.last;
      if (more) work_next(bt, shape, 1, &cur);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ softmax
    const int g = lane >> 2, tq = lane & 3;
    constexpr int XN = kR / 2, CN = kR / 4;        // this thread's scores, and its columns
    // column of index i (two to each of its groups of four scores)
    auto col_of = [&](int i) { return 8 * (i >> 1) + 2 * tq + (i & 1); };
    const uint32_t my_tmem = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const int width = p.latent + p.rope;
    int step = 0;
    for (;;) {
      const Part t = part_of(cur);
      const int row0 = cur.rt * kR, rows = min(kR, work_rows(cur.seq, shape) - row0);
      if (!p.q_packed) {
        // the rows' queries (the scores of the item before have been taken): a row a warp
        const int pieces = blocks * 8;
#pragma unroll 2
        for (int r = warp; r < kR; r += kSoftWarps) {
          const int at = row0 + r;
          const __nv_bfloat16* src = p.q + (cur.seq.q0 + at / H) * p.q_stride + static_cast<long long>(at % H) * width;
          uint4 v[3];
#pragma unroll
          for (int j = 0; j < 3; ++j) {
            const int i = lane + 32 * j;
            v[j] = make_uint4(0u, 0u, 0u, 0u);
            if (r < rows && i * 8 < width) v[j] = *reinterpret_cast<const uint4*>(src + i * 8);
          }
#pragma unroll
          for (int j = 0; j < 3; ++j) {
            const int i = lane + 32 * j;
            if (i < pieces)
              st_shared_v4(q_base + (i >> 3) * (kR * 128) + r * 128 + (((i & 7) ^ (r & 7)) << 4), v[j].x, v[j].y, v[j].z, v[j].w);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kQFull));
      }
      if (tid < kR) {
        const int at = row0 + tid;
        sm->row[tid] = (cur.seq.q0 + at / H) * p.o_stride + static_cast<long long>(at % H) * p.latent;
      }
      const int see_all = visible_keys(cur.seq, row0 / H, shape.cap);      // of all of the tile's rows
      float m[CN], l[CN];
#pragma unroll
      for (int i = 0; i < CN; ++i) {
        // columns of no row start with a reference that no score passes
        m[i] = col_of(i) < rows ? -INFINITY : INFINITY;
        l[i] = 0.f;
      }
      for (int s = t.s0; s < t.s1; ++s, ++step) {
        const int key0 = s * kKeys;
        wait_warp(kSFull + (step & 1), (step >> 1) & 1);
        tc_fence_after();
        uint32_t x[XN];
        tmem_ld_16x256b(my_tmem + (step & 1) * kR, x);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kSFree + (step & 1)));
        const uint32_t bad = *const_cast<volatile uint32_t*>(&sm->bad[step & 15]);
        const bool special = key0 + kKeys > see_all;       // some row misses a key
        uint32_t wild = 0;                                 // of this thread's two keys
        if (__builtin_expect(special || bad != 0, 0)) {
          const int k0 = warp * 16 + g;
          const bool gone = (bad >> warp & 1u) != 0, one = (row0 + rows - 1) / H == row0 / H;      // (one token)
          const int lo = max(0, see_all - key0), hi = min(kKeys, t.keys - key0);
          // this warp's 16 keys' rows in shared memory: 8 lanes a row of 64 channels, four rows at a time
          const int sub = lane >> 3;
          auto each_piece = [&](auto body) {
            int at = step * quads % NU, round = step * quads / NU;
            for (int u = 0; u < quads; ++u) {
              wait_warp(kUFull + at, round & 1);      // (it has come: the products have read it)
              const uint32_t to = u_base + at * kUnitBytes + (warp * 16 + sub) * 128 + (lane & 7) * 16;
#pragma unroll
              for (int q = 0; q < 8; ++q) body(q & 3, to + (q >> 2) * kHalf + (q & 3) * 512);
              if (++at == NU) {
                at = 0;
                ++round;
              }
            }
          };
          uint32_t all = 0;        // keys with values that are not finite
          if (lo < hi && !gone) {
            uint32_t w = 0;        // of key 4 i + sub: bit i
            each_piece([&](int i, uint32_t at) {
              const int key = warp * 16 + 4 * i + sub;
              if (key < lo || key >= hi) return;
              const uint4 u = ld_shared_v4(at);
              const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if ((v[e] & 0x7F80u) == 0x7F80u || (v[e] & 0x7F800000u) == 0x7F800000u) w |= 1u << i;
            });
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t eight = __ballot_sync(0xffffffffu, (w >> i & 1u) != 0);      // bits a key
#pragma unroll
              for (int k = 0; k < 4; ++k) all |= (eight >> (8 * k) & 255u) != 0 ? 1u << (4 * i + k) : 0u;
            }
            wild = all >> g & 0x101u;
          }
#pragma unroll
          for (int i = 0; i < CN; ++i) {
            const int col = col_of(i);
            const int see = col >= rows ? 0 : one ? see_all : visible_keys(cur.seq, (row0 + col) / H, shape.cap);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int k = key0 + k0 + 8 * e;
              uint32_t& v = x[4 * (i >> 1) + 2 * e + (i & 1)];
              if (gone || k >= see) v = 0xFF800000u;                          // -inf
              else if ((wild >> (8 * e) & 1u) != 0) {
                v = 0xFF800000u;
                l[i] = __uint_as_float(0x7FC00000u);                          // NaN
              }
            }
          }
          each_piece([&](int i, uint32_t at) {
            const int key = 4 * i + sub;
            if (gone || warp * 16 + key >= hi || (all >> key & 1u) != 0) st_shared_v4(at, 0u, 0u, 0u, 0u);
          });
        }
        // ---- references
        bool move = false;
#pragma unroll
        for (int i = 0; i < CN; ++i) {
          const int a = 4 * (i >> 1) + (i & 1);
          move |= fmaxf(__uint_as_float(x[a]), __uint_as_float(x[a + 2])) * p.qscale > m[i] + kMoveLog2;
        }
        const bool moved = soft_or(move);
        if (__builtin_expect(moved, 0)) {
#pragma unroll
          for (int i = 0; i < CN; ++i) {
            const int a = 4 * (i >> 1) + (i & 1);
            float top = fmaxf(__uint_as_float(x[a]), __uint_as_float(x[a + 2])) * p.qscale;
#pragma unroll
            for (int off = 4; off <= 16; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            if (g == 0) sm->top[warp][col_of(i)] = top;
          }
          soft_sync();
#pragma unroll
          for (int i = 0; i < CN; ++i) {
            const int col = col_of(i);
            const float to = fmaxf(m[i], fmaxf(fmaxf(sm->top[0][col], sm->top[1][col]), fmaxf(sm->top[2][col], sm->top[3][col])));
            const float c = m[i] == -INFINITY ? 0.f : m[i] == INFINITY ? 1.f : ex2(m[i] - to);
            m[i] = to;
            l[i] *= c;
            if (warp == 0 && g == 0) sm->corr[col] = c;
          }
          soft_sync();
        }
        // ---- weights
        uint32_t w[2][XN / 2];     // parts; pairs of columns: w[.][2 j] of the first key, w[.][2 j + 1] of the second
#pragma unroll
        for (int j = 0; j < CN / 2; ++j) {
          const float2 ref = make_float2(m[2 * j] == -INFINITY ? 0.f : -m[2 * j], m[2 * j + 1] == -INFINITY ? 0.f : -m[2 * j + 1]);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float a = ex2(fmaf(__uint_as_float(x[4 * j + 2 * e]), p.qscale, ref.x));
            const float b = ex2(fmaf(__uint_as_float(x[4 * j + 2 * e + 1]), p.qscale, ref.y));
            l[2 * j] += a;
            l[2 * j + 1] += b;
            w[0][2 * j + e] = pack_bf16(a, b);
            w[1][2 * j + e] = pack_bf16(a - __uint_as_float(w[0][2 * j + e] << 16), b - __uint_as_float(w[0][2 * j + e] & 0xFFFF0000u));
          }
        }
        // P's place and O are free once the previous P.V has run
        if (step > 0) wait_warp(kPvDone, (step - 1) & 1);
        tc_fence_after();
        if (__builtin_expect(moved && s != t.s0, 0)) {
#pragma unroll 1
          for (int c = 0; c < quads * kR; c += 16) {
            uint32_t o[16];
            tmem_ld_32x32b_x16(my_tmem + Tm<kR>::o + c, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * sm->corr[(c + e) % kR]);
            tmem_st_32x32b_x16(my_tmem + Tm<kR>::o + c, o);
          }
          tmem_st_wait();
        }
#pragma unroll
        for (int j = 0; j < CN / 2; ++j)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const uint32_t at = p_base + p_piece<kR>(warp * 16 + g + 8 * e, j) + 4 * tq;
#pragma unroll
            for (int part = 0; part < 2; ++part)
              asm volatile("st.shared.b32 [%0], %1;" ::"r"(at + part * kPartBytes<kR>), "r"(w[part][2 * j + e]) : "memory");
          }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kPFull));
      }
      // ---- the part in this range: written out, or left for the merge
#pragma unroll
      for (int i = 0; i < CN; ++i) {
#pragma unroll
        for (int off = 4; off <= 16; off <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
        if (g == 0) {
          sm->top[warp][col_of(i)] = l[i];
          if (warp == 0) sm->m[col_of(i)] = m[i];
        }
      }
      soft_sync();
      const bool whole = t.begins && t.ends;
      float* slot = p.part + (2 * static_cast<size_t>(blockIdx.x) + (t.begins ? 1 : 0)) * latent_slot(kR, p.latent);
      if (tid < kR) {
        const float sum = (sm->top[0][tid] + sm->top[1][tid]) + (sm->top[2][tid] + sm->top[3][tid]);
        sm->inv[tid] = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
        if (!whole && tid < rows) {
          slot[static_cast<size_t>(kR) * p.latent + tid] = sm->m[tid];
          slot[static_cast<size_t>(kR) * p.latent + kR + tid] = sum;
        }
      }
      soft_sync();
      wait_warp(kPvDone, (step - 1) & 1);
      tc_fence_after();
      {
        // 16 rows of 128 channels at a time, the next ones on their way out of tensor memory. (The loop is not
        // unrolled: fetching that much code took as long as running it.)
        constexpr int B = kR / 16;
        uint32_t o[16];
        const uint32_t from = my_tmem + Tm<kR>::o;
        tmem_ld_32x32b_x16(from, o);
#pragma unroll 1
        for (int k = 0; k < quads * B; ++k) {
          const int c = k % B * 16, ch = k / B * 128 + warp * 32 + lane;
          tmem_ld_wait();
          float v[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(o[e]) * (whole ? sm->inv[c + e] : 1.f);
          if (k + 1 < quads * B) tmem_ld_32x32b_x16(from + (k + 1) * 16, o);
          if (ok) {
            if (whole) {
              // (the rows' places before the first store: one after the other took 150 clocks a row)
              long long at[16];
#pragma unroll
              for (int e = 0; e < 16; ++e) at[e] = sm->row[c + e] + ch;
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (c + e < rows) p.out[at[e]] = __float2bfloat16_rn(v[e]);
            } else {
              float* to = slot + static_cast<size_t>(c) * p.latent + ch;
#pragma unroll
              for (int e = 0; e < 16; ++e, to += p.latent)
                if (c + e < rows) *to = v[e];
            }
          }
          __syncwarp();
        }
        tmem_ld_wait();
      }
      tc_fence_before();
      if (t.begins && !t.ends && ok)
        cut = {cur.seq.q0, cur.rt, (cur.first + cur.nc - 1) / range.per - cur.first / range.per + 1, rows};
      if (t.last) break;
      work_next(bt, shape, 1, &cur);
      soft_sync();         // sm->inv and sm->top have been read
    }
    if (tid == 0) p.cut[blockIdx.x] = cut;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kSWarp) tmem_dealloc(tmem, Tm<kR>::cols);
}

template <int kR>
cudaError_t launch(const LatentAttnLaunch& a, const DeviceInfo& dev, cudaStream_t stream, std::string* msg) {
  const int width = a.layer.latent + a.layer.rope, page_size = 1 << a.layer.page_shift;
  CUtensorMap map, q_map;
  // rows of all tokens and heads in one, if they stand so and a map holds them (strides below 2^40 bytes)
  const long long q_rows = static_cast<long long>(a.batch.n_tokens) * a.H, q_bytes = q_rows * width * 2;
  const bool q_packed =
      (a.q_stride == static_cast<long long>(a.H) * width || a.batch.n_tokens == 1) && q_bytes < (1LL << 40);
  if (!encode_tiles(&map, a.layer.C, width, page_size, a.layer.num_pages, static_cast<cuuint64_t>(width) * 2,
                    static_cast<cuuint64_t>(page_size) * width * 2, page_size < kKeys ? page_size : kKeys, 1) ||
      !encode_tiles(&q_map, a.q, width, q_packed ? q_rows : 1, 1, static_cast<cuuint64_t>(width) * 2,
                    q_packed ? q_bytes : width * 2, kR, 1)) {
    *msg = "(the tensor maps of the pool and the queries cannot be encoded)";
    return cudaErrorInvalidValue;
  }
  TileParams p;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.q_stride = a.q_stride;
  p.o_stride = a.o_stride;
  p.qscale = a.scale * 1.4426950408889634f;
  p.cut = latent_cuts(a.workspace);
  p.part = latent_part(a.workspace);
  p.status = dev.status_word;
  p.batch = a.batch;
  p.num_pages = a.layer.num_pages;
  p.page_shift = a.layer.page_shift;
  p.latent = a.layer.latent;
  p.rope = a.layer.rope;
  // the rings hold the same number of steps, as far as they can
  const int quads = a.layer.latent / 128, blocks = 2 * quads + (a.layer.rope > 0 ? 1 : 0);
  const int room = kSmemBytes - kSmallBytes - blocks * kR * 128 - 2 * kPartBytes<kR>;
  const int steps = room / (quads * kUnitBytes + (a.layer.rope > 0 ? kHalf : 0));
  p.ropes = a.layer.rope == 0 ? 0 : steps < 1 ? 1 : steps > kMaxRopes ? kMaxRopes : steps;
  const int units = (room - p.ropes * kHalf) / kUnitBytes;
  p.units = units < kMaxUnits ? units : kMaxUnits;
  p.q_packed = q_packed ? 1 : 0;
  p.shape.G = a.H;
  p.shape.rows = kR;
  p.shape.chunk_shift = kChunkShift;
  p.shape.coarse = false;
  p.shape.cap = a.batch.width << a.layer.page_shift;
  p.shape.min_rows = 0;
  p.shape.max_rows = 0x7FFFFFFF;
  static SmemOnce once;
  cudaError_t e = allow_smem(latent_tile_kernel<kR>, kSmemBytes, dev.device, &once);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int grid = dev.num_sms < latent_max_blocks(1) ? dev.num_sms : latent_max_blocks(1);
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, latent_tile_kernel<kR>, map, q_map, p);
  if (e != cudaSuccess) return e;
  count_launches(1);
  return launch_latent_merge(a, kR, grid, dev, stream);
}

// Rows of a tile, by the most rows that a sequence can have.
int tile_rows(int H, int max_new) {
  const long long rows = static_cast<long long>(H) * max_new;
  return rows <= 16 ? 16 : rows <= 32 ? 32 : 64;
}

}  // namespace

size_t latent_attention_workspace(int H, int latent, int max_new, bool bf16) {
  if (!bf16) return latent_parts_bytes(kLatentRowsF32, latent, latent_max_blocks(latent_rows_blocks(latent)));
  return latent_parts_bytes(tile_rows(H, max_new), latent, latent_max_blocks(1));
}

cudaError_t launch_latent_attention(const LatentAttnLaunch& a, const DeviceInfo& dev, cudaStream_t stream,
                                    std::string* msg) {
  if (!a.bf16) return launch_latent_rows(a, dev, stream);
  switch (tile_rows(a.H, a.max_new)) {
    case 16: return launch<16>(a, dev, stream, msg);
    case 32: return launch<32>(a, dev, stream, msg);
    default: return launch<64>(a, dev, stream, msg);
  }
}

}  // namespace cxa
