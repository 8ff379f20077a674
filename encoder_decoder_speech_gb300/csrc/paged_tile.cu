// Attention of new tokens over a paged bf16 K/V cache, for sequences with many query rows
// a K/V head (prompts and chunks of them): tcgen05 products over 128-row tiles.
//
//   S = Q K^T (128 rows x a chunk of keys), P = 2^(scale log2(e) S - m), O += P V
//
// A work item is a tile of 128 query rows (128 / G tokens times the G query heads of one
// K/V head), dealt out by paged_work.cuh in chunks of 16 KB of K and of V (128 keys of 64
// channels, 64 keys of 128). Two blocks share an SM, each with its own tile, so that one
// block's products run under the other's exponentials:
//
//  * warp 4 streams by TMA: the item's Q (a box of 128 / G tokens x G heads, which lands
//    token by token, the row order of a tile), and K and V page by page into rings of two
//    and three tiles; the boxes of a chunk are issued by a lane each. A K tile comes back
//    as soon as its scores are done, a V tile after its P.V.
//  * warp 5 issues the products: scores of chunk i + 1 once the softmax warps have read
//    those of chunk i, then P.V of chunk i. P is read from tensor memory, V as it lies in
//    shared memory (rows of keys: an MN-major operand).
//  * warps 0..3 own a row a thread, so that row maxima and sums need no exchange. They take
//    a row's scores into registers at once, which lets the next chunk's scores start while
//    the exponentials run. A row's reference m moves, and O is rescaled, only when a score
//    passes it by more than 2^8 (decided per warp).
//
// Bound, at 64 channels, by the exponentials and their bookkeeping together with the
// products (about 500 clocks each a tile of 128 keys). Tensor memory: S, P and O side by
// side in 256 columns a block.
//
// P is rounded to one bf16 value (2^-9 of each weight, against the 2^-8 of the bf16
// output); sums, references and O are fp32, the sums of the values before rounding.
//
// Keys behind a tile's last visible one weigh 0 and their V rows, which may hold anything,
// are zeroed in shared memory before P.V. Keys that some rows see and others do not weigh
// 0 in the others; if one of them has a V that is not finite (0 * inf), those keys are
// added row by row on the CUDA cores instead.
#include <cuda.h>
#include <cuda_bf16.h>

#include <cmath>
#include <mutex>

#include "paged.cuh"
#include "paged_work.cuh"
#include "ptx.cuh"

namespace cxa {
namespace {

constexpr int kSoftWarps = 4;
constexpr int kTmaWarp = 4, kMmaWarp = 5;
constexpr int kThreads = 192;
constexpr int kTileRows = 128;
constexpr int kTileBytes = 16384;            // K or V of a chunk
constexpr int kKStages = 2, kVStages = 3;
constexpr int kQBytes = 32768;               // two Q tiles of 64 channels, one of 128
constexpr int kBlocksPerSm = 2;
constexpr int kMaxBlocks = 160 * kBlocksPerSm;
constexpr uint32_t kTmemCols = 256;
constexpr float kMoveLog2 = 8.f;

enum Bars { kQFull = 0, kQEmpty = 2, kKFull = 4, kKEmpty = 6, kVFull = 8, kVEmpty = 11, kSFull = 14, kSFree, kPFull, kPvDone, kBars };

struct Small {
  uint64_t bars[kBars];
  WorkScratch work;
  uint32_t bad[4];          // boxes of chunk i whose page is outside the pool, at i % 4
  volatile int abort;
  int tmem;
  int last;
  volatile int acc;         // the segment's first P.V adds to O
};

constexpr int kSmemBytes = kQBytes + (kKStages + kVStages) * kTileBytes + 1024;
static_assert(sizeof(Small) <= 1024, "the small arrays fit behind the tiles");

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
  unsigned int* counters;
  float* part;               // [2 * grid][kDh + 2][128]
  unsigned int* status;
  PagedBatch batch;
  int num_pages, Hkv, page_shift;
  WorkShape shape;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void named_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
__device__ __forceinline__ bool named_or(bool v) {
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
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&p);
}
__device__ __forceinline__ uint32_t tmem_ld_1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
  return r;
}
__device__ __forceinline__ void tmem_st_1(uint32_t taddr, uint32_t r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(r) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
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

template <int kDh>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    paged_tile_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TileParams p) {
  using T = Tile<kDh>;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  const uint32_t q_base = base, k_base = base + kQBytes, v_base = k_base + kKStages * kTileBytes;
  Small* sm = reinterpret_cast<Small*>(smem + kQBytes + (kKStages + kVStages) * kTileBytes);
  auto bar = [&](int i) { return smem_u32(&sm->bars[i]); };
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedBatch& bt = p.batch;
  const int G = p.shape.G;

  // Launched behind paged_rows_kernel of the same call, which lets this grid start only
  // after it has waited for everything before it; the two touch different rows and
  // scratch. This grid waits for that one at its end.
  WorkRange range;
  WorkCursor cur;
  const bool active = work_locate<kThreads>(bt, p.shape, p.Hkv, &sm->work, &range, &cur);
  if (active) {
    if (tid == 0) {
      for (int i = 0; i < kBars; ++i) mbar_init(bar(i), i == kSFree || i == kPFull ? kSoftWarps : 1);
      fence_mbar_init();
      sm->abort = 0;
      sm->acc = 0;
    }
    if (warp == kTmaWarp && lane == 0) {
      prefetch_tmap(&tmQ);
      prefetch_tmap(&tmK);
      prefetch_tmap(&tmV);
    }
    if (warp == kMmaWarp) {
      tmem_alloc(smem_u32(&sm->tmem), kTmemCols);
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
      if (ok && !mbar_wait(bar(i), parity, &sm->abort)) {
        ok = false;
        sm->abort = 1;
        atomicOr(p.status, kStatusTimeout);
      }
      return ok;
    };
    auto wait_warp = [&](int i, uint32_t parity) { // by a whole warp, with one answer
      wait(i, parity);
      ok = __all_sync(0xffffffffu, ok);
      return ok;
    };
    const int n_chunks = static_cast<int>(range.g1 - range.g0);

    if (warp == kTmaWarp) {
      // ---------------------------------------------------------------- copies
      const int ps_shift = min(p.page_shift, T::chunk_shift);
      const int box_rows = 1 << ps_shift;                // keys a box
      const int box = lane / T::halves, half = lane % T::halves;
      const bool mine = box < (T::chunk >> ps_shift);
      const int q_tokens = p.shape.rows / G;
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
          if (lane == 0) mbar_arrive_expect_tx(bar(kQFull + qb), static_cast<uint32_t>(T::halves * p.shape.rows * 128));
          __syncwarp();
          if (lane < T::halves)
            tma_load_3d(q_base + qb * (kQBytes / 2) + lane * (kTileRows * 128), &tmQ, bar(kQFull + qb), lane * 64,
                        cur.h * G, cur.seq.q0 + cur.rt * q_tokens);
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
        const uint32_t bad = __ballot_sync(0xffffffffu, want && page < 0 && half == 0);
        const uint32_t bytes = static_cast<uint32_t>(__popc(__ballot_sync(0xffffffffu, load)) * box_rows * 128);
        const int x = half * 64, y = at & ((1 << p.page_shift) - 1), z = page * p.Hkv + cur.h;
        const uint32_t dst = static_cast<uint32_t>(half * T::half_bytes + box * box_rows * 128);
        const int ks = i % kKStages, vs = i % kVStages;
        if (!wait_warp(kKEmpty + ks, ((i / kKStages) & 1) ^ 1)) break;
        if (lane == 0) {
          uint32_t boxes = 0;    // a bit a box
          for (uint32_t m = bad; m != 0; m &= m - 1) boxes |= 1u << ((__ffs(m) - 1) / T::halves);
          sm->bad[i & 3] = boxes;
          if (bad != 0) atomicOr(p.status, kStatusBadPage);
          mbar_arrive_expect_tx(bar(kKFull + ks), bytes);
        }
        __syncwarp();
        if (load) tma_load_3d(k_base + ks * kTileBytes + dst, &tmK, bar(kKFull + ks), x, y, z);
        sent(kKFull + ks, i / kKStages);
        if (!wait_warp(kVEmpty + vs, ((i / kVStages) & 1) ^ 1)) break;
        if (lane == 0) mbar_arrive_expect_tx(bar(kVFull + vs), bytes);
        __syncwarp();
        if (load) tma_load_3d(v_base + vs * kTileBytes + dst, &tmV, bar(kVFull + vs), x, y, z);
        sent(kVFull + vs, i / kVStages);
        if (++c == cur.nc && i + 1 < n_chunks) {
          work_next(bt, p.shape, p.Hkv, &cur);
          c = 0;
          ++item;
          fresh = true;
        }
      }
      if (!ok)      // the copies under way land before the block ends
        for (int b = 0; b < kBars; ++b)
          if (armed & (1u << b)) mbar_wait(bar(b), (parity >> b) & 1u);
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------------- products
      if (lane == 0) {
        constexpr uint32_t idesc_s = make_idesc(1u, kTileRows, T::chunk);
        constexpr uint32_t idesc_o = make_idesc(1u, kTileRows, 64) | (1u << 16);   // V MN-major
        int c = cur.c, nc = cur.nc;           // of the scores, one chunk ahead
        int item = 0;
        bool fresh = true;
        auto scores = [&](int i) {
          const int qb = item % T::q_bufs, ks = i % kKStages;
          if (fresh && !wait(kQFull + qb, (item / T::q_bufs) & 1)) return;
          fresh = false;
          if (!wait(kKFull + ks, (i / kKStages) & 1)) return;
          if (i > 0 && !wait(kSFree, (i - 1) & 1)) return;
          tc_fence_after();
#pragma unroll
          for (int h = 0; h < T::halves; ++h) {
            const uint64_t qd = smem_desc_k_sw128(q_base + qb * (kQBytes / 2) + h * (kTileRows * 128));
            const uint64_t kd = smem_desc_k_sw128(k_base + ks * kTileBytes + h * T::half_bytes);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_bf16(tmem, qd + 2 * k, kd + 2 * k, idesc_s, h + k != 0 ? 1u : 0u);
          }
          tc_commit(bar(kSFull));
          tc_commit(bar(kKEmpty + ks));
          if (++c == nc && i + 1 < n_chunks) {
            tc_commit(bar(kQEmpty + qb));
            work_next(bt, p.shape, p.Hkv, &cur);
            nc = cur.nc;
            c = 0;
            ++item;
            fresh = true;
          }
        };
        bool first = true;
        scores(0);
        for (int i = 0; i < n_chunks && ok; ++i) {
          const bool starts = first;          // chunk i starts a segment
          first = fresh && i + 1 < n_chunks;  // the scores' cursor stands at chunk i + 1 here
          if (i + 1 < n_chunks) scores(i + 1);
          const int vs = i % kVStages;
          if (!wait(kPFull, i & 1) || !wait(kVFull + vs, (i / kVStages) & 1)) break;
          tc_fence_after();
          const uint32_t acc0 = !starts || sm->acc != 0 ? 1u : 0u;
#pragma unroll
          for (int kb = 0; kb < T::chunk / 16; ++kb)
#pragma unroll
            for (int h = 0; h < T::halves; ++h)
              mma_bf16_ts(tmem + T::o_col + h * 64, tmem + T::p_col + kb * 8,
                          smem_desc_mn_sw128(v_base + vs * kTileBytes + h * T::half_bytes + kb * 2048), idesc_o,
                          kb != 0 ? 1u : acc0);
          tc_commit(bar(kPvDone));
          tc_commit(bar(kVEmpty + vs));
        }
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------------- softmax, a row a thread
      const uint32_t my_tmem = tmem + (static_cast<uint32_t>(warp * 32) << 16);
      const int box_shift = min(p.page_shift, T::chunk_shift);
      const float2 qs2 = make_float2(p.qscale, p.qscale);
      int c = cur.c, c0 = cur.c;
      float m = -INFINITY, l = 0.f;
      int row0 = 0, rows = 0, see = 0, see_all = 0, keys = 0;
      bool starts = true;
      for (int i = 0; i < n_chunks; ++i) {
        if (starts) {
          row0 = cur.rt * p.shape.rows;
          rows = min(p.shape.rows, work_rows(cur.seq, p.shape) - row0);
          see = tid < rows ? visible_keys(cur.seq, (row0 + tid) / G, p.shape.cap) : 0;
          see_all = visible_keys(cur.seq, row0 / G, p.shape.cap);
          keys = tile_keys(cur.seq, p.shape, cur.rt);
          m = -INFINITY;
          l = 0.f;
          c0 = c;
        }
        const int key0 = c << T::chunk_shift;
        wait_warp(kSFull, i & 1);
        tc_fence_after();
        const uint32_t bad = *const_cast<volatile uint32_t*>(&sm->bad[i & 3]);
        const bool special = key0 + T::chunk > see_all || bad != 0;   // some row does not see some key
        const int lim = see - key0;

        // The row's scores, all in registers, so that the next chunk's products can start
        uint32_t x[T::chunk / 32][32];
#pragma unroll
        for (int b = 0; b < T::chunk / 32; ++b) tmem_ld_32x32b_x32(my_tmem + 32 * b, x[b]);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kSFree));
        if (special) {
#pragma unroll
          for (int b = 0; b < T::chunk / 32; ++b)
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int k = 32 * b + e;
              if (k >= lim || ((bad >> (k >> box_shift)) & 1u) != 0) x[b][e] = 0xFF800000u;   // -inf
            }
        }
        float mx[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) mx[j] = -INFINITY;
#pragma unroll
        for (int b = 0; b < T::chunk / 32; ++b)
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            mx[(e / 2) & 3] = fmaxf(mx[(e / 2) & 3], fmaxf(__uint_as_float(x[b][e]), __uint_as_float(x[b][e + 1])));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.qscale;
        // the references of a warp's rows move together, to the largest score so far
        float corr = 1.f;
        const bool moved = __any_sync(0xffffffffu, top > m + kMoveLog2);
        if (moved) {
          const float to = fmaxf(m, top);
          corr = m == -INFINITY ? 0.f : ex2(m - to);
          m = to;
          l *= corr;
        }
        {
          const float ref = m == -INFINITY ? 0.f : -m;
          const float2 ref2 = make_float2(ref, ref);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int b = 0; b < T::chunk / 32; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float2 v = make_float2(__uint_as_float(x[b][2 * e]), __uint_as_float(x[b][2 * e + 1]));
              v = fma2(v, qs2, ref2);
              v.x = ex2(v.x);
              v.y = ex2(v.y);
              sum[e & 1] = add2(sum[e & 1], v);
              x[b / 2][16 * (b & 1) + e] = pack_bf16(v.x, v.y);     // behind what is still to be read
            }
          sum[0] = add2(sum[0], sum[1]);
          l += sum[0].x + sum[0].y;
        }

        // P's place and O are free once the previous P.V has run
        if (i > 0) wait_warp(kPvDone, (i - 1) & 1);
        tc_fence_after();
        if (moved && !starts) {
#pragma unroll
          for (int b = 0; b < kDh / 32; ++b) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(my_tmem + T::o_col + 32 * b, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
            tmem_st_32x32b_x32(my_tmem + T::o_col + 32 * b, o);
          }
        }
#pragma unroll
        for (int b = 0; b < T::chunk / 64; ++b) tmem_st_32x32b_x32(my_tmem + T::p_col + 32 * b, x[b]);
        tmem_st_wait();

        if (special) {
          // keys [lo, hi) of the chunk are seen by some rows and not by others, keys from hi
          // on by none
          const int lo = max(0, see_all - key0), hi = min(T::chunk, keys - key0);
          const int vs = i % kVStages;
          wait_warp(kVFull + vs, (i / kVStages) & 1);
          const int key = tid & (T::chunk - 1), half = tid >> T::chunk_shift;   // this thread's part of V
          const bool has = T::chunk * T::halves > tid;
          const bool key_bad = ((bad >> (key >> box_shift)) & 1u) != 0;
          const uint32_t vt = v_base + vs * kTileBytes;
          const uint32_t vrow = vt + half * T::half_bytes + key * 128;
          bool wild = false;
          if (has && key >= lo && key < hi && !key_bad)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint4 u = ld_shared_v4(vrow + 16 * j);
              const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) wild |= (w[e] & 0x7F80u) == 0x7F80u || (w[e] & 0x7F800000u) == 0x7F800000u;
            }
          wild = named_or(wild);
          if (wild) {
            for (int b = 0; b < kDh / 32; ++b) {
              uint32_t o[32];
              tmem_ld_32x32b_x32(my_tmem + T::o_col + 32 * b, o);
              tmem_ld_wait();
              if (starts)
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0u;
              for (int j = lo; j < hi; ++j) {
                const uint32_t w = tmem_ld_1(my_tmem + T::p_col + (j >> 1));
                tmem_ld_wait();
                if (j < lim && ((bad >> (j >> box_shift)) & 1u) == 0) {
                  const float pj = __uint_as_float((j & 1) ? w & 0xFFFF0000u : w << 16);
                  const uint32_t vr = vt + (b / 2) * T::half_bytes + j * 128;
#pragma unroll
                  for (int q = 0; q < 4; ++q) {
                    const uint4 u = ld_shared_v4(vr + (((4 * (b & 1) + q) ^ (j & 7)) << 4));
                    const uint32_t x[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                      float a0 = __uint_as_float(o[8 * q + 2 * e]), a1 = __uint_as_float(o[8 * q + 2 * e + 1]);
                      a0 = fmaf(pj, __uint_as_float(x[e] << 16), a0);
                      a1 = fmaf(pj, __uint_as_float(x[e] & 0xFFFF0000u), a1);
                      o[8 * q + 2 * e] = __float_as_uint(a0);
                      o[8 * q + 2 * e + 1] = __float_as_uint(a1);
                    }
                  }
                }
                __syncwarp();    // the next load is the whole warp's
              }
              tmem_st_32x32b_x32(my_tmem + T::o_col + 32 * b, o);
              tmem_st_wait();
            }
            for (int j = lo >> 1; 2 * j < hi; ++j) {    // P.V leaves these keys out
              uint32_t w = tmem_ld_1(my_tmem + T::p_col + j);
              tmem_ld_wait();
              w &= 2 * j >= lo ? 0u : 0x0000FFFFu;
              tmem_st_1(my_tmem + T::p_col + j, w);
            }
            tmem_st_wait();
            named_sync();      // V has been read
          }
          if (starts && tid == 0) sm->acc = wild ? 1 : 0;
          if (has && (key_bad || key >= (wild ? lo : hi)))
#pragma unroll
            for (int j = 0; j < 8; ++j) st_shared_v4(vrow + 16 * j, 0u, 0u, 0u, 0u);
          fence_proxy_async_smem();
        } else if (starts && tid == 0) {
          sm->acc = 0;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kPFull));

        const bool ends = c + 1 == cur.nc || i + 1 == n_chunks;
        starts = ends;
        if (ends) {
          // ---- the item's part in this range: written out, or left for the merge
          wait_warp(kPvDone, i & 1);
          tc_fence_after();
          const bool whole = c0 == 0 && c + 1 == cur.nc;
          const int tok = (row0 + tid) / G, hd = cur.h * G + (row0 + tid) % G;
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) +
                               (tid < rows ? (cur.seq.q0 + tok) * p.o_stride + static_cast<long long>(hd) * kDh : 0);
          float* slot = p.part + (2 * static_cast<size_t>(blockIdx.x) + (c0 == 0 ? 1 : 0)) * kTileRows * (kDh + 2);
          auto put = [&](int b, const float (&o)[32], float inv) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint4 u;
              u.x = pack_bf16(o[8 * q] * inv, o[8 * q + 1] * inv);
              u.y = pack_bf16(o[8 * q + 2] * inv, o[8 * q + 3] * inv);
              u.z = pack_bf16(o[8 * q + 4] * inv, o[8 * q + 5] * inv);
              u.w = pack_bf16(o[8 * q + 6] * inv, o[8 * q + 7] * inv);
              *reinterpret_cast<uint4*>(dst + 32 * b + 8 * q) = u;
            }
          };
          const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
          for (int b = 0; b < kDh / 32; ++b) {
            uint32_t w[32];
            tmem_ld_32x32b_x32(my_tmem + T::o_col + 32 * b, w);
            tmem_ld_wait();
            if (tid < rows && ok) {
              float o[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(w[e]);
              if (whole) {
                put(b, o, inv);
              } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) slot[(32 * b + e) * kTileRows + tid] = o[e];
              }
            }
          }
          tc_fence_before();
          if (!whole) {
            if (tid < rows && ok) {
              slot[kDh * kTileRows + tid] = m;
              slot[(kDh + 1) * kTileRows + tid] = l;
            }
            const long long owner0 = cur.first / range.per;
            const int parts = static_cast<int>((cur.first + cur.nc - 1) / range.per - owner0) + 1;
            named_sync();      // the partial state is written
            if (tid == 0) sm->last = 0;
            if (tid == 0 && ok) {
              const unsigned int n = atomic_add_acq_rel_gpu(p.counters + owner0, 1u);
              sm->last = n == static_cast<unsigned int>(parts - 1);
              if (sm->last) p.counters[owner0] = 0u;
            }
            named_sync();
            if (sm->last && tid < rows) {
              auto part = [&](int k) {
                return p.part + (2 * static_cast<size_t>(owner0 + k) + (k == 0 ? 1 : 0)) * kTileRows * (kDh + 2) + tid;
              };
              float M = -INFINITY, L = 0.f;
#pragma unroll 4
              for (int k = 0; k < parts; ++k) M = fmaxf(M, __ldcg(part(k) + kDh * kTileRows));
              const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll 4
              for (int k = 0; k < parts; ++k)
                L += __ldcg(part(k) + (kDh + 1) * kTileRows) * ex2(__ldcg(part(k) + kDh * kTileRows) - ref);
              const float linv = L > 0.f || L != L ? 1.f / L : 0.f;
#pragma unroll 1
              for (int b = 0; b < kDh / 32; ++b) {
                float o[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0.f;
#pragma unroll 2
                for (int k = 0; k < parts; ++k) {
                  const float* src = part(k);
                  const float f = ex2(__ldcg(src + kDh * kTileRows) - ref);
                  float w[32];
#pragma unroll
                  for (int e = 0; e < 32; ++e) w[e] = __ldcg(src + (32 * b + e) * kTileRows);
#pragma unroll
                  for (int e = 0; e < 32; ++e) o[e] = fmaf(f, w[e], o[e]);
                }
                put(b, o, linv);
              }
            }
          }
        }
        if (++c == cur.nc && i + 1 < n_chunks) {
          work_next(bt, p.shape, p.Hkv, &cur);
          c = 0;
        }
      }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encoder() {
  static std::once_flag once;
  static EncodeTiledFn fn = nullptr;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// A 3-D bf16 map of 64-channel boxes, swizzled for the products.
bool encode(CUtensorMap* map, const void* ptr, cuuint64_t d0, cuuint64_t d1, cuuint64_t d2, cuuint64_t s1,
            cuuint64_t s2, int b1, int b2) {
  const EncodeTiledFn fn = encoder();
  const cuuint64_t dims[3] = {d0, d1, d2};
  const cuuint64_t strides[2] = {s1, s2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(b1), static_cast<cuuint32_t>(b2)};
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn != nullptr &&
         fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kCounterBytes = (kMaxBlocks * 4 + 255) / 256 * 256;

template <int kDh>
cudaError_t launch(const PagedAttnLaunch& a, void* workspace, const DeviceInfo& dev, cudaStream_t stream,
                   std::string* msg) {
  using T = Tile<kDh>;
  TileParams prm;
  prm.out = a.out;
  prm.o_stride = a.o_stride;
  prm.qscale = a.scale * 1.4426950408889634f;
  prm.counters = static_cast<unsigned int*>(workspace);
  prm.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kCounterBytes);
  prm.status = dev.status_word;
  prm.batch = a.batch;
  prm.num_pages = a.layer.num_pages;
  prm.Hkv = a.layer.Hkv;
  prm.page_shift = a.layer.page_shift;
  const int G = a.Hq / a.layer.Hkv;
  prm.shape.G = G;
  prm.shape.rows = kTileRows / G * G;      // whole tokens
  prm.shape.chunk_shift = T::chunk_shift;
  prm.shape.cap = a.batch.width << a.layer.page_shift;
  prm.shape.min_rows = kFewRows + 1;
  prm.shape.max_rows = 0x7FFFFFFF;

  const int page_size = 1 << a.layer.page_shift;
  const int box_rows = page_size < T::chunk ? page_size : T::chunk;
  const cuuint64_t slabs = static_cast<cuuint64_t>(a.layer.num_pages) * a.layer.Hkv;
  CUtensorMap tmQ, tmK, tmV;
  if (!encode(&tmQ, a.q, kDh, a.Hq, a.batch.n_tokens, kDh * 2, static_cast<cuuint64_t>(a.q_stride) * 2, G,
              kTileRows / G) ||
      !encode(&tmK, a.layer.K, kDh, page_size, slabs, kDh * 2, static_cast<cuuint64_t>(page_size) * kDh * 2, box_rows,
              1) ||
      !encode(&tmV, a.layer.V, kDh, page_size, slabs, kDh * 2, static_cast<cuuint64_t>(page_size) * kDh * 2, box_rows,
              1)) {
    *msg = "the tensor maps of q and the pool cannot be encoded";
    return cudaErrorInvalidValue;
  }
  cudaError_t e = cudaFuncSetAttribute(paged_tile_kernel<kDh>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(paged_tile_kernel<kDh>, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  int grid = dev.num_sms * kBlocksPerSm;
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
  e = cudaLaunchKernelEx(&cfg, paged_tile_kernel<kDh>, tmQ, tmK, tmV, prm);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace

bool paged_tile_takes(int G, bool act_bf16, int max_new) {
  // A tile holds whole tokens, so G query heads have to fit into it.
  return act_bf16 && G <= kTileRows && static_cast<long long>(max_new) * G > kFewRows;
}

size_t paged_tile_workspace_bytes(int dh) {
  return kCounterBytes + static_cast<size_t>(2 * kMaxBlocks) * kTileRows * (dh + 2) * 4;
}

cudaError_t launch_paged_tile(const PagedAttnLaunch& a, void* workspace, const DeviceInfo& dev, cudaStream_t stream,
                              std::string* msg) {
  return a.dh == 64 ? launch<64>(a, workspace, dev, stream, msg) : launch<128>(a, workspace, dev, stream, msg);
}

}  // namespace cxa
