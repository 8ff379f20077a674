// The expansion of latent rows into pages of keys and values in bf16, as tcgen05 products:
//
//   K_h(t) = [ r_t | c_t WK_h ],  V_h(t) = c_t WV_h
//
// Two blocks work as a pair (cta_group::2) on two tiles of 128 positions, of any sequences, by 256 columns. Each block
// holds its own positions and streams half of the columns' weights: half the traffic of blocks by themselves
// (which took 183 us for 32768 positions, 20 heads of 128, 512 + 64 channels). The columns are blocks of 64,
// those of a head's K and V behind each other and heads in turn: any four of them make a product, so that all
// products are of the full width, whatever heads are made of (products of one head's 192 columns took as long as
// ones of 256). Weights are taken as they are, [latent][columns]: an operand across the channels
// (MN-major) needs no copy of theirs turned round, and one along them is no faster.
//
// All (pairs of tiles, products) are numbered densely, positions first, and a pair takes an equal range of them. The
// positions' latent rows stay in shared memory over all products (128 KB of 512 channels); what streams are the
// weights, 64 channels a stage. (Stages of 32 channels, in smaller boxes, take the copy warp longer than the
// products: 165 us.)
//
//  * warp 9 copies: latent rows page by page, 64 channels at a time, and the weights' stages. All of a pair's
//    copies are counted by the even block's barriers.
//  * warp 8 of the even block issues the products, into two buffers of tensor memory.
//  * warps 0 to 7 take the sums out, a position a lane and 128 columns a group of four warps, round them, and turn
//    them round through shared memory, 64 channels at a time, so that 8 lanes write a row's 128 bytes together
//    (32 bytes a lane straight from registers: 150 us). The rotated part, the same in every head, stays in
//    registers. They give tensor memory back by an arrival without a release: one with it waits until the
//    rows written before are performed (98 us against 76 where 128 latent channels make the products short).
//
// Bound by the products, 2 latent operations a value; the values written (2 bytes each) take nearly as long. 32768
// positions, 20 heads of 128, 512 + 64 channels: 109 us, 1180 TFLOP/s and 3.5 TB/s (main loop alone 67 at
// cuBLAS's rate; without the stores 85). 24 sequences of up to 1500 positions, 8 heads of 64, 256 + 32: 24 us, of
// which the floor of bytes is 9.5: start (barriers, tensor memory and maps are set up behind the wait for the kernel
// before), and 408 products over 76 pairs, so that pairs with six set the end.
#include <cuda.h>
#include <cuda_bf16.h>

#include "cluster.cuh"
#include "expand.cuh"
#include "ptx.cuh"
#include "span_work.cuh"
#include "tc_util.cuh"

namespace cxa {
namespace {

constexpr int kRows = 128;
constexpr int kOutWarps = 8, kMmaWarp = kOutWarps, kTmaWarp = kMmaWarp + 1, kThreads = (kTmaWarp + 1) * 32;
constexpr int kBlocks = 4, kCols = 64;    // blocks of a product, and columns of a block
constexpr int kABlock = 16384;            // 64 channels of 128 positions
constexpr int kStep = 64;                 // channels of a stage of the weights
constexpr int kBox = kStep * kCols * 2;   // of a block
constexpr int kStage = kBlocks / 2 * kBox;
constexpr int kMaxStages = 16, kMaxA = 8;
constexpr int kPutBytes = 32 * kCols * 2;  // 32 rows of them, as they are written
constexpr int kOutBytes = kOutWarps * kPutBytes;      // a buffer of each warp
constexpr int kSmemBytes = 232448, kSmallBytes = 3 << 10;

enum Bars {
  kAFull = 0,
  kAEmpty = kAFull + kMaxA,
  kBFull = kAEmpty + kMaxA,
  kBEmpty = kBFull + kMaxStages,
  kDFull = kBEmpty + kMaxStages,
  kDFree = kDFull + 2,
  kBars = kDFree + 2
};
struct Small {
  uint64_t bars[kBars];
  SpanScratch span;
  volatile int abort;
  int tmem;
};
static_assert(sizeof(Small) <= kSmallBytes, "the small arrays fit");

struct TileParams {
  const __nv_bfloat16* C;
  __nv_bfloat16 *K, *V;
  unsigned int* status;
  int B, num_pages, page_shift, width, latent, rope;
  int to_pages, to_shift, to_width, H, dh;
  const int *from, *kv_len, *table, *to_table;
  int k_blocks, head_blocks, blocks, products;      // blocks of a head's K, of a head, of all heads
  int k_first;               // the first channel of K's blocks
  int stages;
};

__global__ void __launch_bounds__(kThreads, 1)
    expand_tile_kernel(const __grid_constant__ CUtensorMap tmC, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TileParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const int a_blocks = p.latent / 64, steps = a_blocks;
  const uint32_t a_base = smem_u32(smem), b_base = a_base + a_blocks * kABlock;
  const uint32_t s_base = b_base + p.stages * kStage;
  Small* sm = reinterpret_cast<Small*>(smem + kSmemBytes - kSmallBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nope = p.dh - p.rope;
  const uint32_t rank = cluster_rank();
  const bool even = rank == 0;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int cap = p.width << p.page_shift, to_cap = p.to_width << p.to_shift;
  auto tiles = [&](int b) {
    const ExpandSpan s = expand_span(p.from, p.kv_len, cap, b);
    return s.hi > s.lo ? (s.hi + kRows - 1) / kRows - s.lo / kRows : 0;
  };
  auto count = [&](int b) {
    if (blockIdx.x == 0 && expand_passes(p.from, p.kv_len, cap, b)) atomicOr(p.status, kStatusBadPage);
    return tiles(b);
  };
  // this pair's work [g0, g1), and the sequence of its first tile; the same in both blocks
  int g0 = 0, g1 = 0, total = 0, b = 0, first = 0;
  if (!span_find<kThreads>(
          p.B, count, &sm->span,
          [&](int n) {
            const long long pairs = static_cast<long long>(n + 1) / 2 * p.products, by = gridDim.x / 2, at = blockIdx.x / 2;
            total = n;
            if (pairs > 0x7FFFFFFFLL - 1024) return -1;
            g0 = static_cast<int>(pairs / by * at + min(at, pairs % by));
            g1 = g0 + static_cast<int>(pairs / by + (at < pairs % by ? 1 : 0));
            return g0 < g1 ? g0 / p.products * 2 : -1;
          },
          &b, &first))
    return;
  Waits w = {smem_u32(sm->bars), &sm->abort, p.status, true};
  if (tid == 0) {
    for (int i = 0; i < kBars; ++i) mbar_init(w.bar(i), i >= kDFree ? 2 * kOutWarps : 1);
    fence_mbar_init();
    sm->abort = 0;
  }
  if (warp == kTmaWarp && lane == 0) {
    prefetch_tmap(&tmC);
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  if (warp == kMmaWarp) {
    tmem_alloc_pair(smem_u32(&sm->tmem), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();      // both blocks' barriers are there before anything arrives from the other
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, static_cast<uint32_t>(sm->tmem), 0);

  // To tile i of all (i < total, not before the last one asked for): b is its sequence.
  auto seek = [&](int i) {
    for (int n = tiles(b); i - first >= n; n = tiles(b)) {
      first += n;
      ++b;
    }
    return (expand_span(p.from, p.kv_len, cap, b).lo / kRows + (i - first)) * kRows;      // its first position
  };

  if (warp == kTmaWarp) {
    fence_proxy_async_global();
    const int box_shift = min(p.page_shift, 7), box_rows = 1 << box_shift, per_tile = kRows >> box_shift;
    int stage = 0, tile = 0, page = -1, y = 0;
    uint32_t round = 0, armed = 0, parity = 0, a_armed = 0, a_parity = 0, a_bytes = 0;
    for (int g = g0; g < g1 && w.ok; ++g) {
      const int grp = g % p.products;
      const bool fresh = g == g0 || grp == 0;
      if (fresh) {
        // the boxes of both blocks' tiles, a lane each: the even block counts them all
        page = -1;
        int boxes_there = 0;
        for (int t = 0; t < 2; ++t) {
          const int i = g / p.products * 2 + t;
          int got = -1, slot = 0;
          if (i < total) {
            const int at = seek(i) + lane * box_rows;
            const ExpandSpan span = expand_span(p.from, p.kv_len, cap, b);
            if (lane < per_tile && at < span.hi && at + box_rows > span.lo)
              got = paged_lookup(p.table + static_cast<size_t>(b) * p.width, p.width, p.page_shift, p.num_pages, at);
            slot = at & ((1 << p.page_shift) - 1);
          }
          boxes_there += __popc(__ballot_sync(0xffffffffu, got >= 0));
          if (t == static_cast<int>(rank)) {
            page = got;
            y = slot;
          }
        }
        a_bytes = static_cast<uint32_t>(boxes_there * box_rows * 128);
        ++tile;
      }
      // this block's half of the columns: a block of them a lane
      const int id = grp * kBlocks + static_cast<int>(rank) * (kBlocks / 2) + lane, h = id / p.head_blocks, j = id % p.head_blocks;
      const bool mine = lane < kBlocks / 2 && id < p.blocks, v = j >= p.k_blocks;
      const int col = v ? h * p.dh + (j - p.k_blocks) * kCols : h * nope + p.k_first - p.rope + j * kCols;
      const uint32_t b_bytes = static_cast<uint32_t>(min(kBlocks, p.blocks - grp * kBlocks) * kBox);
      for (int k = 0; k < steps; ++k) {
        if (fresh) {
          if (!w.warp(kAEmpty + k, tile & 1, kStatusTimeout)) break;      // (the first passes: tile is 1)
          if (even && lane == 0) mbar_arrive_expect_tx(w.bar(kAFull + k), a_bytes);
          __syncwarp();
          if (page >= 0)
            tma_load_3d_pair(a_base + k * kABlock + lane * box_rows * 128, &tmC, mapa_shared(w.bar(kAFull + k), 0), k * 64,
                             y, page);
          a_armed |= 1u << k;
          a_parity = (a_parity & ~(1u << k)) | (static_cast<uint32_t>(tile - 1) & 1u) << k;
        }
        if (!w.warp(kBEmpty + stage, (round & 1) ^ 1, kStatusTimeout)) break;
        if (even && lane == 0) mbar_arrive_expect_tx(w.bar(kBFull + stage), b_bytes);
        __syncwarp();
        if (mine)
          tma_load_2d_pair(b_base + stage * kStage + lane * kBox, v ? &tmV : &tmK, mapa_shared(w.bar(kBFull + stage), 0), col,
                           k * kStep);
        armed |= 1u << stage;
        parity = (parity & ~(1u << stage)) | (round & 1u) << stage;
        if (++stage == p.stages) {
          stage = 0;
          ++round;
        }
      }
    }
    if (!w.ok && even) {      // the copies under way land before the pair ends
      for (int i = 0; i < p.stages; ++i)
        if (armed & (1u << i)) mbar_wait(w.bar(kBFull + i), (parity >> i) & 1u);
      for (int i = 0; i < a_blocks; ++i)
        if (a_armed & (1u << i)) mbar_wait(w.bar(kAFull + i), (a_parity >> i) & 1u);
    }
  } else if (warp == kMmaWarp) {
    constexpr uint64_t hi = desc_high(1024);
    const uint32_t idesc = make_idesc(1u, 2 * kRows, kBlocks * kCols) | 1u << 16;
    int stage = 0, tile = 0;
    uint32_t round = 0;
    for (int g = g0, i = 0; even && g < g1 && w.ok; ++g, ++i) {
      const int grp = g % p.products;
      const bool fresh = g == g0 || grp == 0, last = g + 1 == g1 || grp + 1 == p.products;
      tile += fresh ? 1 : 0;
      if (!w.warp(kDFree + (i & 1), ((i >> 1) & 1) ^ 1, kStatusTimeout)) break;
      for (int k = 0; k < steps; ++k) {
        if (fresh && !w.warp(kAFull + k, (tile - 1) & 1, kStatusTimeout)) break;
        if (!w.warp(kBFull + stage, round & 1, kStatusTimeout)) break;
        tc_fence_after();
        // (known to be the same in every lane, the operands' addresses need no carrying over from one)
        const int at = __shfl_sync(0xffffffffu, stage | k << 8 | (i & 1) << 16, 0);
        const uint32_t al = desc_low(a_base + (at >> 8 & 255) * kABlock, 16), bl = desc_low(b_base + (at & 255) * kStage, kBox);
        const uint32_t d = tmem + (at >> 16) * 256, first_k = (at >> 8 & 255) == 0 ? 0u : 1u;
        if (elect_one()) {
#pragma unroll
          for (int s = 0; s < kStep / 16; ++s)      // 16 channels: 32 bytes of a position's row, 16 rows of the weights
            mma_bf16_pair(d, hi | (al + 2 * s), hi | (bl + s * (2048 >> 4)), idesc, s != 0 ? 1u : first_k);
          tc_commit_pair(w.bar(kBEmpty + stage), 0x3);
          if (last) tc_commit_pair(w.bar(kAEmpty + k), 0x3);
          if (k + 1 == steps) tc_commit_pair(w.bar(kDFull + (i & 1)), 0x3);
        }
        __syncwarp();
        if (++stage == p.stages) {
          stage = 0;
          ++round;
        }
      }
    }
    __syncwarp();
  } else {
    // a position a lane, two of a product's four blocks of columns
    const int quad = warp & 3, half = warp >> 2;
    const uint32_t my_tmem = tmem + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(half * (kBlocks / 2 * kCols));
    const uint32_t buf = s_base + warp * kPutBytes;
    const uint32_t mine = lane * 128, swz = static_cast<uint32_t>(lane & 7) << 4;      // its row of a buffer
    const int sub = lane >> 3, piece = lane & 7;
    // the pool's rows (of head 0) that this lane writes a 16-byte piece of (-1: none), and that piece of their
    // rotated parts
    long long to[8];
    uint4 rotated[8];
    for (int g = g0, i = 0; g < g1; ++g, ++i) {
      const int grp = g % p.products;
      long long row = -1;
      if (g == g0 || grp == 0) {
        const int nth = g / p.products * 2 + static_cast<int>(rank);
        const int t = nth < total ? seek(nth) + quad * 32 + lane : 0;
        long long dst = -1;
        const ExpandSpan span = nth < total ? expand_span(p.from, p.kv_len, cap, b) : ExpandSpan{0, 0};
        if (t >= span.lo && t < span.hi) {
          const int sp = paged_lookup(p.table + static_cast<size_t>(b) * p.width, p.width, p.page_shift, p.num_pages, t);
          const int dp = paged_lookup(p.to_table + static_cast<size_t>(b) * p.to_width, p.to_width, p.to_shift, p.to_pages,
                                      t < to_cap ? t : -1);
          if (sp < 0 || dp < 0) {
            atomicOr(p.status, kStatusBadPage);
          } else {
            dst = ((static_cast<long long>(dp) * p.H) << p.to_shift) + (t & ((1 << p.to_shift) - 1));
            row = ((static_cast<long long>(sp) << p.page_shift) + (t & ((1 << p.page_shift) - 1))) * (p.latent + p.rope);
          }
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) to[n] = __shfl_sync(0xffffffffu, dst, n * 4 + sub);
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const long long from = __shfl_sync(0xffffffffu, row, n * 4 + sub);
          if (from >= 0 && piece * 8 < p.rope)
            rotated[n] = *reinterpret_cast<const uint4*>(p.C + from + p.latent + piece * 8);
        }
      }
      w.warp(kDFull + (i & 1), (i >> 1) & 1, kStatusTimeout);
      tc_fence_after();
      const uint32_t d = my_tmem + (i & 1) * 256;
      const int id = grp * kBlocks + half * (kBlocks / 2);
      int h = id / p.head_blocks, j = id % p.head_blocks;
      uint32_t x[2][32];
      tmem_ld_32x32b_x32(d, x[0]);
      tmem_ld_32x32b_x32(d + 32, x[1]);
#pragma unroll
      for (int n = 0; n < kBlocks / 2; ++n) {
        tmem_ld_wait();
        uint32_t v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e)
          v[e] = pack_bf16(__uint_as_float(x[e >> 4][2 * e & 31]), __uint_as_float(x[e >> 4][(2 * e & 31) + 1]));
        if (n == 0) {      // under what is done with the first block
          tmem_ld_32x32b_x32(d + kCols, x[0]);
          tmem_ld_32x32b_x32(d + kCols + 32, x[1]);
        } else {
          tc_fence_before();
          __syncwarp();
          // the even block's products wait for both
          if (lane == 0) mbar_arrive_cluster_relaxed(w.bar(kDFree + (i & 1)), 0);
        }
        if (id + n < p.blocks && w.ok) {
          const bool is_k = j < p.k_blocks;
          const int c0 = is_k ? p.k_first + j * kCols : (j - p.k_blocks) * kCols;
          const int skip = is_k && j == 0 ? p.rope - p.k_first : 0;      // channels of the rotated part (below 64)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            st_shared_v4(buf + mine + ((16u * e) ^ swz), v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          __syncwarp();
          // 8 lanes a row
          const long long at = (static_cast<long long>(h) << p.to_shift) * p.dh + piece * 8;
          __nv_bfloat16* base = (is_k ? p.K : p.V) + at + c0;
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            uint4 u = ld_shared_v4(buf + (r * 4 + sub) * 128 + ((piece ^ ((r * 4 + sub) & 7)) << 4));
            if (piece * 8 < skip) u = rotated[r];
            if (to[r] >= 0) *reinterpret_cast<uint4*>(base + to[r] * p.dh) = u;
          }
          // (a rotated part of 64 channels goes with the block behind it)
          if (is_k && j == 0 && p.k_first > 0)
#pragma unroll
            for (int r = 0; r < 8; ++r)
              if (to[r] >= 0) *reinterpret_cast<uint4*>(p.K + at + to[r] * p.dh) = rotated[r];
          __syncwarp();
          if (++j == p.head_blocks) {
            j = 0;
            ++h;
          }
        }
      }
    }
  }
  tc_fence_before();
  cluster_sync();      // neither block leaves while the pair's products or arrivals may still touch it
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc_pair(tmem, 512);
}

// A 2-D bf16 map of boxes of 64 columns by 64 rows of a [rows][cols] matrix.
bool encode_weights(CUtensorMap* map, const void* ptr, int rows, int cols) {
  const EncodeTiledFn fn = tensor_map_encoder();
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * 2};
  const cuuint32_t box[2] = {kCols, kStep}, estr[2] = {1, 1};
  return fn != nullptr &&
         fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_latent_expand(const LatentExpandLaunch& a, const DeviceInfo& dev, cudaStream_t stream,
                                 std::string* msg) {
  if (!a.bf16) return launch_expand_rows(a, dev, stream);
  const int width = a.layer.latent + a.layer.rope, page_size = 1 << a.layer.page_shift, H = a.to.Hkv;
  const int nope = a.dh - a.layer.rope;
  CUtensorMap c, k, v;
  if (!encode_tiles(&c, a.layer.C, width, page_size, a.layer.num_pages, static_cast<cuuint64_t>(width) * 2,
                    static_cast<cuuint64_t>(page_size) * width * 2, page_size < kRows ? page_size : kRows, 1) ||
      !encode_weights(&k, a.WK, a.layer.latent, H * nope) || !encode_weights(&v, a.WV, a.layer.latent, H * a.dh)) {
    *msg = "(the tensor maps of the pool and the weights cannot be encoded)";
    return cudaErrorInvalidValue;
  }
  TileParams p;
  p.C = static_cast<const __nv_bfloat16*>(a.layer.C);
  p.K = static_cast<__nv_bfloat16*>(a.to.K);
  p.V = static_cast<__nv_bfloat16*>(a.to.V);
  p.status = dev.status_word;
  p.B = a.B;
  p.num_pages = a.layer.num_pages;
  p.page_shift = a.layer.page_shift;
  p.width = a.width;
  p.latent = a.layer.latent;
  p.rope = a.layer.rope;
  p.to_pages = a.to.num_pages;
  p.to_shift = a.to.page_shift;
  p.to_width = a.to_width;
  p.H = H;
  p.dh = a.dh;
  p.from = a.from;
  p.kv_len = a.kv_len;
  p.table = a.table;
  p.to_table = a.to_table;
  p.k_first = a.layer.rope / kCols * kCols;
  p.k_blocks = (a.dh - p.k_first) / kCols;
  p.head_blocks = p.k_blocks + a.dh / kCols;
  p.blocks = H * p.head_blocks;
  p.products = (p.blocks + kBlocks - 1) / kBlocks;
  const int stages = (kSmemBytes - kSmallBytes - kOutBytes - p.latent / 64 * kABlock) / kStage;
  p.stages = stages < kMaxStages ? stages : kMaxStages;
  static SmemOnce once;
  cudaError_t e = allow_smem(expand_tile_kernel, kSmemBytes, dev.device, &once);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // the pairs that are resident at once, asked for once a device
  static int resident[128];
  int pairs = dev.device >= 0 && dev.device < 128 ? resident[dev.device] : 0;
  if (pairs == 0) {
    e = cudaOccupancyMaxActiveClusters(&pairs, expand_tile_kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (pairs < 1) {
      *msg = "(pairs of blocks cannot be resident)";
      return cudaErrorInvalidValue;
    }
    if (dev.device >= 0 && dev.device < 128) resident[dev.device] = pairs;      // (two threads may both: no harm)
  }
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, expand_tile_kernel, c, k, v, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace cxa
