// Eviction from a paged cache by gathered attention weight.
//
// evict_select_kernel finds, for every (layer, sequence, K/V head), the keep heaviest positions (the
// first and the last ones before all others) and lists them in order. A cluster of up to 8 blocks has the
// item's keys (weights as integers in their order) in shared memory, read once; passes over their digits, with
// histograms added up over distributed shared memory, find the keep-th largest; one more writes the
// positions above it, and of those equal to it the first ones. (A block an item, which read the weights anew in
// each pass: 225 us for 32 lists of 65536; a cluster 29, of which the first reads of the weights take 5 to 10, the
// passes 3 each.) Items of up to 4096 positions take one block, those of up to 16384 four. evict_copy_kernel
// copies the listed rows of K, V and weights, a block 32 of them (rows looked up and read two or four at a time by
// a thread: slower, 83 and 89 us).
// Bound by memory: weights are read once, what stays is read and written once. 4 sequences of up to 65536 keys of
// 8 heads of 128 down to 8192, bf16: 79 us, 44 of them the copy at 6.2 TB/s; six layers of 16 windows
// of 448 keys down to 112: 18.9 us, latency of the two kernels.
#include <algorithm>

#include "cluster.cuh"
#include "latent.cuh"
#include "ptx.cuh"

namespace cxa {
namespace {

constexpr int kMaxCluster = 8;
constexpr int kShort = 4096;         // positions of an item that one block takes
// Keys in a block's shared memory; more are read again. Fewer where an SM has more than one block.
constexpr int kMaxRoom = 49152, kSharedRoom = 21504;
constexpr int kCopyThreads = 128, kCopyRows = 32;

struct EvictParams {
  EvictLaunch a;
  unsigned int* status;
};

// Larger for larger weights, 0xFFFFFFFF for positions that stay in any case; 0 for NaN.
__device__ __forceinline__ uint32_t order_key(float w, bool stays) {
  if (stays) return 0xFFFFFFFFu;
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The word at the same shared-memory offset as `local`, in cluster block `rank`.
__device__ __forceinline__ int ld_cluster(const int* local, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(local), rank)) : "memory");
  return v;
}

// The keys that a sequence has.
__device__ __forceinline__ int length_of(const EvictLaunch& a, int b) {
  return min(max(0, a.kv_len[b]), a.width << a.page_shift);
}

// The blocks that take an item of so many positions.
__host__ __device__ constexpr int blocks_of(long long positions) {
  return positions <= kShort ? 1 : positions <= 4 * kShort ? kMaxCluster / 2 : kMaxCluster;
}

// Alone: one block an item, digits of 8 bits; otherwise a cluster of 4 or 8, digits of 11, 11 and 10.
// By all threads of the block, or of the cluster.
template <bool kAlone, int kThreads>
__device__ __forceinline__ void select_item(const EvictParams& p, int item, int kv, int blocks, uint32_t* s_key, int room) {
  constexpr int kWarps = kThreads / 32, kBins = kAlone ? 256 : 2048, kPasses = kAlone ? 4 : 3;
  constexpr int kHists = kAlone ? 1 : kPasses;        // (one a pass: other blocks may still read the last one's)
  __shared__ __align__(16) int s_hist[kHists][kBins];              // of this block
  __shared__ int s_group[kHists][kAlone ? 1 : kBins / 32];         // sums of 32 of them
  __shared__ int s_scan[2][kWarps];
  __shared__ int s_count[2];
  __shared__ uint32_t s_prefix;
  __shared__ int s_left;
  const EvictLaunch& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (kAlone) blocks = 1;
  const int rank = kAlone ? 0 : static_cast<int>(cluster_rank());
  const int h = item % a.Hkv, b = item / a.Hkv % a.B, l = item / a.Hkv / a.B;
  const int m = min(kv, a.keep);
  if (tid == 0 && rank == 0 && a.kv_len[b] > kv) atomicOr(p.status, kStatusBadPage);
  if (l == 0 && h == 0 && tid == 0 && rank == 0) a.out_len[b] = m;
  int* kept = a.kept + static_cast<size_t>(item) * a.keep;
  for (int i = m + rank * kThreads + tid; i < a.keep; i += blocks * kThreads) kept[i] = -1;
  if (m == kv) {        // (the same in the whole cluster)
    for (int i = rank * kThreads + tid; i < m; i += blocks * kThreads) kept[i] = i;
    return;
  }
  const int* row = a.table + static_cast<size_t>(b) * a.width;
  const float* W = a.W + (static_cast<size_t>(l) * a.num_pages * a.Hkv << a.page_shift);
  auto stays = [&](int t) { return t < a.first || t >= kv - a.recent; };
  auto page_of = [&](int t) { return paged_lookup(row, a.width, a.page_shift, a.num_pages, t); };
  auto weight = [&](int page, int t) {
    return __ldcg(W + ((static_cast<size_t>(page) * a.Hkv + h) << a.page_shift) + (t & ((1 << a.page_shift) - 1)));
  };
  auto key_of = [&](int t) {
    const int page = stays(t) ? -2 : page_of(t);
    if (page == -1) atomicOr(p.status, kStatusBadPage);
    return order_key(page < 0 ? 0.f : weight(page, t), stays(t));
  };
  // this block's positions [lo, lo + n)
  const int per = ((kv + blocks - 1) / blocks + 31) / 32 * 32;
  const int lo = min(kv, rank * per), n = min(kv, lo + per) - lo, held = min(n, room);
  // (a batch of pages is looked up before their weights are: one after the other took 5 to 12 us of 8192 keys)
  constexpr int kBatch = kAlone ? 2 : 8;
  for (int i = tid; i < held; i += kBatch * kThreads) {
    int page[kBatch];
    float w[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int at = i + j * kThreads;
      page[j] = at < held && !stays(lo + at) ? page_of(lo + at) : -2;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) w[j] = page[j] >= 0 ? weight(page[j], lo + i + j * kThreads) : 0.f;
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int at = i + j * kThreads;
      if (page[j] == -1) atomicOr(p.status, kStatusBadPage);
      if (at < held) s_key[at] = order_key(w[j], stays(lo + at));
    }
  }
  auto key = [&](int i) { return i < held ? s_key[i] : key_of(lo + i); };
  uint32_t prefix = 0;
  int left = m;               // to be taken among the keys that share the prefix
  int above = 0;              // keys above the bins that are looked at
  // Of counts c in 32 lanes, the later ones above, the lane in which the count from above reaches `left`.
  auto find = [&](int c) {
    int sum = c;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int o = __shfl_down_sync(0xffffffffu, sum, off);
      if (lane + off < 32) sum += o;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, above + sum >= left && above + sum - c < left);
    const int at = 31 - __clz(hit | 1u);
    above += __shfl_sync(0xffffffffu, sum - c, at);
    return at;
  };
#pragma unroll 1
  for (int pass = 0; pass < kPasses; ++pass) {
    const int shift = kAlone ? 24 - 8 * pass : pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int top = kAlone ? 32 - 8 * pass : pass == 0 ? 32 : pass == 1 ? 21 : 10;
    int* hist = s_hist[kAlone ? 0 : pass];
    if (kAlone || pass == 0) {
      for (int i = tid; i < kHists * kBins; i += kThreads) s_hist[0][i] = 0;
      __syncthreads();
    }
    for (int i = tid; i < n; i += kThreads) {
      const uint32_t k = key(i);
      if (pass == 0 || (k >> top) == (prefix >> top)) atomicAdd(&hist[(k >> shift) & ((1u << (top - shift)) - 1u)], 1);
    }
    __syncthreads();
    if constexpr (!kAlone) {
      for (int g = warp; g < kBins / 32; g += kWarps) {
        const int sum = __reduce_add_sync(0xffffffffu, hist[g * 32 + lane]);
        if (lane == 0) s_group[pass][g] = sum;
      }
      cluster_sync();
    }
    above = 0;
    if constexpr (kAlone) {
      if (warp == 0) {
        int c[8], sum = 0;      // this lane's bins
        *reinterpret_cast<int4*>(&c[0]) = *reinterpret_cast<const int4*>(&hist[lane * 8]);
        *reinterpret_cast<int4*>(&c[4]) = *reinterpret_cast<const int4*>(&hist[lane * 8 + 4]);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += c[i];
        const int at = find(sum);
        if (lane == at) {
          int bin = 7;
#pragma unroll
          for (int i = 7; i > 0; --i)
            if (bin == i && above + c[i] < left) {
              above += c[i];
              bin = i - 1;
            }
          s_prefix = prefix | static_cast<uint32_t>(lane * 8 + bin) << shift;
          s_left = left - above;
        }
      }
    } else {
      if (warp == 0) {
        // the sum over the cluster, all reads under way at once; 64 groups in the order of their bins, two a lane
        auto over_all = [&](const int* local) {
          int sum = 0;
#pragma unroll
          for (int c = 0; c < kMaxCluster; ++c)
            if (c < blocks) sum += ld_cluster(local, static_cast<uint32_t>(c));
          return sum;
        };
        const int c0 = over_all(&s_group[pass][lane * 2]), c1 = over_all(&s_group[pass][lane * 2 + 1]);
        const int two = find(c0 + c1);
        const int upper_count = __shfl_sync(0xffffffffu, c1, two);
        const bool upper = above + upper_count >= left;
        if (!upper) above += upper_count;
        const int group = two * 2 + (upper ? 1 : 0);
        const int bin = find(over_all(&hist[group * 32 + lane]));
        if (lane == 0) {
          s_prefix = prefix | static_cast<uint32_t>(group * 32 + bin) << shift;
          s_left = left - above;
        }
      }
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_left;
  }
  // prefix is the m-th largest key; `left` of the positions that have it stay. Each warp has a run of the
  // block's positions: how many of both there are in it, and with what stands before it, where they go.
  const int run = ((n + kWarps - 1) / kWarps + 31) / 32 * 32, i0 = min(n, warp * run), i1 = min(n, i0 + run);
  int count = 0, tied = 0;
#pragma unroll 4
  for (int i = i0; i < i1; i += 32) {
    const uint32_t k = i + lane < i1 ? key(i + lane) : 0u;
    count += __popc(__ballot_sync(0xffffffffu, i + lane < i1 && k > prefix));
    tied += __popc(__ballot_sync(0xffffffffu, i + lane < i1 && k == prefix));
  }
  if (lane == 0) {
    s_scan[0][warp] = count;
    s_scan[1][warp] = tied;
  }
  __syncthreads();
  int out = lane < warp ? s_scan[0][lane] : 0, ties = lane < warp ? s_scan[1][lane] : 0;      // in the positions before
  if constexpr (!kAlone) {
    if (warp == 0) {
      int x = lane < kWarps ? s_scan[0][lane] : 0, y = lane < kWarps ? s_scan[1][lane] : 0;
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, off);
        y += __shfl_xor_sync(0xffffffffu, y, off);
      }
      if (lane == 0) {
        s_count[0] = x;
        s_count[1] = y;
      }
    }
    cluster_sync();
    if (lane < rank) {
      out += ld_cluster(&s_count[0], static_cast<uint32_t>(lane));
      ties += ld_cluster(&s_count[1], static_cast<uint32_t>(lane));
    }
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) {
    out += __shfl_xor_sync(0xffffffffu, out, off);
    ties += __shfl_xor_sync(0xffffffffu, ties, off);
  }
  const uint32_t below = (1u << lane) - 1u;
  for (int i = i0; i < i1; i += 32) {
    const uint32_t k = i + lane < i1 ? key(i + lane) : 0u;
    const bool more = i + lane < i1 && k > prefix, tie = i + lane < i1 && k == prefix;
    const uint32_t ma = __ballot_sync(0xffffffffu, more), mt = __ballot_sync(0xffffffffu, tie);
    const int my_tie = ties + __popc(mt & below);
    // behind all larger ones before it, and the ties before it that stay
    const int at = out + __popc(ma & below) + min(my_tie, left);
    if ((more || (tie && my_tie < left)) && at < m) kept[at] = lo + i + lane;
    out += __popc(ma);
    ties += __popc(mt);
  }
  if constexpr (!kAlone) cluster_sync();      // no block goes on while another may read its counts
}

// Tables of up to kShort positions: a block an item.
constexpr int kSmallThreads = 256;
__global__ void __launch_bounds__(kSmallThreads) evict_select_kernel(const __grid_constant__ EvictParams p, int room) {
  extern __shared__ uint32_t s_key[];        // [room]
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int item = blockIdx.x;
  select_item<true, kSmallThreads>(p, item, length_of(p.a, item / p.a.Hkv % p.a.B), 1, s_key, room);
}

// Wider ones: a cluster of `launched` blocks an item, of which those stay that its sequence has work for; the others
// leave. 768 windows of up to 448 keys: 22 us in a table of 512 positions, 65 in one of 1,048,576, and 565 there where
// all blocks took part, with room for the table's keys. (A grid that stays and deals itself the items: 45 us there, but
// 61 in place of 53 for 128 of up to 8000 keys, and 235 in place of 172 for 128 of up to 120,000.)
constexpr int kWideThreads = 512;
// (by itself, so that it costs the other way no registers: 80.5 us, 79.2 so, for 32 lists of up to 65536)
__device__ __noinline__ void select_short(const EvictParams& p, int item, int kv, uint32_t* s_key, int room) {
  select_item<true, kWideThreads>(p, item, kv, 1, s_key, room);
}
__global__ void __launch_bounds__(kWideThreads, 4)
    evict_select_wide_kernel(const __grid_constant__ EvictParams p, int launched, int room) {
  extern __shared__ uint32_t s_key[];        // [room]
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int item = blockIdx.x / launched, kv = length_of(p.a, item / p.a.Hkv % p.a.B);
  const int blocks = blocks_of(kv);          // (<= launched, as kv fits the table)
  if (static_cast<int>(cluster_rank()) >= blocks) return;      // (a cluster's barrier is of the threads that are left)
  if (blocks == 1)
    select_short(p, item, kv, s_key, room);
  else
    select_item<false, kWideThreads>(p, item, kv, blocks, s_key, room);
}

__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const __grid_constant__ EvictParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const EvictLaunch& a = p.a;
  const int chunks = (a.keep + kCopyRows - 1) / kCopyRows;
  const int item = blockIdx.x / chunks, chunk = blockIdx.x % chunks;
  const int h = item % a.Hkv, b = item / a.Hkv % a.B, l = item / a.Hkv / a.B;
  const int m = min(min(max(0, a.kv_len[b]), a.width << a.page_shift), a.keep);
  const int mask = (1 << a.page_shift) - 1, pieces = a.row_bytes / 16;
  const int* from = a.table + static_cast<size_t>(b) * a.width;
  const int* to = a.out_table + static_cast<size_t>(b) * a.out_width;
  const int* kept = a.kept + static_cast<size_t>(item) * a.keep;
  const uint8_t* K = static_cast<const uint8_t*>(a.K) + a.layer_bytes * l;
  const uint8_t* V = static_cast<const uint8_t*>(a.V) + a.layer_bytes * l;
  const size_t w_layer = static_cast<size_t>(l) * a.num_pages * a.Hkv << a.page_shift;
  const int lanes = pieces, per = kCopyThreads / lanes;
  const int sub = threadIdx.x / lanes, piece = threadIdx.x % lanes;
  for (int i = chunk * kCopyRows + sub; i < min(m, (chunk + 1) * kCopyRows); i += per) {
    const int t = __ldcg(kept + i);
    const int sp = paged_lookup(from, a.width, a.page_shift, a.num_pages, t);
    const int dp = paged_lookup(to, a.out_width, a.page_shift, a.num_pages, i);
    if (sp < 0 || dp < 0) {
      if (piece == 0) atomicOr(p.status, kStatusBadPage);
      continue;
    }
    const size_t src = ((static_cast<size_t>(sp) * a.Hkv + h) << a.page_shift) + (t & mask);
    const size_t dst = ((static_cast<size_t>(dp) * a.Hkv + h) << a.page_shift) + (i & mask);
    const uint4 k = *reinterpret_cast<const uint4*>(K + src * a.row_bytes + piece * 16);
    const uint4 v = *reinterpret_cast<const uint4*>(V + src * a.row_bytes + piece * 16);
    *reinterpret_cast<uint4*>(const_cast<uint8_t*>(K) + dst * a.row_bytes + piece * 16) = k;
    *reinterpret_cast<uint4*>(const_cast<uint8_t*>(V) + dst * a.row_bytes + piece * 16) = v;
    if (piece == 0) a.W[w_layer + dst] = a.W[w_layer + src];
  }
}

}  // namespace

cudaError_t launch_evict(const EvictLaunch& a, const DeviceInfo& dev, cudaStream_t stream) {
  EvictParams p = {a, dev.status_word};
  const long long items = static_cast<long long>(a.nl) * a.B * a.Hkv;
  const long long cap = static_cast<long long>(a.width) << a.page_shift;
  const int blocks = blocks_of(cap);
  const bool small = blocks == 1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(blocks);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.stream = stream;
  cfg.attrs = attr;
  cudaError_t e = cudaSuccess;
  if (small) {
    cfg.gridDim = dim3(static_cast<unsigned>(items));
    cfg.blockDim = dim3(kSmallThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(cap) * 4;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p, static_cast<int>(cap));
  } else {
    static SmemOnce once;
    if ((e = allow_smem(evict_select_wide_kernel, kMaxRoom * 4, dev.device, &once)) != cudaSuccess) return e;
    // (Sequences may be short in a wide table: what room costs is blocks an SM, of those too that leave at once.)
    const long long want = std::max((cap + blocks - 1) / blocks + 32, static_cast<long long>(kShort));
    const int room = static_cast<int>(std::min<long long>(want, items * blocks <= dev.num_sms ? kMaxRoom : kSharedRoom));
    cfg.gridDim = dim3(static_cast<unsigned>(items * blocks));
    cfg.blockDim = dim3(kWideThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(room) * 4;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, evict_select_wide_kernel, p, blocks, room);
  }
  if (e != cudaSuccess) return e;
  count_launches(1);
  cfg.gridDim = dim3(static_cast<unsigned>(items * ((a.keep + kCopyRows - 1) / kCopyRows)));
  cfg.blockDim = dim3(kCopyThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, evict_copy_kernel, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace cxa
