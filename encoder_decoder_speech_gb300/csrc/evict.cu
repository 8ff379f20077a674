// Eviction from a paged cache by gathered attention weight.
//
// evict_select_kernel finds, for every (layer, sequence, K/V head), the keep heaviest positions (the
// first and the last ones before all others) and lists them in order. A cluster of up to 8 blocks has the
// item's keys (weights as integers in their order) in shared memory, read once; three passes over their digits
// of 11, 11 and 10 bits, histograms added up over distributed shared memory, find the keep-th largest; one more
// writes the positions above it, and of those equal to it the first ones. (A block an item, which read the
// weights anew in each pass: 225 us for 32 lists of 65536.) evict_copy_kernel copies the listed rows of K, V and
// weights, a block 64 of them. Bound by memory: weights are read once, what stays is read and written once.
#include "cluster.cuh"
#include "latent.cuh"
#include "ptx.cuh"

namespace cxa {
namespace {

constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;
constexpr int kMaxRoom = 49152;      // keys in a block's shared memory; more are read again
constexpr int kCopyThreads = 256, kCopyRows = 64;

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

template <int kThreads>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(const __grid_constant__ EvictParams p, int blocks, int room) {
  constexpr int kWarps = kThreads / 32;
  extern __shared__ uint32_t s_key[];        // [room]
  __shared__ int s_hist[kBins], s_sum[kBins];      // of this block; of its share of the bins, over the cluster
  __shared__ int s_group[32];                      // of 32 groups of the share's bins
  __shared__ int s_scan[2][kWarps];
  __shared__ int s_count[2];
  __shared__ uint32_t s_prefix;
  __shared__ int s_left;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const EvictLaunch& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = blocks > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int item = blockIdx.x / blocks, h = item % a.Hkv, b = item / a.Hkv % a.B, l = item / a.Hkv / a.B;
  const int cap = a.width << a.page_shift;
  const int given = max(0, a.kv_len[b]), kv = min(given, cap), m = min(kv, a.keep);
  if (tid == 0 && rank == 0 && given > cap) atomicOr(p.status, kStatusBadPage);
  if (l == 0 && h == 0 && tid == 0 && rank == 0) a.out_len[b] = m;
  int* kept = a.kept + static_cast<size_t>(item) * a.keep;
  for (int i = m + rank * kThreads + tid; i < a.keep; i += blocks * kThreads) kept[i] = -1;
  if (m == kv) {        // (the same in the whole cluster)
    for (int i = rank * kThreads + tid; i < m; i += blocks * kThreads) kept[i] = i;
    return;
  }
  auto all_sync = [&]() {
    if (blocks > 1)
      cluster_sync();
    else
      __syncthreads();
  };
  auto remote = [&](const int* x, int r) { return blocks > 1 ? ld_cluster(x, static_cast<uint32_t>(r)) : *x; };
  const int* row = a.table + static_cast<size_t>(b) * a.width;
  const float* W = a.W + (static_cast<size_t>(l) * a.num_pages * a.Hkv << a.page_shift);
  auto key_of = [&](int t) {
    const bool stays = t < a.first || t >= kv - a.recent;
    float w = 0.f;
    if (!stays) {
      const int page = paged_lookup(row, a.width, a.page_shift, a.num_pages, t);
      if (page < 0) atomicOr(p.status, kStatusBadPage);
      w = page < 0 ? 0.f : __ldg(W + ((static_cast<size_t>(page) * a.Hkv + h) << a.page_shift) + (t & ((1 << a.page_shift) - 1)));
    }
    return order_key(w, stays);
  };
  // this block's positions [lo, lo + n)
  const int per = ((kv + blocks - 1) / blocks + 31) / 32 * 32;
  const int lo = min(kv, rank * per), n = min(kv, lo + per) - lo;
#pragma unroll 4
  for (int i = tid; i < min(n, room); i += kThreads) s_key[i] = key_of(lo + i);
  auto key = [&](int i) { return i < room ? s_key[i] : key_of(lo + i); };
  uint32_t prefix = 0;
  int left = m;               // to be taken among the keys that share the prefix
  const int share = kBins / blocks;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, top = pass == 0 ? 32 : pass == 1 ? 21 : 10;
    for (int i = tid; i < kBins; i += kThreads) s_hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const uint32_t k = key(i);
      if (pass == 0 || (k >> top) == (prefix >> top)) atomicAdd(&s_hist[(k >> shift) & ((1u << (top - shift)) - 1u)], 1);
    }
    all_sync();
    const int each = share / 32;      // bins of a group: 8 to 64
    for (int i = tid; i < share; i += kThreads) {
      int sum = 0;
      for (int c = 0; c < blocks; ++c) sum += remote(&s_hist[rank * share + i], c);
      s_sum[i] = sum;
    }
    __syncthreads();
    for (int g = warp; g < 32; g += kWarps) {
      int sum = (lane < each ? s_sum[g * each + lane] : 0) + (lane + 32 < each ? s_sum[g * each + lane + 32] : 0);
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      if (lane == 0) s_group[g] = sum;
    }
    __syncthreads();
    if (warp == 0) {
      int sum = s_group[lane];
#pragma unroll
      for (int off = 16; off >= 1; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
      if (lane == 0) s_count[0] = sum;
    }
    all_sync();
    if (warp == 0) {
      // the share, the group in it and the bin in that, in which the count from above reaches `left`
      int above = 0;
      auto find = [&](int c) {      // a lane's count; the lane, `above` then counts what is above it
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
      const int at = find(lane < blocks ? remote(&s_count[0], lane) : 0);
      const int group = find(remote(&s_group[lane], at));
      const int two = each == 64 ? 2 : 1, first = group * each + lane * two;      // of this lane's bins
      const bool has = lane * two < each;
      const int c0 = has ? remote(&s_sum[first], at) : 0, c1 = has && two == 2 ? remote(&s_sum[first + 1], at) : 0;
      const int in = find(c0 + c1);
      if (lane == in) {
        const bool upper = two == 2 && above + c1 >= left;
        const int bin = first + (upper ? 1 : 0);
        s_prefix = prefix | static_cast<uint32_t>(at * share + bin) << shift;
        s_left = left - (above + (two == 2 && !upper ? c1 : 0));
      }
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_left;
    __syncthreads();
  }
  // prefix is the m-th largest key; `left` of the positions that have it stay
  int counts[2] = {0, 0};
  for (int i = tid; i < n; i += kThreads) {
    const uint32_t k = key(i);
    counts[0] += k > prefix ? 1 : 0;
    counts[1] += k == prefix ? 1 : 0;
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) counts[q] += __shfl_xor_sync(0xffffffffu, counts[q], off);
    if (lane == 0) s_scan[q][warp] = counts[q];
  }
  __syncthreads();
  if (tid < 2) {
    int sum = 0;
    for (int i = 0; i < kWarps; ++i) sum += s_scan[tid][i];
    s_count[tid] = sum;
  }
  all_sync();
  int out = 0, ties = 0;      // in the positions before
  for (int c = 0; c < rank; ++c) {
    out += remote(&s_count[0], c);
    ties += remote(&s_count[1], c);
  }
  out += min(ties, left);
  for (int i0 = 0; i0 < n; i0 += kThreads) {
    const int i = i0 + tid;
    const uint32_t k = i < n ? key(i) : 0u;
    const bool above = i < n && k > prefix, tie = i < n && k == prefix;
    const uint32_t ma = __ballot_sync(0xffffffffu, above), mt = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) {
      s_scan[0][warp] = __popc(ma);
      s_scan[1][warp] = __popc(mt);
    }
    __syncthreads();
    int na = 0, nt = 0, ba = 0, bt = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        ba += s_scan[0][w];
        bt += s_scan[1][w];
      }
      na += s_scan[0][w];
      nt += s_scan[1][w];
    }
    const uint32_t below = (1u << lane) - 1u;
    const int my_above = ba + __popc(ma & below), my_tie = ties + bt + __popc(mt & below);
    // ties before this position, of those that stay
    const int at = out + my_above + (min(my_tie, left) - min(ties, left));
    if (above || (tie && my_tie < left)) kept[at] = lo + i;
    out += na + (min(ties + nt, left) - min(ties, left));
    ties += nt;
    __syncthreads();
  }
  if (blocks > 1) cluster_sync();      // no block leaves while another may read its counts
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
  // blocks of 2048 positions and more, up to 8 an item
  int blocks = 1;
  while (blocks < kMaxCluster && cap / blocks > 4096) blocks *= 2;
  const long long want = (cap + blocks - 1) / blocks + 32;
  const int room = static_cast<int>(want < kMaxRoom ? want : kMaxRoom);
  const bool small = blocks == 1;
  cudaError_t e = cudaSuccess;
  static SmemOnce once;
  if (!small && (e = allow_smem(evict_select_kernel<1024>, kMaxRoom * 4, dev.device, &once)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items * blocks));
  cfg.blockDim = dim3(small ? 256 : 1024);
  cfg.dynamicSmemBytes = static_cast<size_t>(room) * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(blocks);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = small ? 1 : 2;
  e = small ? cudaLaunchKernelEx(&cfg, evict_select_kernel<256>, p, blocks, room)
            : cudaLaunchKernelEx(&cfg, evict_select_kernel<1024>, p, blocks, room);
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
