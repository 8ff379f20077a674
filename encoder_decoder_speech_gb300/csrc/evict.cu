// Eviction from a paged cache by gathered attention weight.
//
// evict_select_kernel finds, for every (layer, sequence, K/V head), the keep heaviest positions (the
// first and the last ones before all others) and lists them in order: the keep-th largest weight bit
// group by bit group from histograms, then one pass that writes the positions above it, and of those
// equal to it the first ones. evict_copy_kernel copies the listed rows of K, V and weights, a block 64
// of them. Bound by memory: weights are read from HBM once (and again from L2), what stays is read and
// written once.
#include "latent.cuh"
#include "ptx.cuh"

namespace cxa {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kBits = 8, kBins = 1 << kBits;
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

__global__ void __launch_bounds__(kThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ int s_hist[kBins];
  __shared__ int s_scan[2][kWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_left;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const EvictLaunch& a = p.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int item = blockIdx.x, h = item % a.Hkv, b = item / a.Hkv % a.B, l = item / a.Hkv / a.B;
  const int cap = a.width << a.page_shift;
  const int given = max(0, a.kv_len[b]), kv = min(given, cap), m = min(kv, a.keep);
  if (tid == 0 && given > cap) atomicOr(p.status, kStatusBadPage);
  if (l == 0 && h == 0 && tid == 0) a.out_len[b] = m;
  int* kept = a.kept + static_cast<size_t>(item) * a.keep;
  for (int i = m + tid; i < a.keep; i += kThreads) kept[i] = -1;
  if (m == kv) {
    for (int i = tid; i < m; i += kThreads) kept[i] = i;
    return;
  }
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
  uint32_t prefix = 0;
  int left = m;               // to be taken among the keys that share the prefix
  for (int shift = 32 - kBits; shift >= 0; shift -= kBits) {
    if (tid < kBins) s_hist[tid] = 0;
    __syncthreads();
    for (int t = tid; t < kv; t += kThreads) {
      const uint32_t k = key_of(t);
      if (shift == 32 - kBits || (k >> (shift + kBits)) == (prefix >> (shift + kBits)))
        atomicAdd(&s_hist[(k >> shift) & (kBins - 1)], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // the bin in which the count from above reaches `left`: lane i has bins 8 i .. 8 i + 7
      int sum = 0;
#pragma unroll
      for (int i = 0; i < kBins / 32; ++i) sum += s_hist[lane * (kBins / 32) + i];
      int above = sum;        // of this lane's bins and those above
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_down_sync(0xffffffffu, above, off);
        if (lane + off < 32) above += o;
      }
      above -= sum;
      if (above < left && above + sum >= left) {
        int bin = (lane + 1) * (kBins / 32) - 1;
        for (int c = s_hist[bin]; above + c < left; c = s_hist[bin]) {
          above += c;
          --bin;
        }
        s_prefix = prefix | static_cast<uint32_t>(bin) << shift;
        s_left = left - above;
      }
    }
    __syncthreads();
    prefix = s_prefix;
    left = s_left;
    __syncthreads();
  }
  // prefix is the m-th largest key; `left` of the positions that have it stay
  int out = 0, ties = 0;      // so far, in all positions before
  for (int t0 = 0; t0 < kv; t0 += kThreads) {
    const int t = t0 + tid;
    const uint32_t k = t < kv ? key_of(t) : 0u;
    const bool above = t < kv && k > prefix, tie = t < kv && k == prefix;
    const uint32_t ma = __ballot_sync(0xffffffffu, above), mt = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) {
      s_scan[0][warp] = __popc(ma);
      s_scan[1][warp] = __popc(mt);
    }
    __syncthreads();
    int na = 0, nt = 0, ba = 0, bt = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) {
        ba += s_scan[0][i];
        bt += s_scan[1][i];
      }
      na += s_scan[0][i];
      nt += s_scan[1][i];
    }
    const uint32_t below = (1u << lane) - 1u;
    const int my_above = ba + __popc(ma & below), my_tie = ties + bt + __popc(mt & below);
    // ties before this position, of those that stay
    const int at = out + my_above + (min(my_tie, left) - min(ties, left));
    if (above || (tie && my_tie < left)) kept[at] = t;
    out += na + (min(ties + nt, left) - min(ties, left));
    ties += nt;
    __syncthreads();
  }
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
  cudaLaunchConfig_t cfg = {};
  const long long items = static_cast<long long>(a.nl) * a.B * a.Hkv;
  cfg.gridDim = dim3(static_cast<unsigned>(items));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p);
  if (e != cudaSuccess) return e;
  count_launches(1);
  cfg.gridDim = dim3(static_cast<unsigned>(items * ((a.keep + kCopyRows - 1) / kCopyRows)));
  cfg.blockDim = dim3(kCopyThreads);
  e = cudaLaunchKernelEx(&cfg, evict_copy_kernel, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace cxa
