// The merge of the latent attention's cut items: out = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k
// over an item's parts k, for every row. The parts were written a moment ago and lie in L2; bound by
// the latency of reading them. A unit is a warp's row where parts are few (a batch), a block's 128 channels of
// a row where they are many (one long context).
#include <cuda_bf16.h>

#include "latent_parts.cuh"
#include "ptx.cuh"

namespace cxa {
namespace {

constexpr int kThreads = 320, kWarps = kThreads / 32;
static_assert(kThreads >= kLatentMaxBlocks, "a thread a block's item, and a part");
constexpr int kWarpParts = 16;     // parts that a warp merges by itself

struct MergeParams {
  const LatentCut* cut;
  const float* part;
  void* out;
  long long o_stride;
  int blocks, R, latent, H;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void store4(float* p, const float4& v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float4& v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  uint2 u;
  u.x = *reinterpret_cast<const uint32_t*>(&a);
  u.y = *reinterpret_cast<const uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = u;
}
__device__ __forceinline__ float4 fma4(float f, const float4& v, const float4& a) {
  return make_float4(fmaf(f, v.x, a.x), fmaf(f, v.y, a.y), fmaf(f, v.z, a.z), fmaf(f, v.w, a.w));
}

template <typename TO>
__global__ void __launch_bounds__(kThreads) latent_merge_kernel(const __grid_constant__ MergeParams p) {
  __shared__ LatentCut s_cut[kLatentMaxBlocks];
  __shared__ int s_end[2][kThreads];          // ends of the items' units: of few parts, of many
  __shared__ unsigned long long s_warp[kWarps];
  __shared__ float s_w[kLatentMaxBlocks];
  __shared__ float s_red[2][kWarps];
  __shared__ float4 s_acc[kWarps][32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cols = p.latent / 128;
  const size_t slot = latent_slot(p.R, p.latent);
  int few = 0, many = 0;
  if (tid < p.blocks) {
    const int4 v = __ldcg(reinterpret_cast<const int4*>(p.cut) + tid);
    const LatentCut c = {v.x, v.y, v.z, v.w};
    s_cut[tid] = c;
    if (c.parts > kWarpParts)
      many = c.rows * cols;
    else if (c.parts > 0)
      few = c.rows;
  }
  // both kinds' counts summed up to each item in one number, 32 bits of each
  unsigned long long sum = static_cast<unsigned long long>(many) << 32 | static_cast<unsigned>(few);
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const unsigned long long o = __shfl_up_sync(0xffffffffu, sum, off);
    if (lane >= off) sum += o;
  }
  if (lane == 31) s_warp[warp] = sum;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWarps; ++i)
    if (i < warp) sum += s_warp[i];
  s_end[0][tid] = static_cast<int>(sum & 0xFFFFFFFFu);
  s_end[1][tid] = static_cast<int>(sum >> 32);
  __syncthreads();
  // the item that holds unit u, and the unit's number in it
  auto find = [&](int k, int u, int* in) {
    int lo = 0, hi = p.blocks - 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_end[k][mid] > u) hi = mid; else lo = mid + 1;
    }
    *in = u - (lo > 0 ? s_end[k][lo - 1] : 0);
    return lo;
  };
  auto part = [&](int owner, int k) { return p.part + (2 * static_cast<size_t>(owner + k) + (k == 0 ? 1 : 0)) * slot; };
  auto dst = [&](const LatentCut& c, int row, int col) {
    const int at = c.rt * p.R + row;
    return static_cast<TO*>(p.out) + (c.q0 + at / p.H) * p.o_stride + static_cast<long long>(at % p.H) * p.latent +
           col * 128 + lane * 4;
  };

  for (int u = blockIdx.x; u < s_end[1][kThreads - 1]; u += gridDim.x) {
    int in;
    const int owner = find(1, u, &in), row = in / cols, col = in - row * cols;
    const LatentCut c = s_cut[owner];
    const bool has = tid < c.parts;            // (parts <= blocks <= kThreads)
    const float* ml = part(owner, has ? tid : 0) + static_cast<size_t>(p.R) * p.latent + row;
    const float m = has ? __ldcg(ml) : -INFINITY, l = has ? __ldcg(ml + p.R) : 0.f;
    float M = m;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    if (lane == 0) s_red[0][warp] = M;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWarps; ++i) M = fmaxf(M, s_red[0][i]);
    const float w = m == -INFINITY ? 0.f : ex2(m - M);
    float L = l * w;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
    if (lane == 0) s_red[1][warp] = L;
    if (has) s_w[tid] = w;
    __syncthreads();
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const size_t at = static_cast<size_t>(row) * p.latent + col * 128 + lane * 4;
#pragma unroll 8
    for (int k = warp; k < c.parts; k += kWarps)
      acc = fma4(s_w[k], __ldcg(reinterpret_cast<const float4*>(part(owner, k) + at)), acc);
    s_acc[warp][lane] = acc;
    __syncthreads();
    if (warp == 0) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) sum += s_red[1][i];
#pragma unroll
      for (int i = 1; i < kWarps; ++i) acc = fma4(1.f, s_acc[i][lane], acc);
      const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
      store4(dst(c, row, col), make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
    }
    __syncthreads();
  }
  for (int u = blockIdx.x * kWarps + warp; u < s_end[0][kThreads - 1]; u += gridDim.x * kWarps) {
    int row;
    const int owner = find(0, u, &row);
    const LatentCut c = s_cut[owner];
    const bool has = lane < c.parts;
    const float* ml = part(owner, has ? lane : 0) + static_cast<size_t>(p.R) * p.latent + row;
    const float m = has ? __ldcg(ml) : -INFINITY, l = has ? __ldcg(ml + p.R) : 0.f;
    const size_t at = static_cast<size_t>(row) * p.latent + lane * 4;
    float M = m;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    const float w = m == -INFINITY ? 0.f : ex2(m - M);
    float L = l * w;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
    float4 acc[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
    for (int k = 0; k < c.parts; ++k) {
      const float wk = __shfl_sync(0xffffffffu, w, k);
      const float* src = part(owner, k) + at;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q < cols) acc[q] = fma4(wk, __ldcg(reinterpret_cast<const float4*>(src + q * 128)), acc[q]);
    }
    const float inv = L > 0.f || L != L ? 1.f / L : 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (q < cols)
        store4(dst(c, row, q), make_float4(acc[q].x * inv, acc[q].y * inv, acc[q].z * inv, acc[q].w * inv));
  }
}

}  // namespace

cudaError_t launch_latent_merge(const LatentAttnLaunch& a, int R, int blocks, const DeviceInfo& dev,
                                cudaStream_t stream) {
  MergeParams p;
  p.cut = latent_cuts(a.workspace);
  p.part = latent_part(a.workspace);
  p.out = a.out;
  p.o_stride = a.o_stride;
  p.blocks = blocks;
  p.R = R;
  p.latent = a.layer.latent;
  p.H = a.H;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(dev.num_sms * 4));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = a.bf16 ? cudaLaunchKernelEx(&cfg, latent_merge_kernel<__nv_bfloat16>, p)
                               : cudaLaunchKernelEx(&cfg, latent_merge_kernel<float>, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace cxa
