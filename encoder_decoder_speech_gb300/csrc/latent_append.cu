// The append to a latent cache: new tokens' latent vectors, RMS-normalised, and their rotated parts
// into rows of their pages.
//
//   row(t) = [ c_t * rsqrt(mean(c_t^2) + eps) * w  |  R(position) kr_t ]
//
// Bound by memory, each value read once and written once; a step of 16 tokens by the latency of
// three dependent reads (sequence, page, row). A warp takes one token: it has the whole row under way
// before it looks up where the row goes, holds it in registers, adds the squares up across its lanes
// and writes. The rotated part is a pair a lane. 16,391 tokens of 512 + 64 channels, bf16: 12.6 us, 3.0 TB/s on tensors
// that L2 holds in part; 16 tokens: 8 us a call, the host's.
#include <cuda_bf16.h>

#include "latent.cuh"
#include "paged_find.cuh"
#include "ptx.cuh"

namespace cxa {
namespace {

constexpr int kWarps = 4;

struct AppendParams {
  const void *c, *kr;
  long long c_stride, kr_stride;
  const float* weight;
  float eps;
  int norm, wide;             // wide: the weights are 16-byte aligned
  unsigned int* status;
  PagedBatch batch;
  LatentLayer layer;
  RotaryArg rot;
};

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}
__device__ __forceinline__ void store4(float* p, const float4& v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float4& v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  uint2 u;
  u.x = *reinterpret_cast<const uint32_t*>(&a);
  u.y = *reinterpret_cast<const uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = u;
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

template <typename TA, typename TP>
__global__ void __launch_bounds__(kWarps * 32) latent_append_kernel(const __grid_constant__ AppendParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const long long at = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (at >= p.batch.n_tokens) return;
  const int token = static_cast<int>(at);
  const int dc = p.layer.latent, dr = p.layer.rope, quads = dc / 128, pairs = p.rot.pairs;

  // the row on its way
  const TA* c = static_cast<const TA*>(p.c) + token * p.c_stride;
  const TA* kr = static_cast<const TA*>(p.kr) + token * p.kr_stride;
  float4 x[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < quads) x[j] = load4(c + j * 128 + lane * 4);
  // lane i: pair i of the rotated part; channels that do not turn: 2 * pairs + lane, + 32
  const int lo = p.rot.interleaved ? 2 * lane : lane, hi = p.rot.interleaved ? 2 * lane + 1 : lane + pairs;
  const int e0 = 2 * pairs + lane, e1 = e0 + 32;
  float a = 0.f, b = 0.f, s0 = 0.f, s1 = 0.f;
  if (lane < pairs) {
    a = to_f(kr[lo]);
    b = to_f(kr[hi]);
  }
  if (e0 < dr) s0 = to_f(kr[e0]);
  if (e1 < dr) s1 = to_f(kr[e1]);

  float4 g[4];      // weights
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    g[j] = make_float4(1.f, 1.f, 1.f, 1.f);
    if (j < quads && p.norm && p.weight != nullptr) {
      const float* from = p.weight + j * 128 + lane * 4;
      g[j] = p.wide ? __ldg(reinterpret_cast<const float4*>(from))
                    : make_float4(__ldg(from), __ldg(from + 1), __ldg(from + 2), __ldg(from + 3));
    }
  }

  const int seq = find_seq(p.batch.q_start, p.batch.B, token, lane);
  if (seq < 0) return;
  const PagedSeq s = paged_seq(p.batch.q_start, p.batch.kv_len, seq, p.batch.n_tokens);
  if (token - s.q0 >= s.n) return;          // a row behind the last sequence
  const int pos = s.kv - s.n + (token - s.q0);
  if (pos < 0) return;
  const int page = paged_lookup(p.batch.table + static_cast<size_t>(seq) * p.batch.width, p.batch.width,
                                p.layer.page_shift, p.layer.num_pages, pos);
  if (page < 0) {
    if (lane == 0) atomicOr(p.status, kStatusBadPage);
    return;
  }
  TP* row = static_cast<TP*>(p.layer.C) +
            ((static_cast<long long>(page) << p.layer.page_shift) + (pos & ((1 << p.layer.page_shift) - 1))) * (dc + dr);
  float r = 1.f;
  if (p.norm) {
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < quads) sq += x[j].x * x[j].x + x[j].y * x[j].y + x[j].z * x[j].z + x[j].w * x[j].w;
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, off);
    r = rsqrtf(sq / static_cast<float>(dc) + p.eps);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < quads)
      store4(row + j * 128 + lane * 4,
             make_float4(x[j].x * r * g[j].x, x[j].y * r * g[j].y, x[j].z * r * g[j].z, x[j].w * r * g[j].w));
  if (lane < pairs) {
    const unsigned long long ph = static_cast<unsigned long long>(static_cast<long long>(pos)) * p.rot.step[lane];
    float sn, cs;
    // half turns in [-1, 1); the 32 high bits of the phase are finer than fp32 holds
    sincospif(static_cast<float>(static_cast<int>(ph >> 32)) * 4.6566128730773926e-10f, &sn, &cs);
    cs *= p.rot.factor;
    sn *= p.rot.factor;
    put(row + dc + lo, a * cs - b * sn);
    put(row + dc + hi, a * sn + b * cs);
  }
  if (e0 < dr) put(row + dc + e0, s0);
  if (e1 < dr) put(row + dc + e1, s1);
}

template <typename TA, typename TP>
cudaError_t launch(const LatentAppendLaunch& a, const DeviceInfo& dev, cudaStream_t stream) {
  AppendParams p;
  p.c = a.c;
  p.kr = a.kr;
  p.c_stride = a.c_stride;
  p.kr_stride = a.kr_stride;
  p.weight = a.weight;
  p.eps = a.eps;
  p.norm = a.norm ? 1 : 0;
  p.wide = reinterpret_cast<uintptr_t>(a.weight) % 16 == 0 ? 1 : 0;
  p.status = dev.status_word;
  p.batch = a.batch;
  p.layer = a.layer;
  p.rot = a.rot;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((static_cast<long long>(a.batch.n_tokens) + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, latent_append_kernel<TA, TP>, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace

cudaError_t launch_latent_append(const LatentAppendLaunch& a, const DeviceInfo& dev, cudaStream_t stream) {
  using bf = __nv_bfloat16;
  if (a.act_bf16) return launch<bf, bf>(a, dev, stream);
  return a.pool_bf16 ? launch<float, bf>(a, dev, stream) : launch<float, float>(a, dev, stream);
}

}  // namespace cxa
