// The expansion of latent rows into pages of keys and values in fp32, on the CUDA cores:
//
//   K_h(t) = [ r_t | c_t WK_h ],  V_h(t) = c_t WV_h
//
// as one product of positions by the columns of all heads' WK and WV side by side, in tiles of 64 x 64
// with 4 x 4 sums a thread, 16 latent channels at a time. Bound by the products: 2 latent operations a
// value.
#include "expand.cuh"
#include "ptx.cuh"
#include "span_work.cuh"

namespace cxa {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64, kStep = 16;

struct ExpandParams {
  LatentExpandLaunch a;
  unsigned int* status;
};

__global__ void __launch_bounds__(kThreads) expand_rows_kernel(const __grid_constant__ ExpandParams p) {
  __shared__ SpanScratch s_span;
  __shared__ __align__(16) float s_a[kStep][kTile + 4], s_b[kStep][kTile + 4];
  __shared__ long long s_src[kTile], s_dst[kTile];      // rows of the pools, -1: none
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const LatentExpandLaunch& a = p.a;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int H = a.to.Hkv, dh = a.dh, rope = a.layer.rope, dc = a.layer.latent, width = dc + rope, nope = dh - rope;
  const int cap = a.width << a.layer.page_shift, to_cap = a.to_width << a.to.page_shift;
  // columns: WK's, WV's, and the rotated part's copies
  const int kc = H * nope, vc = H * dh;
  const int col_tiles = (kc + kTile - 1) / kTile + (vc + kTile - 1) / kTile, k_tiles = (kc + kTile - 1) / kTile;
  auto tiles = [&](int b) {
    const ExpandSpan s = expand_span(a.from, a.kv_len, cap, b);
    return (s.hi - s.lo + kTile - 1) / kTile;
  };
  SpanRange range;
  if (!span_locate<kThreads>(a.B, tiles, &s_span, &range)) return;
  int b = range.b, first = range.first;
  for (int g = range.g0; g < range.g1; ++g) {
    while (g - first >= tiles(b)) first += tiles(b++);
    const ExpandSpan span = expand_span(a.from, a.kv_len, cap, b);
    const int t0 = span.lo + (g - first) * kTile;
    __syncthreads();
    if (tid < kTile) {
      const int t = t0 + tid;
      long long src = -1, dst = -1;
      if (t < span.hi) {
        const int sp = paged_lookup(a.table + static_cast<size_t>(b) * a.width, a.width, a.layer.page_shift,
                                    a.layer.num_pages, t);
        const int dp = paged_lookup(a.to_table + static_cast<size_t>(b) * a.to_width, a.to_width, a.to.page_shift,
                                    a.to.num_pages, t < to_cap ? t : -1);
        if (sp < 0 || dp < 0) {
          atomicOr(p.status, kStatusBadPage);
        } else {
          src = ((static_cast<long long>(sp) << a.layer.page_shift) + (t & ((1 << a.layer.page_shift) - 1))) * width;
          dst = ((static_cast<long long>(dp) * H) << a.to.page_shift) + (t & ((1 << a.to.page_shift) - 1));
        }
      }
      s_src[tid] = src;
      s_dst[tid] = dst;
    }
    __syncthreads();
    const float* C = static_cast<const float*>(a.layer.C);
    for (int ct = blockIdx.y; ct < col_tiles; ct += gridDim.y) {
      const bool is_v = ct >= k_tiles;
      const int n0 = (is_v ? ct - k_tiles : ct) * kTile, nc = is_v ? vc : kc;
      const float* W = static_cast<const float*>(is_v ? a.WV : a.WK);
      float acc[4][4] = {};
      for (int k0 = 0; k0 < dc; k0 += kStep) {
        __syncthreads();
        for (int i = tid; i < kTile * kStep; i += kThreads) {
          const int r = i / kStep, k = i % kStep;
          s_a[k][r] = s_src[r] >= 0 ? C[s_src[r] + k0 + k] : 0.f;
          const int kk = i / kTile, n = i % kTile;
          s_b[kk][n] = n0 + n < nc ? W[static_cast<size_t>(k0 + kk) * nc + n0 + n] : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
          const float4 x = *reinterpret_cast<const float4*>(&s_a[k][ty * 4]);
          const float4 y = *reinterpret_cast<const float4*>(&s_b[k][tx * 4]);
          const float xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xs[i], ys[j], acc[i][j]);
        }
      }
      float* out = static_cast<float*>(is_v ? a.to.V : a.to.K);
      const int each = is_v ? dh : nope, skip = is_v ? 0 : rope;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx * 4 + j;
        if (n >= nc) continue;
        const int h = n / each, ch = skip + n % each;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const long long dst = s_dst[ty * 4 + i];
          if (dst >= 0) out[(dst + (static_cast<long long>(h) << a.to.page_shift)) * dh + ch] = acc[i][j];
        }
      }
    }
    // the rotated part, the same in every head
    if (rope > 0 && blockIdx.y == 0)
      for (int i = tid; i < kTile * rope; i += kThreads) {
        const int r = i / rope, ch = i % rope;
        if (s_dst[r] < 0) continue;
        const float x = C[s_src[r] + dc + ch];
        for (int h = 0; h < H; ++h)
          static_cast<float*>(a.to.K)[(s_dst[r] + (static_cast<long long>(h) << a.to.page_shift)) * dh + ch] = x;
      }
  }
}

}  // namespace

cudaError_t launch_expand_rows(const LatentExpandLaunch& a, const DeviceInfo& dev, cudaStream_t stream) {
  ExpandParams p = {a, dev.status_word};
  cudaLaunchConfig_t cfg = {};
  // the blocks of a column go over all positions, those of a row over all columns
  cfg.gridDim = dim3(static_cast<unsigned>(dev.num_sms), 4);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, expand_rows_kernel, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace cxa
