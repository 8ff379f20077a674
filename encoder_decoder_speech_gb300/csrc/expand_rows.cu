// The expansion of latent rows into pages of keys and values in fp32, on the CUDA cores:
//
//   K_h(t) = [ r_t | c_t WK_h ],  V_h(t) = c_t WV_h
//
// as one product of positions by the columns of all heads' WK and WV side by side, in tiles of 64 x 128
// with 4 x 8 sums a thread, 16 latent channels at a time, the next ones under way meanwhile. Bound by the
// products: 2 latent operations a value. 8 sequences of up to 1000 positions, 8 heads of 64, 512 + 48 channels: 117 us,
// 26 TFLOP/s (tiles of 64 x 64 with the loads in the way of the products: 14; of 128 x 128: 26, and 16 against 27
// where that leaves too few of them).
#include "expand.cuh"
#include "ptx.cuh"
#include "span_work.cuh"

namespace cxa {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 64, kCols = 128, kStep = 16;

struct ExpandParams {
  LatentExpandLaunch a;
  unsigned int* status;
};

__global__ void __launch_bounds__(kThreads) expand_rows_kernel(const __grid_constant__ ExpandParams p) {
  __shared__ SpanScratch s_span;
  __shared__ __align__(16) float s_a[2][kStep][kTile + 4], s_b[2][kStep][kCols];
  __shared__ long long s_src[kTile], s_dst[kTile];      // rows of the pools, -1: none
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const LatentExpandLaunch& a = p.a;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int H = a.to.Hkv, dh = a.dh, rope = a.layer.rope, dc = a.layer.latent, width = dc + rope, nope = dh - rope;
  const int cap = a.width << a.layer.page_shift, to_cap = a.to_width << a.to.page_shift;
  // columns: WK's, WV's, and the rotated part's copies
  const int kc = H * nope, vc = H * dh;
  const int k_tiles = (kc + kCols - 1) / kCols, col_tiles = k_tiles + (vc + kCols - 1) / kCols;
  auto tiles = [&](int b) {
    const ExpandSpan s = expand_span(a.from, a.kv_len, cap, b);
    return (s.hi - s.lo + kTile - 1) / kTile;
  };
  SpanRange range;
  auto count = [&](int b) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && expand_passes(a.from, a.kv_len, cap, b)) atomicOr(p.status, kStatusBadPage);
    return tiles(b);
  };
  if (!span_locate<kThreads>(a.B, count, &s_span, &range)) return;
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
      const int n0 = (is_v ? ct - k_tiles : ct) * kCols, nc = is_v ? vc : kc;
      const float* W = static_cast<const float*>(is_v ? a.WV : a.WK);
      float acc[4][8] = {};
      // this thread's part of a step: four channels of a position, eight columns of a channel
      const int ar = tid >> 2, ak = (tid & 3) * 4, bk = tid >> 4, bn = (tid & 15) * 8;
      const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
      float4 ra, rb[2];
      auto load = [&](int k0) {
        ra = s_src[ar] >= 0 ? *reinterpret_cast<const float4*>(C + s_src[ar] + k0 + ak) : zero;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          rb[i] = n0 + bn + 4 * i < nc
                      ? __ldg(reinterpret_cast<const float4*>(W + static_cast<size_t>(k0 + bk) * nc + n0 + bn + 4 * i))
                      : zero;
      };
      load(0);
      for (int k0 = 0, st = 0; k0 < dc; k0 += kStep, st ^= 1) {
        s_a[st][ak][ar] = ra.x;
        s_a[st][ak + 1][ar] = ra.y;
        s_a[st][ak + 2][ar] = ra.z;
        s_a[st][ak + 3][ar] = ra.w;
#pragma unroll
        for (int i = 0; i < 2; ++i) *reinterpret_cast<float4*>(&s_b[st][bk][bn + 4 * i]) = rb[i];
        __syncthreads();      // (the other buffer is free: every thread has passed the barrier before)
        if (k0 + kStep < dc) load(k0 + kStep);
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
          const float4 x = *reinterpret_cast<const float4*>(&s_a[st][k][ty * 4]);
          const float xs[4] = {x.x, x.y, x.z, x.w};
          float ys[8];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float4 y = *reinterpret_cast<const float4*>(&s_b[st][k][64 * i + tx * 4]);
            ys[4 * i] = y.x, ys[4 * i + 1] = y.y, ys[4 * i + 2] = y.z, ys[4 * i + 3] = y.w;
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) acc[i][j] = fmaf(xs[i], ys[j], acc[i][j]);
        }
      }
      __syncthreads();      // the buffers have been read
      float* out = static_cast<float*>(is_v ? a.to.V : a.to.K);
      const int each = is_v ? dh : nope, skip = is_v ? 0 : rope;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int n = n0 + 64 * i + tx * 4;      // four columns of one head: heads have multiples of 16
        if (n >= nc) continue;
        const int h = n / each, ch = skip + n % each;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const long long dst = s_dst[ty * 4 + r];
          if (dst >= 0)
            *reinterpret_cast<float4*>(out + (dst + (static_cast<long long>(h) << a.to.page_shift)) * dh + ch) =
                make_float4(acc[r][4 * i], acc[r][4 * i + 1], acc[r][4 * i + 2], acc[r][4 * i + 3]);
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
  cfg.gridDim = dim3(static_cast<unsigned>(dev.num_sms), 8);
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
