// Head norms and the position rotation of queries and keys in one pass, and the append
// of new tokens to a paged K/V cache with both applied on the way.
//
//   y = x * rsqrt(mean(x^2) + eps) * w            per head, over its dh channels
//   (a, b) -> f * (a cos t - b sin t, a sin t + b cos t),  t = position * frequency[i]
//
// for the first 2 * pairs channels of the head (pair i is (2i, 2i+1) or (i, i + pairs));
// the rest pass through. Both are linear in x once 1 / rms is known, so a channel of the
// result is rms^-1 * (x * A + partner * B) with A = w f cos t and B = -+ w' f sin t (w' the
// partner's weight): A and B depend on the token and the lane, not on the head, and stay
// in registers over the token's heads. (w f cos t is rounded to fp32 on the way: one rounding
// more than x w first, 4.8e-8 of an fp32 result in all against 3.6e-8.)
//
// Bound by memory: every value is read once and written once. What stands between is kept
// short, or the instructions bind (with 175 of them for 16 bytes a lane: 83 us for 24,000
// tokens of 40 heads, against 45 us now): a lane holds two groups of four channels of a
// head that are each other's partners (the half layout) or hold their partners themselves
// (interleaved), so that no value is fetched from another lane, and works on pairs
// (fma.f32x2). A warp takes one token, with the loads of kBatch heads under way before the
// first is used. The phases are computed once a token, one pair a lane, from a 64-bit
// fixed-point turn (RotaryArg), and handed round through shared memory. With few tokens the
// heads are dealt to several warps.
#include <cuda_bf16.h>

#include <type_traits>

#include "paged.cuh"
#include "ptx.cuh"

namespace cxa {
namespace {

constexpr int kWarps = 4;
constexpr int kBatch = 4;         // heads' loads under way in a lane
// Blocks an SM that the registers are cut to: the append's threads hold more, fp32 loads twice
// the registers. Measured, in us: bf16 without the append (24,000 tokens of 40 heads) 8 blocks
// 45.6, 7 blocks 47.5, 9 blocks 51.3; with it (16,391 tokens) 7 blocks 67.9, 8 blocks 69.7, 9
// blocks 76.7; fp32 without (5,333 tokens of 10 heads) 6 blocks 6.1, 5 blocks 6.7, 7 blocks
// 8.1; with it (1,237 tokens of 6 heads) 5 blocks 3.9, 6 blocks 4.6, 7 blocks 4.9. Half as many
// blocks of 8 warps: 46.9, 71.1, 6.4 and 4.6.
template <typename TA, bool kAppend>
constexpr int kBlocksPerSm = (sizeof(TA) == 2 ? 8 : 6) - (kAppend ? 1 : 0);

struct NrParams {
  const void *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  void *q_out, *k_out;
  long long qo_stride, ko_stride;
  int Hq, Hk, n_tokens, splits;
  const int* pos;
  const float *wq, *wk;
  float eps;
  int norm;
  unsigned int* status;
  PagedBatch batch;
  PagedLayer layer;
  RotaryArg rot;
};

__device__ __forceinline__ float lo_bf16(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&p);
}

// Four channels, as loaded and as pairs of floats.
template <typename T>
struct Quad;
template <>
struct Quad<float> {
  using Raw = uint4;
  __device__ static void unpack(const Raw& u, float2 (&x)[2]) {
    x[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    x[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
};
template <>
struct Quad<__nv_bfloat16> {
  using Raw = uint2;
  __device__ static void unpack(const Raw& u, float2 (&x)[2]) {
    x[0] = make_float2(lo_bf16(u.x), hi_bf16(u.x));
    x[1] = make_float2(lo_bf16(u.y), hi_bf16(u.y));
  }
};
__device__ __forceinline__ void store_quad(float* p, const float2 (&y)[2]) {
  *reinterpret_cast<float4*>(p) = make_float4(y[0].x, y[0].y, y[1].x, y[1].y);
}
__device__ __forceinline__ void store_quad(__nv_bfloat16* p, const float2 (&y)[2]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(y[0].x, y[0].y), pack_bf16(y[1].x, y[1].y));
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)),
        "l"(reinterpret_cast<unsigned long long&>(c)));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<unsigned long long&>(d))
      : "l"(reinterpret_cast<unsigned long long&>(a)), "l"(reinterpret_cast<unsigned long long&>(b)));
  return d;
}
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// The sequence whose rows hold token t, by the whole warp: the last b with
// q_start[b] <= t, 32 candidates a step. -1 if t lies before the first row.
__device__ __forceinline__ int find_seq(const int* q_start, int B, int t, int lane) {
  int lo = 0, len = B;   // the answer, if any, lies in [lo, lo + len)
  if (__ldg(q_start) > t) return -1;
  while (len > 1) {
    const int step = (len + 31) / 32;
    const int at = lane * step;
    const unsigned m = __ballot_sync(0xffffffffu, at < len && __ldg(q_start + lo + min(at, len - 1)) <= t);
    const int last = 31 - __clz(m | 1u);
    lo += last * step;
    len = min(step, len - last * step);
  }
  return lo;
}

// How a lane's two groups of channels turn: the groups are partners; each holds its own
// partners, or is not turned; or (pairs that do not fill groups) partners lie anywhere.
enum Mode { kPartners = 0, kInside = 1, kAnywhere = 2 };

template <typename TA, typename TP, int kDh, bool kAppend, int kMode>
__global__ void __launch_bounds__(kWarps * 32, kBlocksPerSm<TA, kAppend>) norm_rope_kernel(const __grid_constant__ NrParams p) {
  using Raw = typename Quad<TA>::Raw;
  constexpr int LPH = kDh / 8;             // lanes a head
  constexpr int HPI = 32 / LPH;            // heads a warp reads at once
  __shared__ float s_w[2][kDh];            // weights of q and k
  __shared__ __align__(16) float s_cos[kWarps][kDh / 2], s_sin[kWarps][kDh / 2];   // times f, of the token's pairs

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = lane / LPH, li = lane % LPH;
  const int pairs = p.rot.pairs;
  // first channels of the lane's groups
  const bool turns = kMode == kPartners ? li < pairs / 4 : true;
  const int ca = kMode == kPartners && turns ? 4 * li : kMode == kPartners ? 2 * pairs + 8 * (li - pairs / 4) : 8 * li;
  const int cb = kMode == kPartners && turns ? ca + pairs : ca + 4;
  if (p.norm) {
    for (int i = threadIdx.x; i < 2 * kDh; i += kWarps * 32) {
      const float* w = i < kDh ? p.wq : p.wk;
      s_w[i / kDh][i % kDh] = w != nullptr ? __ldg(w + i % kDh) : 1.f;
    }
    __syncthreads();
  }

  const long long item = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const long long tok_ll = item / p.splits;
  if (tok_ll >= p.n_tokens) return;
  const int token = static_cast<int>(tok_ll), part = static_cast<int>(item - tok_ll * p.splits);
  const int itq = (p.Hq + HPI - 1) / HPI, itk = (p.Hk + HPI - 1) / HPI;
  const int iters = itq + itk * (kAppend ? 2 : 1);
  const int per = (iters + p.splits - 1) / p.splits;
  const int it0 = part * per, it1 = min(iters, it0 + per);
  if (it0 >= it1) return;

  int pos = 0;
  bool write_kv = false;
  long long kv_row = 0;   // of head 0 in the page; heads are page_size rows apart
  if constexpr (kAppend) {
    const int b = find_seq(p.batch.q_start, p.batch.B, token, lane);
    if (b < 0) return;
    const PagedSeq s = paged_seq(p.batch.q_start, p.batch.kv_len, b, p.n_tokens);
    if (token - s.q0 >= s.n) return;      // a row behind the last sequence
    pos = s.kv - s.n + (token - s.q0);
    if (it1 > itq && pos >= 0) {
      const int page = paged_lookup(p.batch.table + static_cast<size_t>(b) * p.batch.width, p.batch.width,
                                    p.layer.page_shift, p.layer.num_pages, pos);
      write_kv = page >= 0;
      if (!write_kv && lane == 0) atomicOr(p.status, kStatusBadPage);
      kv_row = ((static_cast<long long>(max(page, 0)) * p.layer.Hkv) << p.layer.page_shift) +
               (pos & ((1 << p.layer.page_shift) - 1));
    }
  } else {
    pos = __ldg(p.pos + token);
  }

  bool have_phases = false;
  auto phases = [&]() {
    have_phases = true;
    for (int i = lane; i < pairs; i += 32) {
      const unsigned long long ph = static_cast<unsigned long long>(static_cast<long long>(pos)) * p.rot.step[i];
      float sn, cs;
      // half turns in [-1, 1); the 32 high bits of the phase are finer than fp32 holds
      sincospif(static_cast<float>(static_cast<int>(ph >> 32)) * 4.6566128730773926e-10f, &sn, &cs);
      s_cos[warp][i] = cs * p.rot.factor;
      s_sin[warp][i] = sn * p.rot.factor;
    }
    __syncwarp();
  };

  // Iterations [i0, i1) of one tensor: head h = it * HPI + sub from src, to dst + h * hop.
  auto heads = [&](auto kind, const TA* src, int i0, int i1, int H, auto* dst, long long hop) {
    constexpr int kKind = decltype(kind)::value;     // q, k, v
    float2 A[4], B[4];      // y = x A + partner B of the lane's channels: two pairs a group
    int h0 = i0 * HPI + sub;
    src += static_cast<long long>(h0) * kDh;
    dst += h0 * hop;
    for (int it = i0; it < i1; it += kBatch) {
      Raw ra[kBatch], rb[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        ra[u] = Raw{};
        rb[u] = Raw{};
        if (it + u < i1 && h0 + u * HPI < H) {
          ra[u] = *reinterpret_cast<const Raw*>(src + u * HPI * kDh + ca);
          rb[u] = *reinterpret_cast<const Raw*>(src + u * HPI * kDh + cb);
        }
      }
      if (kKind < 2 && it == i0) {
        if (!have_phases) phases();
        float c[8], sn[8], w[8], v[8];       // cosine and signed sine, own weight and the partner's
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = p.norm ? s_w[kKind & 1][e < 4 ? ca + e : cb + e - 4] : 1.f;
        if (kMode == kPartners) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            c[e] = c[e + 4] = turns ? s_cos[warp][ca + e] : 1.f;
            sn[e + 4] = turns ? s_sin[warp][ca + e] : 0.f;
            sn[e] = -sn[e + 4];
            v[e] = w[e + 4];
            v[e + 4] = w[e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int ch = ca + e;
            const bool on = ch < 2 * pairs;
            const int pr = kMode == kInside ? ch / 2 : ch < pairs ? ch : ch - pairs;
            const bool low = kMode == kInside ? (ch & 1) == 0 : ch < pairs;
            c[e] = on ? s_cos[warp][pr] : 1.f;
            sn[e] = on ? (low ? -s_sin[warp][pr] : s_sin[warp][pr]) : 0.f;
            v[e] = kMode == kInside ? w[e ^ 1] : on && p.norm ? s_w[kKind & 1][low ? ch + pairs : ch - pairs] : 1.f;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          A[e] = make_float2(w[2 * e] * c[2 * e], w[2 * e + 1] * c[2 * e + 1]);
          B[e] = make_float2(v[2 * e] * sn[2 * e], v[2 * e + 1] * sn[2 * e + 1]);
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (it + u >= i1) break;             // the same in every lane
        const bool real = h0 + u * HPI < H;
        float2 a[2], b[2];                   // the lane's groups
        Quad<TA>::unpack(ra[u], a);
        Quad<TA>::unpack(rb[u], b);
        if (kKind < 2) {
          float2 o[4];                       // partners; channels that do not turn see none, whatever it holds
          if (kMode == kPartners) {
            o[0] = turns ? b[0] : make_float2(0.f, 0.f);
            o[1] = turns ? b[1] : make_float2(0.f, 0.f);
            o[2] = turns ? a[0] : make_float2(0.f, 0.f);
            o[3] = turns ? a[1] : make_float2(0.f, 0.f);
          } else if (kMode == kInside) {
            o[0] = ca < 2 * pairs ? make_float2(a[0].y, a[0].x) : make_float2(0.f, 0.f);
            o[1] = ca + 2 < 2 * pairs ? make_float2(a[1].y, a[1].x) : make_float2(0.f, 0.f);
            o[2] = ca + 4 < 2 * pairs ? make_float2(b[0].y, b[0].x) : make_float2(0.f, 0.f);
            o[3] = ca + 6 < 2 * pairs ? make_float2(b[1].y, b[1].x) : make_float2(0.f, 0.f);
          } else {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int ch = ca + e, partner = ch < pairs ? ch + pairs : ch - pairs;
              v[e] = ch < 2 * pairs && real ? to_float(src[u * HPI * kDh + partner]) : 0.f;
            }
            __syncwarp();                    // every lane has read before one writes in place
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = make_float2(v[2 * e], v[2 * e + 1]);
          }
          float2 r2 = make_float2(1.f, 1.f);
          if (p.norm) {
            const float2 ss = fma2(b[1], b[1], fma2(b[0], b[0], fma2(a[1], a[1], mul2(a[0], a[0]))));
            float sq = ss.x + ss.y;
#pragma unroll
            for (int off = LPH / 2; off >= 1; off >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, off);
            r2.x = r2.y = rsqrtf(sq * (1.f / kDh) + p.eps);
          }
          a[0] = mul2(fma2(o[0], B[0], mul2(a[0], A[0])), r2);
          a[1] = mul2(fma2(o[1], B[1], mul2(a[1], A[1])), r2);
          b[0] = mul2(fma2(o[2], B[2], mul2(b[0], A[2])), r2);
          b[1] = mul2(fma2(o[3], B[3], mul2(b[1], A[3])), r2);
        }
        if (real) {
          store_quad(dst + u * HPI * hop + ca, a);
          store_quad(dst + u * HPI * hop + cb, b);
        }
      }
      h0 += kBatch * HPI;
      src += kBatch * HPI * kDh;
      dst += kBatch * HPI * hop;
    }
  };
  using Q = std::integral_constant<int, 0>;
  using K = std::integral_constant<int, 1>;
  using V = std::integral_constant<int, 2>;
  if (it0 < itq)
    heads(Q{}, static_cast<const TA*>(p.q) + token * p.q_stride, it0, min(it1, itq), p.Hq,
          static_cast<TA*>(p.q_out) + token * p.qo_stride, kDh);
  if constexpr (kAppend) {
    if (!write_kv) return;
    const long long hop = static_cast<long long>(kDh) << p.layer.page_shift;
    if (it1 > itq && it0 < itq + itk)
      heads(K{}, static_cast<const TA*>(p.k) + token * p.k_stride, max(it0, itq) - itq, min(it1, itq + itk) - itq, p.Hk,
            static_cast<TP*>(p.layer.K) + kv_row * kDh, hop);
    if (it1 > itq + itk)
      heads(V{}, static_cast<const TA*>(p.v) + token * p.v_stride, max(it0, itq + itk) - itq - itk, it1 - itq - itk, p.Hk,
            static_cast<TP*>(p.layer.V) + kv_row * kDh, hop);
  } else if (it1 > itq) {
    heads(K{}, static_cast<const TA*>(p.k) + token * p.k_stride, max(it0, itq) - itq, it1 - itq, p.Hk,
          static_cast<TA*>(p.k_out) + token * p.ko_stride, kDh);
  }
}

template <typename TA, typename TP, int kDh, bool kAppend>
cudaError_t launch(const NormRopeLaunch& a, const DeviceInfo& dev, cudaStream_t stream) {
  NrParams p;
  p.q = a.q;
  p.k = a.k;
  p.v = a.v;
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.q_out = a.q_out;
  p.k_out = a.k_out;
  p.qo_stride = a.qo_stride;
  p.ko_stride = a.ko_stride;
  p.Hq = a.Hq;
  p.Hk = a.Hk;
  p.n_tokens = a.n_tokens;
  p.pos = a.pos;
  p.wq = a.wq;
  p.wk = a.wk;
  p.eps = a.eps;
  p.norm = a.norm ? 1 : 0;
  p.status = dev.status_word;
  p.batch = a.batch;
  p.layer = a.layer;
  p.rot = a.rot;
  // one warp a token from 16 warps an SM up; with fewer tokens their heads are split
  constexpr int HPI = 32 / (kDh / 8);
  const int iters = (a.Hq + HPI - 1) / HPI + (a.Hk + HPI - 1) / HPI * (kAppend ? 2 : 1);
  const long long want = (16LL * dev.num_sms + a.n_tokens - 1) / a.n_tokens;
  p.splits = static_cast<int>(want < 1 ? 1 : want > iters ? iters : want);
  const long long warps = static_cast<long long>(a.n_tokens) * p.splits;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((warps + kWarps - 1) / kWarps));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int mode = a.rot.pairs == 0 || a.rot.interleaved ? kInside : a.rot.pairs % 4 == 0 ? kPartners : kAnywhere;
  const cudaError_t e = mode == kPartners ? cudaLaunchKernelEx(&cfg, norm_rope_kernel<TA, TP, kDh, kAppend, kPartners>, p)
                        : mode == kInside ? cudaLaunchKernelEx(&cfg, norm_rope_kernel<TA, TP, kDh, kAppend, kInside>, p)
                                          : cudaLaunchKernelEx(&cfg, norm_rope_kernel<TA, TP, kDh, kAppend, kAnywhere>, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

template <int kDh>
cudaError_t launch_dh(const NormRopeLaunch& a, const DeviceInfo& dev, cudaStream_t stream) {
  using bf = __nv_bfloat16;
  if (!a.append)
    return a.act_bf16 ? launch<bf, bf, kDh, false>(a, dev, stream) : launch<float, float, kDh, false>(a, dev, stream);
  if (a.act_bf16) return launch<bf, bf, kDh, true>(a, dev, stream);
  return a.pool_bf16 ? launch<float, bf, kDh, true>(a, dev, stream) : launch<float, float, kDh, true>(a, dev, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeLaunch& a, const DeviceInfo& dev, cudaStream_t stream) {
  return a.dh == 64 ? launch_dh<64>(a, dev, stream) : launch_dh<128>(a, dev, stream);
}

}  // namespace cxa
