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
// in registers over the token's heads.
//
// Bound by memory: every value is read once and written once, about 6 operations each. A
// warp takes one token; a head is read by dh * size / 16 lanes, 16 bytes a lane, and
// kBatch such loads are under way before the first is used. The phases are computed once
// a token, one pair a lane, from a 64-bit fixed-point turn (RotaryArg), and handed round
// through shared memory. With few tokens the heads are dealt to several warps.
#include <cuda_bf16.h>

#include "paged.cuh"
#include "ptx.cuh"

namespace cxa {
namespace {

constexpr int kWarps = 8;
constexpr int kBatch = 4;    // heads' loads under way in a lane

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

// 16 bytes of T as floats.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int n = 4;
  __device__ static void unpack(const uint4& u, float (&x)[4]) {
    x[0] = __uint_as_float(u.x);
    x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z);
    x[3] = __uint_as_float(u.w);
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int n = 8;
  __device__ static void unpack(const uint4& u, float (&x)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = lo_bf16(w[i]);
      x[2 * i + 1] = hi_bf16(w[i]);
    }
  }
};

__device__ __forceinline__ void store_vec(float* p, const float (&y)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(y[0], y[1], y[2], y[3]);
}
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&y)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
}
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&y)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                                            pack_bf16(y[6], y[7]));
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

template <typename TA, typename TP, int kDh, bool kAppend>
__global__ void __launch_bounds__(kWarps * 32) norm_rope_kernel(const __grid_constant__ NrParams p) {
  constexpr int VE = Vec<TA>::n;           // channels a lane holds
  constexpr int LPH = kDh / VE;            // lanes a head
  constexpr int HPI = 32 / LPH;            // heads a warp reads at once
  __shared__ float2 s_cs[kWarps][kDh / 2]; // f * (cos, sin) of the token's pairs

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * kWarps + warp;
  const long long tok_ll = item / p.splits;
  if (tok_ll >= p.n_tokens) return;
  const int token = static_cast<int>(tok_ll), part = static_cast<int>(item - tok_ll * p.splits);
  const int sub = lane / LPH, c0 = (lane % LPH) * VE;

  const int itq = (p.Hq + HPI - 1) / HPI, itk = (p.Hk + HPI - 1) / HPI;
  const int iters = itq + itk * (kAppend ? 2 : 1);
  const int per = (iters + p.splits - 1) / p.splits;
  const int it0 = part * per, it1 = min(iters, it0 + per);
  if (it0 >= it1) return;

  int pos = 0;
  bool write_kv = false;
  size_t kv_row = 0;      // of head 0 in the page; heads are page_size rows apart
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
      kv_row = ((static_cast<size_t>(write_kv ? page : 0) * p.layer.Hkv) << p.layer.page_shift) +
               (pos & ((1 << p.layer.page_shift) - 1));
    }
  } else {
    pos = __ldg(p.pos + token);
  }

  const int pairs = p.rot.pairs;
  bool have_cs = false;
  auto phases = [&]() {
    have_cs = true;
    for (int i = lane; i < pairs; i += 32) {
      const unsigned long long ph = static_cast<unsigned long long>(static_cast<long long>(pos)) * p.rot.step[i];
      float sn, cs;
      // half turns in [-1, 1); the 32 high bits of the phase are finer than fp32 holds
      sincospif(static_cast<float>(static_cast<int>(ph >> 32)) * 4.6566128730773926e-10f, &sn, &cs);
      s_cs[warp][i] = make_float2(cs * p.rot.factor, sn * p.rot.factor);
    }
    __syncwarp();
  };

  // Normalise and rotate heads [a0 * HPI, a1 * HPI) of one tensor; dst(h, y) stores this
  // lane's channels of head h.
  auto run = [&](const TA* src, int H, const float* w, int a0, int a1, auto dst) {
    float A[VE], B[VE];
    bool first = true;
    // whole 16-byte groups swap places: the partner sits in another lane, else in this one
    const bool shift_lanes = !p.rot.interleaved && pairs % VE == 0;
    const int shift = shift_lanes ? pairs / VE : 0;
    const int from = c0 < pairs ? lane + shift : c0 < 2 * pairs ? lane - shift : lane;
    const bool in_lane = p.rot.interleaved || pairs == 0;
    for (int i = a0; i < a1; i += kBatch) {
      uint4 raw[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int h = (i + u) * HPI + sub;
        raw[u] = make_uint4(0, 0, 0, 0);
        if (i + u < a1 && h < H) raw[u] = *reinterpret_cast<const uint4*>(src + h * kDh + c0);
      }
      if (!have_cs) phases();
      if (first) {
        first = false;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const int c = c0 + e;
          A[e] = p.norm && w != nullptr ? __ldg(w + c) : 1.f;
          B[e] = 0.f;
          if (c < 2 * pairs) {
            const int pr = p.rot.interleaved ? c / 2 : c < pairs ? c : c - pairs;
            const bool low = p.rot.interleaved ? (c & 1) == 0 : c < pairs;
            const int partner = p.rot.interleaved ? c ^ 1 : low ? c + pairs : c - pairs;
            const float2 cs = s_cs[warp][pr];
            B[e] = (low ? -cs.y : cs.y) * (p.norm && w != nullptr ? __ldg(w + partner) : 1.f);
            A[e] *= cs.x;
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        if (i + u >= a1) break;          // the same in every lane
        const int h = (i + u) * HPI + sub;
        float x[VE], y[VE];
        Vec<TA>::unpack(raw[u], x);
        float r = 1.f;
        if (p.norm) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < VE; ++e) ss += x[e] * x[e];
#pragma unroll
          for (int off = LPH / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
          r = rsqrtf(ss * (1.f / kDh) + p.eps);
        }
        float o[VE];                     // the partners
        if (in_lane) {
#pragma unroll
          for (int e = 0; e < VE; ++e) o[e] = x[e ^ 1];
        } else if (shift_lanes) {
          uint4 t;
          t.x = __shfl_sync(0xffffffffu, raw[u].x, from);
          t.y = __shfl_sync(0xffffffffu, raw[u].y, from);
          t.z = __shfl_sync(0xffffffffu, raw[u].z, from);
          t.w = __shfl_sync(0xffffffffu, raw[u].w, from);
          Vec<TA>::unpack(t, o);
        } else {                         // pairs not a multiple of a lane's channels: read again
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            const int c = c0 + e;
            o[e] = 0.f;
            if (c < 2 * pairs && h < H) o[e] = to_float(src[h * kDh + (c < pairs ? c + pairs : c - pairs)]);
          }
          __syncwarp();                  // every lane has read before one writes in place
        }
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          // channels behind the rotated ones see no partner, whatever it holds
          const float rotated = c0 + e < 2 * pairs ? fmaf(o[e], B[e], x[e] * A[e]) : x[e] * A[e];
          y[e] = rotated * r;
        }
        if (h < H) dst(h, y);
      }
    }
  };

  if (it0 < itq) {
    TA* out = static_cast<TA*>(p.q_out) + static_cast<long long>(token) * p.qo_stride;
    run(static_cast<const TA*>(p.q) + static_cast<long long>(token) * p.q_stride, p.Hq, p.wq, it0, min(it1, itq),
        [&](int h, const float(&y)[VE]) { store_vec(out + h * kDh + c0, y); });
  }
  if constexpr (!kAppend) {
    if (it1 > itq) {
      TA* out = static_cast<TA*>(p.k_out) + static_cast<long long>(token) * p.ko_stride;
      run(static_cast<const TA*>(p.k) + static_cast<long long>(token) * p.k_stride, p.Hk, p.wk, max(it0, itq) - itq,
          it1 - itq, [&](int h, const float(&y)[VE]) { store_vec(out + h * kDh + c0, y); });
    }
  } else {
    if (!write_kv) return;
    if (it1 > itq && it0 < itq + itk) {
      TP* out = static_cast<TP*>(p.layer.K) + kv_row * kDh;
      run(static_cast<const TA*>(p.k) + static_cast<long long>(token) * p.k_stride, p.Hk, p.wk, max(it0, itq) - itq,
          min(it1, itq + itk) - itq, [&](int h, const float(&y)[VE]) {
            store_vec(out + (static_cast<size_t>(h) << p.layer.page_shift) * kDh + c0, y);
          });
    }
    if (it1 > itq + itk) {
      const TA* src = static_cast<const TA*>(p.v) + static_cast<long long>(token) * p.v_stride;
      TP* out = static_cast<TP*>(p.layer.V) + kv_row * kDh;
      const int a0 = max(it0, itq + itk) - itq - itk, a1 = it1 - itq - itk;
      for (int i = a0; i < a1; i += kBatch) {
        uint4 raw[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int h = (i + u) * HPI + sub;
          raw[u] = make_uint4(0, 0, 0, 0);
          if (i + u < a1 && h < p.Hk) raw[u] = *reinterpret_cast<const uint4*>(src + h * kDh + c0);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const int h = (i + u) * HPI + sub;
          if (i + u < a1 && h < p.Hk) {
            float x[VE];
            Vec<TA>::unpack(raw[u], x);
            store_vec(out + (static_cast<size_t>(h) << p.layer.page_shift) * kDh + c0, x);
          }
        }
      }
    }
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
  constexpr int HPI = 32 / (kDh / Vec<TA>::n);
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, norm_rope_kernel<TA, TP, kDh, kAppend>, p);
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
