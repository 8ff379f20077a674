// The attention weight that keys of a paged cache gather, on the CUDA cores.
//
//   W_j = decay W_j + sum over rows r that see j of 2^(s_rj - ref_r),   s = scale log2(e) q K^T,
//   ref_r = log2 sum_j 2^s_rj
//
// in two passes over the scores, each a product of a tile of 32 query rows and 64 keys: the first,
// dealt out as the attention is (paged_work.cuh), finds the references; in the second a block has the
// keys of a tile for all rows that see them, so that every W is written once, by one thread, and sums
// run in one order. Bound by the products, 2 dh operations a score and pass: 256 tokens in each of two sequences of up to
// 2000 keys, 8 heads of 64, fp32: 123 us, 9.5 TFLOP/s over both passes (a thread reads six vectors of four from shared
// memory for 32 products; larger tiles have not been tried).
#include <cuda_bf16.h>

#include <cmath>

#include "paged_work.cuh"
#include "ptx.cuh"
#include "span_work.cuh"
#include "weights.cuh"
#include "weights_few.cuh"

namespace cxa {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 32, kKeys = 64;
static_assert(kRows <= kWeightsMaxRows, "partial states fit");

struct WeightsParams {
  const void* q;
  long long q_stride;
  float* W;
  float decay, qscale;
  unsigned int* counters;
  float* ref;               // [Hkv][n_tokens][G]
  float* part;              // [2 * grid][kRows][2]
  unsigned int* status;
  PagedBatch batch;
  PagedLayer layer;
  WorkShape shape;
  ScoreRule rule;           // of the second pass: nothing to do if scores were kept
};

// The references of a head's rows.
__device__ __forceinline__ float* refs_of(const WeightsParams& p, const PagedSeq& s, int h) {
  return p.ref + (static_cast<size_t>(h) * p.batch.n_tokens + s.q0) * p.shape.G;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xFFFF0000u));
}

template <typename T, int kDh>
struct Tiles {
  static constexpr int row = kDh + 4;        // floats
  float q[kRows][row];
  float k[kKeys][row];
};

// Rows row0 .. of head h's query rows of a sequence (token by token, G heads a token).
template <typename T, int kDh>
__device__ void load_q(Tiles<T, kDh>* t, const WeightsParams& p, const PagedSeq& seq, int h, int row0, int rows) {
  const int G = p.shape.G;
  for (int i = threadIdx.x; i < kRows * (kDh / 4); i += kThreads) {
    const int r = i / (kDh / 4), c = i % (kDh / 4) * 4, at = row0 + r;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows)
      v = load4(static_cast<const T*>(p.q) + (seq.q0 + at / G) * p.q_stride +
                static_cast<long long>(h * G + at % G) * kDh + c);
    *reinterpret_cast<float4*>(&t->q[r][c]) = v;
  }
}
// Keys key0 .. of head h of sequence b, those from `keys` on and those of bad pages zero.
template <typename T, int kDh>
__device__ void load_k(Tiles<T, kDh>* t, const WeightsParams& p, int b, int h, int key0, int keys) {
  const PagedLayer& ly = p.layer;
  const int* row = p.batch.table + static_cast<size_t>(b) * p.batch.width;
  for (int i = threadIdx.x; i < kKeys * (kDh / 4); i += kThreads) {
    const int k = i / (kDh / 4), c = i % (kDh / 4) * 4, key = key0 + k;
    const int page = key < keys ? paged_lookup(row, p.batch.width, ly.page_shift, ly.num_pages, key) : -1;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (page >= 0)
      v = load4(static_cast<const T*>(ly.K) +
                (((static_cast<size_t>(page) * ly.Hkv + h) << ly.page_shift) + (key & ((1 << ly.page_shift) - 1))) * kDh + c);
    else if (key < keys && c == 0)
      atomicOr(p.status, kStatusBadPage);
    *reinterpret_cast<float4*>(&t->k[k][c]) = v;
  }
}
// This thread's scores: rows 2 ty, 2 ty + 1 and keys tx + 16 j.
template <typename T, int kDh>
__device__ __forceinline__ void scores(const Tiles<T, kDh>* t, float (&s)[2][4]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
  for (int c = 0; c < kDh; c += 4) {
    float4 q[2], k[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) q[i] = *reinterpret_cast<const float4*>(&t->q[2 * ty + i][c]);
#pragma unroll
    for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const float4*>(&t->k[tx + 16 * j][c]);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s[i][j] = fmaf(q[i].w, k[j].w, fmaf(q[i].z, k[j].z, fmaf(q[i].y, k[j].y, fmaf(q[i].x, k[j].x, s[i][j]))));
  }
}

// ---- first pass: the rows' references
template <typename T, int kDh>
__global__ void __launch_bounds__(kThreads) weights_ref_kernel(const __grid_constant__ WeightsParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  Tiles<T, kDh>* t = reinterpret_cast<Tiles<T, kDh>*>(smem);
  __shared__ WorkScratch s_work;
  __shared__ int s_last;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const PagedBatch& bt = p.batch;
  const int Hkv = p.layer.Hkv, G = p.shape.G;
  WorkRange range;
  WorkCursor cur;
  WorkShape shape = p.shape;
  if (!work_locate<kThreads, false>(bt, shape, Hkv, &s_work, &range, &cur, p.status)) return;
  for (;;) {
    const int end = min(range.g1, cur.first + cur.nc), c0 = cur.c, c1 = end - cur.first;
    const PagedSeq seq = cur.seq;
    const int row0 = cur.rt * kRows, rows = min(kRows, work_rows(seq, shape) - row0);
    const int keys = tile_keys(seq, shape, cur.rt);
    __syncthreads();
    load_q(t, p, seq, cur.h, row0, rows);
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int see[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
      see[i] = 2 * ty + i < rows ? visible_keys(seq, (row0 + 2 * ty + i) / G, shape.cap) : 0;
    for (int c = c0; c < c1; ++c) {
      const int key0 = c * kKeys;
      __syncthreads();
      load_k(t, p, cur.b, cur.h, key0, keys);
      __syncthreads();
      float s[2][4];
      scores(t, s);
      const int* row = bt.table + static_cast<size_t>(cur.b) * bt.width;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = key0 + tx + 16 * j;
          const bool on = key < see[i] && paged_lookup(row, bt.width, p.layer.page_shift, p.layer.num_pages, key) >= 0;
          s[i][j] = on ? s[i][j] * p.qscale : -INFINITY;
          top = fmaxf(top, s[i][j]);
        }
        const float to = fmaxf(m[i], top);
        l[i] *= m[i] == -INFINITY ? 0.f : ex2(m[i] - to);
#pragma unroll
        for (int j = 0; j < 4; ++j) l[i] += s[i][j] == -INFINITY ? 0.f : ex2(s[i][j] - to);
        m[i] = to;
      }
    }
    // the row's 16 threads together
    float M[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      M[i] = m[i];
#pragma unroll
      for (int off = 8; off >= 1; off >>= 1) M[i] = fmaxf(M[i], __shfl_xor_sync(0xffffffffu, M[i], off));
      l[i] *= m[i] == -INFINITY ? 0.f : ex2(m[i] - M[i]);
#pragma unroll
      for (int off = 8; off >= 1; off >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], off);
    }
    float* refs = refs_of(p, seq, cur.h) + row0;
    auto put = [&](int r, float M_, float L_) { refs[r] = log_sum(M_, L_); };
    const bool whole = c0 == 0 && c1 == cur.nc;
    if (whole) {
      if (tx < 2 && 2 * ty + tx < rows) put(2 * ty + tx, tx == 0 ? M[0] : M[1], tx == 0 ? l[0] : l[1]);
    } else {
      float* slot = p.part + (2 * static_cast<size_t>(blockIdx.x) + (c0 == 0 ? 1 : 0)) * (kRows * 2);
      if (tx < 2) {
        slot[2 * ty + tx] = tx == 0 ? M[0] : M[1];
        slot[kRows + 2 * ty + tx] = tx == 0 ? l[0] : l[1];
      }
      const int owner = cur.first / range.per, parts = (cur.first + cur.nc - 1) / range.per - owner + 1;
      __syncthreads();
      if (tid == 0) {
        s_last = atomic_add_acq_rel_gpu(p.counters + owner, 1u) == static_cast<unsigned int>(parts - 1);
        if (s_last) p.counters[owner] = 0u;
      }
      __syncthreads();
      if (s_last && tid < rows) {
        float A = -INFINITY, L = 0.f;
        auto part = [&](int k) { return p.part + (2 * static_cast<size_t>(owner + k) + (k == 0 ? 1 : 0)) * (kRows * 2) + tid; };
#pragma unroll 4
        for (int k = 0; k < parts; ++k) A = fmaxf(A, __ldcg(part(k)));
#pragma unroll 4
        for (int k = 0; k < parts; ++k) {
          const float x = __ldcg(part(k));
          L += x == -INFINITY ? 0.f : __ldcg(part(k) + kRows) * ex2(x - A);
        }
        put(tid, A, L);
      }
    }
    if (end >= range.g1) break;
    work_next(bt, shape, Hkv, &cur);
  }
}

// ---- second pass: sums over the rows of a tile of keys
template <typename T, int kDh>
__global__ void __launch_bounds__(kThreads) weights_sum_kernel(const __grid_constant__ WeightsParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  Tiles<T, kDh>* t = reinterpret_cast<Tiles<T, kDh>*>(smem);
  __shared__ SpanScratch s_span;
  __shared__ float s_sum[kKeys][17];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const PagedBatch& bt = p.batch;
  const int Hkv = p.layer.Hkv, G = p.shape.G, cap = p.shape.cap;
  if (scores_kept(p.rule)) return;
  auto key_tiles = [&](int b) {
    const PagedSeq s = paged_seq(bt.q_start, bt.kv_len, b, bt.n_tokens);
    return work_rows(s, p.shape) == 0 ? 0 : (min(s.kv, cap) + kKeys - 1) / kKeys;
  };
  SpanRange range;
  if (!span_locate<kThreads>(bt.B, [&](int b) {
        const long long u = static_cast<long long>(key_tiles(b)) * Hkv;
        return static_cast<int>(min(u, static_cast<long long>(kCountLimit)));
      }, &s_span, &range))
    return;
  int b = range.b, first = range.first;
  for (int g = range.g0; g < range.g1; ++g) {
    while (g - first >= key_tiles(b) * Hkv) {
      first += key_tiles(b) * Hkv;
      ++b;
    }
    const PagedSeq seq = paged_seq(bt.q_start, bt.kv_len, b, bt.n_tokens);
    const int tiles = key_tiles(b), h = (g - first) / tiles, key0 = (g - first) % tiles * kKeys;
    const int keys = min(seq.kv, cap);
    const int* row = bt.table + static_cast<size_t>(b) * bt.width;
    __syncthreads();
    load_k(t, p, b, h, key0, keys);
    bool ok[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int key = key0 + tx + 16 * j;
      ok[j] = key < keys && paged_lookup(row, bt.width, p.layer.page_shift, p.layer.num_pages, key) >= 0;
    }
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    // the first token that sees the tile's first key
    const int i0 = max(0, key0 - (seq.kv - seq.n));
    const int all = seq.n * G;
    for (int row0 = i0 * G / kRows * kRows; row0 < all; row0 += kRows) {
      __syncthreads();
      load_q(t, p, seq, h, row0, min(kRows, all - row0));
      __syncthreads();
      float s[2][4];
      scores(t, s);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int at = row0 + 2 * ty + i;
        if (at >= all) continue;
        const int see = visible_keys(seq, at / G, cap);
        const float ref = __ldcg(refs_of(p, seq, h) + at);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (ok[j] && key0 + tx + 16 * j < see) sum[j] += ex2(s[i][j] * p.qscale - ref);
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 4; ++j) s_sum[tx + 16 * j][ty] = sum[j];
    __syncthreads();
    if (tid < kKeys && key0 + tid < keys) {
      const int key = key0 + tid;
      const int page = paged_lookup(row, bt.width, p.layer.page_shift, p.layer.num_pages, key);
      if (page >= 0) {
        float add = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) add += s_sum[tid][i];
        float* w = p.W + ((static_cast<size_t>(page) * Hkv + h) << p.layer.page_shift) + (key & ((1 << p.layer.page_shift) - 1));
        *w = (key >= seq.kv - seq.n || p.decay == 0.f ? 0.f : p.decay * *w) + add;
      }
    }
  }
}

template <typename T, int kDh>
cudaError_t launch(const WeightsLaunch& a, const ScoreRule* rule, const DeviceInfo& dev, cudaStream_t stream) {
  WeightsParams p;
  p.q = a.q;
  p.q_stride = a.q_stride;
  p.W = a.weights;
  p.decay = a.decay;
  p.qscale = a.scale * 1.4426950408889634f;
  const WeightsPlaces at = weights_places(a);
  p.counters = at.counters;
  p.ref = at.ref;
  p.part = at.part;
  p.rule = rule != nullptr ? *rule : ScoreRule{};
  p.status = dev.status_word;
  p.batch = a.batch;
  p.layer = a.layer;
  p.shape.G = a.Hq / a.layer.Hkv;
  p.shape.rows = kRows;
  p.shape.chunk_shift = 6;
  p.shape.coarse = false;
  p.shape.cap = a.batch.width << a.layer.page_shift;
  p.shape.min_rows = 0;
  p.shape.max_rows = rule != nullptr ? rule->max_rows : 0x7FFFFFFF;
  constexpr int smem = sizeof(Tiles<T, kDh>);
  static SmemOnce once[2];
  cudaError_t e = allow_smem(weights_ref_kernel<T, kDh>, smem, dev.device, &once[0]);
  if (e == cudaSuccess) e = allow_smem(weights_sum_kernel<T, kDh>, smem, dev.device, &once[1]);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int grid = 2 * dev.num_sms < kWeightsMaxBlocks ? 2 * dev.num_sms : kWeightsMaxBlocks;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (rule == nullptr) {
    e = cudaLaunchKernelEx(&cfg, weights_ref_kernel<T, kDh>, p);
    if (e != cudaSuccess) return e;
    count_launches(1);
  }
  e = cudaLaunchKernelEx(&cfg, weights_sum_kernel<T, kDh>, p);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

}  // namespace

cudaError_t launch_weights_rows(const WeightsLaunch& a, const ScoreRule* rule, const DeviceInfo& dev, cudaStream_t stream) {
  using bf = __nv_bfloat16;
  if (a.bf16) return a.dh == 64 ? launch<bf, 64>(a, rule, dev, stream) : launch<bf, 128>(a, rule, dev, stream);
  return a.dh == 64 ? launch<float, 64>(a, rule, dev, stream) : launch<float, 128>(a, rule, dev, stream);
}

}  // namespace cxa
