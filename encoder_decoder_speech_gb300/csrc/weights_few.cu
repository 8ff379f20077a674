// The gathered attention weights of few query rows a K/V head (16 at most) in fp32, on the CUDA cores, and the
// addition of stored scores' weights, fp32 and bf16 (weights_tile.cu).
//
//   ref_r = log2 sum_j 2^s_rj,   W_j = decay W_j + sum_r 2^(s_rj - ref_r),   s = scale log2(e) q K^T
//
// weights_few_rows_kernel is bound by reading K: chunks of 128 keys come by cp.async two ahead, a thread takes
// one key's row from shared memory and the rows' queries as broadcasts, up to four rows at a time (always four:
// 2 us and 19 more of the two calls below), and stores the scores (4 bytes a row and key, against 4 dh bytes
// of the key itself). 16 single tokens over up to 4000 keys of 8 heads of 64: 31 us; 32 over up to 8000 keys of 8 heads
// of 128: 122 us, 4.5 TB/s.
// weights_add_kernel reads them back, mostly from L2, and adds the weights to W.
#include "ptx.cuh"
#include "weights_few.cuh"

namespace cxa {
namespace {

constexpr int kThreads = kFewKeys, kStages = 3;

struct FewParams {
  const float* q;
  long long q_stride;
  float qscale;
  unsigned int* counters;
  float* ref;               // [Hkv][n_tokens][G]
  float* part;              // [2 * grid][kScoreRows][2]
  float* scores;
  ScoreRule rule;
  unsigned int* status;
  PagedBatch batch;
  PagedLayer layer;
  WorkShape shape;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <int kDh>
struct Shape {
  static constexpr int row = kDh + 4;        // floats: threads' rows fall into different banks
  static constexpr int smem = (kStages * kFewKeys * row + kScoreRows * kDh) * 4;
  static constexpr int per_sm = kDh == 64 ? 2 : 1;
};

// A key's products with kN rows of queries.
template <int kDh, int kN>
__device__ __forceinline__ void products(const float* key, const float* q, float* x) {
  float s[kN][2];
#pragma unroll
  for (int r = 0; r < kN; ++r) s[r][0] = s[r][1] = 0.f;
#pragma unroll 8
  for (int i = 0; i < kDh; i += 4) {
    const float4 k = *reinterpret_cast<const float4*>(key + i);
#pragma unroll
    for (int r = 0; r < kN; ++r) {
      const float4 v = *reinterpret_cast<const float4*>(q + r * kDh + i);
      s[r][0] = fmaf(v.y, k.y, fmaf(v.x, k.x, s[r][0]));
      s[r][1] = fmaf(v.w, k.w, fmaf(v.z, k.z, s[r][1]));
    }
  }
#pragma unroll
  for (int r = 0; r < kN; ++r) x[r] = s[r][0] + s[r][1];
}

template <int kDh>
__global__ void __launch_bounds__(kThreads, Shape<kDh>::per_sm)
    weights_few_rows_kernel(const __grid_constant__ FewParams p) {
  using S = Shape<kDh>;
  extern __shared__ __align__(16) float smem[];
  float* const s_q = smem + kStages * kFewKeys * S::row;       // [kScoreRows][kDh]
  __shared__ WorkScratch s_work;
  __shared__ FewShared s_few;
  __shared__ uint32_t s_bad[kStages];        // groups of 16 keys whose page is outside the pool
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PagedBatch& bt = p.batch;
  const int Hkv = p.layer.Hkv, shift = p.layer.page_shift, G = p.shape.G;
  WorkRange range;
  WorkCursor cur;
  WorkShape shape = p.shape;
  const bool kept = p.rule.ask ? score_ask<kThreads>(p.rule, bt, G, Hkv, shape.cap, &s_work) : p.rule.kept;
  if (!work_locate<kThreads, false>(bt, shape, Hkv, &s_work, &range, &cur, p.status)) return;
  const int n_chunks = range.g1 - range.g0;

  // ---- the copies' place in the work, up to two chunks ahead
  WorkCursor at = cur;
  int at_c = cur.c, asked = 0;      // chunks looked up
  // the pages of the next chunk's groups of 16 keys, in lanes 0 to 7 (-1: outside the pool, -2: no keys)
  auto look = [&]() {
    int page = -2;
    const int key = at_c * kFewKeys + lane * 16;
    if (asked < n_chunks && lane < kFewKeys / 16 && key < tile_keys(at.seq, shape, at.rt))
      page = paged_lookup(bt.table + static_cast<size_t>(at.b) * bt.width, bt.width, shift, p.layer.num_pages, key);
    return page;
  };
  int pages = look();
  auto fetch = [&](int stage) {
    if (asked < n_chunks) {
      const int keys = tile_keys(at.seq, shape, at.rt);
      const uint32_t bad = __ballot_sync(0xffffffffu, pages == -1);
      if (warp == 0 && lane == 0) {
        s_bad[stage] = bad;
        if (bad != 0) atomicOr(p.status, kStatusBadPage);
      }
      constexpr int pieces = kDh / 4, per = kThreads / pieces;      // of 16 bytes; keys at a time
      const int piece = tid % pieces, sub = tid / pieces;
      const float* K = static_cast<const float*>(p.layer.K);
#pragma unroll
      for (int k0 = 0; k0 < kFewKeys; k0 += per) {
        const int k = k0 + sub, key = at_c * kFewKeys + k;
        const int page = __shfl_sync(0xffffffffu, pages, k >> 4);
        if (page >= 0 && key < keys)
          cp_async16(smem_u32(smem + (stage * kFewKeys + k) * S::row + piece * 4),
                     K + (((static_cast<size_t>(page) * Hkv + at.h) << shift) + (key & ((1 << shift) - 1))) * kDh + piece * 4);
      }
      if (++asked < n_chunks && ++at_c == at.nc) {
        work_next(bt, shape, Hkv, &at);
        at_c = 0;
      }
      pages = look();
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) fetch(i);

  int stage = 0;
  for (;;) {
    const int end = min(range.g1, cur.first + cur.nc), c0 = cur.c, c1 = end - cur.first;
    const PagedSeq seq = cur.seq;
    const int rows = work_rows(seq, shape);      // one tile an item
    const int see_all = visible_keys(seq, 0, shape.cap);
    __syncthreads();                             // the queries of the item before have been read
    for (int e = tid; e < kScoreRows * (kDh / 4); e += kThreads) {
      const int r = e / (kDh / 4), c = e % (kDh / 4) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows)
        v = *reinterpret_cast<const float4*>(p.q + (seq.q0 + r / G) * p.q_stride +
                                             static_cast<long long>(cur.h * G + r % G) * kDh + c);
      *reinterpret_cast<float4*>(s_q + r * kDh + c) = v;
    }
    float m[kScoreRows], l[kScoreRows];
#pragma unroll
    for (int r = 0; r < kScoreRows; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
    }
    for (int c = c0; c < c1; ++c) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncthreads();      // the chunk is there, and the one before has been read
      fetch(stage == 0 ? kStages - 1 : stage - 1);
      const float* row = smem + (stage * kFewKeys + tid) * S::row;
      float x[kScoreRows];
#pragma unroll
      for (int r0 = 0; r0 < kScoreRows; r0 += 4) {
        if (r0 >= rows) break;
        const float* q = s_q + r0 * kDh;
        if (rows - r0 == 1)
          products<kDh, 1>(row, q, x + r0);
        else if (rows - r0 == 2)
          products<kDh, 2>(row, q, x + r0);
        else
          products<kDh, 4>(row, q, x + r0);
      }
      const int key = c * kFewKeys + tid;
      const bool gone = (s_bad[stage] >> (tid >> 4) & 1u) != 0 || key >= shape.cap;
      const int hidden = gone ? kScoreRows : (c + 1) * kFewKeys > see_all ? min(max(key - (seq.kv - seq.n), 0), kScoreRows) * G : 0;
      float* to = kept ? p.scores + static_cast<size_t>(cur.first + c) * p.rule.max_rows * kFewKeys + tid : nullptr;
      few_take(x, rows, hidden, p.qscale, to, m, l);
      if (++stage == kStages) stage = 0;
    }
    few_finish(&s_few, m, l, rows, cur, range, c0, c1, true, p.part, p.counters,
               p.ref + (static_cast<size_t>(cur.h) * bt.n_tokens + seq.q0) * G);
    if (end >= range.g1) break;
    work_next(bt, shape, Hkv, &cur);
  }
}

constexpr int kAddBlocks = 16;      // an SM, small ones: a block of 512 threads waits longer for its last (127 us, 124 so)
__global__ void __launch_bounds__(kThreads, kAddBlocks) weights_add_kernel(const __grid_constant__ WeightsAdd p) {
  __shared__ WorkScratch s_work;
  __shared__ float s_ref[kScoreRows];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  const PagedBatch& bt = p.batch;
  WorkRange range;
  WorkCursor cur;
  WorkShape shape = p.shape;
  if (!scores_kept(p.rule)) return;
  if (!work_locate<kThreads, false>(bt, shape, p.Hkv, &s_work, &range, &cur)) return;
  for (;;) {
    const int end = min(range.g1, cur.first + cur.nc), c0 = cur.c, c1 = end - cur.first;
    const PagedSeq seq = cur.seq;
    const int rows = work_rows(seq, shape), keys = min(seq.kv, shape.cap);
    const int* row = bt.table + static_cast<size_t>(cur.b) * bt.width;
    __syncthreads();
    if (tid < rows) s_ref[tid] = __ldcg(p.ref + (static_cast<size_t>(cur.h) * bt.n_tokens + seq.q0) * shape.G + tid);
    __syncthreads();
#pragma unroll 4
    for (int c = c0; c < c1; ++c) {
      const int key = c * kFewKeys + tid;
      const int page = key < keys ? paged_lookup(row, bt.width, p.page_shift, p.num_pages, key) : -1;
      const float* from = p.scores + static_cast<size_t>(cur.first + c) * p.rule.max_rows * kFewKeys + tid;
      float add = 0.f;
#pragma unroll 4
      for (int r = 0; r < rows; ++r) add += few_rescale(__ldcg(from + r * kFewKeys), s_ref[r]);      // (0 of a hidden key)
      if (page >= 0) {
        float* W = p.W + ((static_cast<size_t>(page) * p.Hkv + cur.h) << p.page_shift) + (key & ((1 << p.page_shift) - 1));
        *W = (key >= seq.kv - seq.n || p.decay == 0.f ? 0.f : p.decay * *W) + add;
      }
    }
    if (end >= range.g1) return;
    work_next(bt, shape, p.Hkv, &cur);
  }
}

template <int kDh>
cudaError_t launch(const WeightsLaunch& a, const DeviceInfo& dev, cudaStream_t stream) {
  using S = Shape<kDh>;
  FewParams p;
  p.q = static_cast<const float*>(a.q);
  p.q_stride = a.q_stride;
  p.qscale = a.scale * 1.4426950408889634f;
  const WeightsPlaces at = weights_places(a);
  p.counters = at.counters;
  p.ref = at.ref;
  p.part = at.part;
  p.scores = at.scores;
  p.status = dev.status_word;
  p.batch = a.batch;
  p.layer = a.layer;
  p.shape.G = a.Hq / a.layer.Hkv;
  p.rule = score_rule(
      weights_split(a.batch.B, a.batch.width, a.layer.page_shift, a.layer.num_pages, a.layer.Hkv, p.shape.G, a.max_new),
      at);
  p.shape.rows = kScoreRows;
  p.shape.chunk_shift = kFewChunkShift;
  p.shape.coarse = false;
  p.shape.cap = a.batch.width << a.layer.page_shift;
  p.shape.min_rows = 0;
  p.shape.max_rows = p.rule.max_rows;      // (the room for scores holds no more)
  p.shape.alone = true;
  static SmemOnce once;
  cudaError_t e = allow_smem(weights_few_rows_kernel<kDh>, S::smem, dev.device, &once);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const int grid = dev.num_sms * S::per_sm < kWeightsMaxBlocks ? dev.num_sms * S::per_sm : kWeightsMaxBlocks;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, weights_few_rows_kernel<kDh>, p);
  if (e != cudaSuccess) return e;
  count_launches(1);
  if (!p.rule.kept && (e = launch_weights_rows(a, &p.rule, dev, stream)) != cudaSuccess) return e;
  if (!p.rule.kept && !p.rule.ask) return e;
  WeightsAdd add = {p.rule, p.batch, p.shape, a.layer.num_pages, a.layer.Hkv, a.layer.page_shift, p.scores, p.ref, a.weights,
                    a.decay};
  return launch_weights_add(add, dev, stream);
}

}  // namespace

cudaError_t launch_weights_add(const WeightsAdd& a, const DeviceInfo& dev, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(dev.num_sms * kAddBlocks));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, weights_add_kernel, a);
  if (e == cudaSuccess) count_launches(1);
  return e;
}

cudaError_t launch_weights_few_rows(const WeightsLaunch& a, const DeviceInfo& dev, cudaStream_t stream) {
  return a.dh == 64 ? launch<64>(a, dev, stream) : launch<128>(a, dev, stream);
}

}  // namespace cxa
