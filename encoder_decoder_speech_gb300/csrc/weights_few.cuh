// What the kernels of the gathered weights for few query rows share: one to 16 rows of a K/V head, in chunks
// of 128 keys, a key a thread. Each thread keeps references and sums of its own until an item's end and stores
// its scores; weights_add_kernel (weights_few.cu) reads them back.
#pragma once

#include <cmath>

#include "paged_work.cuh"
#include "weights.cuh"

namespace cxa {

constexpr int kScoreRows = 16, kFewKeys = 128, kFewChunkShift = 7;

// In shared memory.
struct FewShared {
  float m[4][kScoreRows], l[4][kScoreRows];
  int last;
};

// Whether the scores of sequences with few rows are kept, by all kThreads threads of a first kernel's block, which
// leaves it for the kernels behind. (rule.ask)
template <int kThreads>
__device__ bool score_ask(const ScoreRule& rule, const PagedBatch& bt, int G, int Hkv, int cap, WorkScratch* sm) {
  int chunks = 0;
  for (int b = threadIdx.x; b < bt.B; b += kThreads) {
    const PagedSeq s = paged_seq(bt.q_start, bt.kv_len, b, bt.n_tokens);
    const long long rows = static_cast<long long>(s.n) * G;
    if (rows == 0 || rows > rule.max_rows) continue;
    const long long n = static_cast<long long>(max(1, (min(s.kv, cap) + kFewKeys - 1) / kFewKeys)) * Hkv;
    chunks = count_add(chunks, static_cast<int>(min(n, static_cast<long long>(kCountLimit))));
  }
#pragma unroll
  for (int off = 16; off >= 1; off >>= 1) chunks = count_add(chunks, __shfl_xor_sync(0xffffffffu, chunks, off));
  if ((threadIdx.x & 31) == 0) sm->scan[0][threadIdx.x >> 5] = chunks;
  __syncthreads();
  chunks = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) chunks = count_add(chunks, sm->scan[0][i]);
  __syncthreads();
  const bool kept = chunks <= rule.room;
  if (blockIdx.x == 0 && threadIdx.x == 0) *rule.word = kept ? 1u : 0u;
  return kept;
}
// In the kernels behind.
__device__ __forceinline__ bool scores_kept(const ScoreRule& rule) {
  return rule.ask ? __ldcg(rule.word) != 0u : rule.kept;
}

// For a rescaling from reference m to `to`.
__device__ __forceinline__ float few_rescale(float m, float to) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(m - to));
  return m == -INFINITY ? 0.f : y;
}
// log2 of a sum with reference M; +inf for a row that sees no key.
__device__ __forceinline__ float log_sum(float M, float L) { return L > 0.f || L != L ? M + log2f(L) : INFINITY; }

// Scores x of a key, on their way to the rows' references and to `to` (if not null). Rows before `hidden`
// do not see the key.
__device__ __forceinline__ void few_take(const float (&x)[kScoreRows], int rows, int hidden, float qscale, float* to,
                                         float (&m)[kScoreRows], float (&l)[kScoreRows]) {
#pragma unroll
  for (int r = 0; r < kScoreRows; ++r) {
    if (r >= rows) break;
    const float s = r >= hidden ? x[r] * qscale : -INFINITY;
    if (to != nullptr) __stcg(to + r * kFewKeys, s);
    const float up = fmaxf(m[r], s);
    l[r] = l[r] * few_rescale(m[r], up) + few_rescale(s, up);
    m[r] = up;
  }
}

// The keys of an item's chunks [c0, c1) together, by 128 threads; the rows' references, once the item's parts
// are all there. `ok` is false after a wait that ran out: nothing is written then.
__device__ __forceinline__ void few_finish(FewShared* sm, const float (&m)[kScoreRows], const float (&l)[kScoreRows], int rows,
                                           const WorkCursor& cur, const WorkRange& range, int c0, int c1, bool ok,
                                           float* part_base, unsigned int* counters, float* refs) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
#pragma unroll
  for (int r = 0; r < kScoreRows; ++r) {
    if (r >= rows) break;
    float M = m[r];
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float L = l[r] * few_rescale(m[r], M);
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) L += __shfl_xor_sync(0xffffffffu, L, off);
    if (lane == 0) {
      sm->m[warp][r] = M;
      sm->l[warp][r] = L;
    }
  }
  asm volatile("bar.sync 1, 128;" ::: "memory");
  const bool whole = c0 == 0 && c1 == cur.nc;
  float M = -INFINITY, L = 0.f;
  if (tid < rows) {
#pragma unroll
    for (int q = 0; q < 4; ++q) M = fmaxf(M, sm->m[q][tid]);
#pragma unroll
    for (int q = 0; q < 4; ++q) L += sm->l[q][tid] * few_rescale(sm->m[q][tid], M);
    if (!whole) {
      float* slot = part_base + (2 * static_cast<size_t>(blockIdx.x) + (c0 == 0 ? 1 : 0)) * (kScoreRows * 2);
      slot[tid] = M;
      slot[kScoreRows + tid] = L;
    }
  }
  bool write = whole && ok;
  if (!whole) {
    const int owner = cur.first / range.per, parts = (cur.first + cur.nc - 1) / range.per - owner + 1;
    asm volatile("bar.sync 1, 128;" ::: "memory");
    if (tid == 0) {
      bool last = false;
      if (ok) {
        last = atomic_add_acq_rel_gpu(counters + owner, 1u) == static_cast<unsigned int>(parts - 1);
        if (last) counters[owner] = 0u;
      }
      sm->last = last;
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    write = sm->last != 0;
    if (write && tid < rows) {
      auto part = [&](int k) {
        return part_base + (2 * static_cast<size_t>(owner + k) + (k == 0 ? 1 : 0)) * (kScoreRows * 2) + tid;
      };
      M = -INFINITY;
      L = 0.f;
#pragma unroll 8
      for (int k = 0; k < parts; ++k) M = fmaxf(M, __ldcg(part(k)));
#pragma unroll 8
      for (int k = 0; k < parts; ++k) L += __ldcg(part(k) + kScoreRows) * few_rescale(__ldcg(part(k)), M);
    }
  }
  if (write && tid < rows) refs[tid] = log_sum(M, L);
}

// Adds the weights of stored scores to W, if there are any.
struct WeightsAdd {
  ScoreRule rule;
  PagedBatch batch;
  WorkShape shape;         // of the kernel that stored them
  int num_pages, Hkv, page_shift;
  const float* scores;     // of chunk c, row r: [c * rule.max_rows + r][kFewKeys]
  const float* ref;        // [Hkv][n_tokens][G]
  float* W;
  float decay;
};
cudaError_t launch_weights_add(const WeightsAdd& a, const DeviceInfo& dev, cudaStream_t stream);

}  // namespace cxa
