// What the kernels of the gathered attention weights share.
#pragma once

#include "latent.cuh"

namespace cxa {

// The workspace: the counters of the paged attention's workspace (the first kernel's arrivals use
// the few-rows kernel's), a word (ScoreRule), the rows' references, the partial states of items that were cut, and the
// scores of sequences with few rows. A row's reference is log2 of the sum of its weights' numerators, +inf where
// it sees no key, so that p_j = 2^(s_j - ref) either way. References are [Hkv][n_tokens][G].
constexpr int kWeightsMaxBlocks = 160 * 2;
constexpr int kWeightsMaxRows = 256;            // of an item
static_assert(kWeightsMaxBlocks * 3 <= static_cast<int>(kRowsCounters), "the arrivals fit the shared counters");
inline size_t weights_ref_bytes(long long rows) { return (static_cast<size_t>(rows) * 4 + 255) / 256 * 256; }
constexpr size_t kWeightsPartBytes = static_cast<size_t>(2 * kWeightsMaxBlocks) * kWeightsMaxRows * 2 * 4;

// Sequences with few query rows leave their scores for the second pass, which then need not read K again, if there
// is room for all of them. How many chunks of 128 keys they have is known to the device alone: the host knows the
// width of the table, which may be that of the longest context that a server allows. (64 single tokens over up to
// 8192 keys of 8 heads of 128, a table of 32768: 496 us where the width decided that there is no room.)
struct ScoreRule {
  int room;                // chunks that have room
  int max_rows;            // of a sequence with few rows
  bool others;             // there are sequences of many rows, with whom those of few go if their scores are not kept
  bool ask;                // whether the device decides, in the first kernel; `kept` says it already otherwise
  bool kept;
  unsigned int* word;      // where the first kernel leaves what it found, for the others
};

// Chunks of 128 keys that a call can have, as far as the host knows, and the bytes of a chunk's scores.
constexpr size_t kMaxScoreBytes = 256u << 20;      // that are kept at most
// (sequences of a batch share no page, so that the pool bounds them too; against that, chunks are counted all the same)
inline double weights_pool_chunks(int B, int num_pages, int page_shift, int Hkv) {
  return static_cast<double>(Hkv) * (((static_cast<long long>(num_pages) << page_shift) + 127) / 128 + B);
}
inline double weights_chunks(int B, int width, int page_shift, int Hkv) {
  return static_cast<double>(B) * Hkv * ((static_cast<long long>(width) << page_shift >> 7) + 1);
}
constexpr size_t score_chunk_bytes(int rows) { return static_cast<size_t>(rows) * 128 * 4; }

// The places of all these in a workspace.
struct WeightsPlaces {
  unsigned int *counters, *word;
  float *ref, *part, *scores;
  size_t score_bytes;        // behind `scores`
};
inline size_t weights_fixed_bytes(long long rows) {
  return kPagedCounterBytes + 256 + weights_ref_bytes(rows) + kWeightsPartBytes;
}
inline WeightsPlaces weights_places(const WeightsLaunch& a) {
  const long long rows = static_cast<long long>(a.batch.n_tokens) * a.Hq;
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  WeightsPlaces p;
  p.counters = reinterpret_cast<unsigned int*>(ws);
  p.word = reinterpret_cast<unsigned int*>(ws + kPagedCounterBytes);
  p.ref = reinterpret_cast<float*>(ws + kPagedCounterBytes + 256);
  p.part = reinterpret_cast<float*>(ws + kPagedCounterBytes + 256 + weights_ref_bytes(rows));
  p.scores = reinterpret_cast<float*>(ws + weights_fixed_bytes(rows));
  p.score_bytes = a.workspace_bytes - weights_fixed_bytes(rows);
  return p;
}

// Which sequences have few rows, and what is known of their scores.
struct WeightsSplit {
  int few_rows;       // 0: none do
  bool many;          // whether there can be others
  double chunks;      // that the call can have
  size_t most;        // bytes of scores that it makes use of
};
WeightsSplit weights_split(int B, int width, int page_shift, int num_pages, int Hkv, int G, int max_new);
ScoreRule score_rule(const WeightsSplit& s, const WeightsPlaces& at);

// fp32, sequences of at most 16 query rows a K/V head (weights_few.cu).
cudaError_t launch_weights_few_rows(const WeightsLaunch& a, const DeviceInfo& dev, cudaStream_t stream);
// fp32, and bf16 with more query heads a K/V head than a tile holds, on the CUDA cores (weights_rows.cu). With a
// rule the second pass alone, if scores were not kept, for sequences of up to rule->max_rows.
cudaError_t launch_weights_rows(const WeightsLaunch& a, const ScoreRule* rule, const DeviceInfo& dev, cudaStream_t stream);
// bf16 (weights_tile.cu): sequences of few query rows a K/V head go one way, the others another.
cudaError_t launch_weights_tile(const WeightsLaunch& a, const DeviceInfo& dev, cudaStream_t stream, std::string* msg);

}  // namespace cxa
