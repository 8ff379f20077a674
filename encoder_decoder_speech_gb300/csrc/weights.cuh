// What the kernels of the gathered attention weights share.
#pragma once

#include "latent.cuh"

namespace cxa {

// The workspace: the counters of the paged attention's workspace (the first kernel's arrivals use
// the few-rows kernel's), the rows' references, the partial states of items that were cut, and the
// scores of calls with few rows. A row's reference is log2 of the sum of its weights' numerators, +inf where
// it sees no key, so that p_j = 2^(s_j - ref) either way.
constexpr int kWeightsMaxBlocks = 160 * 2;
constexpr int kWeightsMaxRows = 256;            // of an item
static_assert(kWeightsMaxBlocks * 3 <= static_cast<int>(kRowsCounters), "the arrivals fit the shared counters");
inline size_t weights_ref_bytes(long long rows) { return (static_cast<size_t>(rows) * 4 + 255) / 256 * 256; }
constexpr size_t kWeightsPartBytes = static_cast<size_t>(2 * kWeightsMaxBlocks) * kWeightsMaxRows * 2 * 4;

// Chunks of 128 keys that a call can have, as far as the host knows, and the room that the scores of `rows` query
// rows a head take in them; 0 if it is too much, so that they are not kept.
constexpr size_t kMaxScoreBytes = 256u << 20;
inline double weights_chunks(int B, int width, int page_shift, int Hkv) {
  return static_cast<double>(B) * Hkv * ((static_cast<long long>(width) << page_shift >> 7) + 1);
}
inline size_t weights_score_bytes(int B, int width, int page_shift, int Hkv, int rows) {
  const double n = weights_chunks(B, width, page_shift, Hkv) * rows * (128 * 4);
  return n <= static_cast<double>(kMaxScoreBytes) ? static_cast<size_t>(n) : 0;
}

// fp32, sequences of at most 16 query rows a K/V head whose scores have room (weights_few.cu).
cudaError_t launch_weights_few_rows(const WeightsLaunch& a, const DeviceInfo& dev, cudaStream_t stream);
// fp32, and bf16 with more query heads a K/V head than a tile holds, on the CUDA cores (weights_rows.cu).
cudaError_t launch_weights_rows(const WeightsLaunch& a, const DeviceInfo& dev, cudaStream_t stream);
// bf16 (weights_tile.cu): sequences of up to few_rows query rows a K/V head go one way, the others
// another; score_bytes is the room that the former's scores take (0: too much, they are not kept).
struct WeightsSplit {
  int few_rows;       // 0: none do
  bool many;          // whether there can be others
  size_t score_bytes;
};
WeightsSplit weights_split(int B, int width, int page_shift, int Hkv, int G, int max_new);
cudaError_t launch_weights_tile(const WeightsLaunch& a, const DeviceInfo& dev, cudaStream_t stream, std::string* msg);

}  // namespace cxa
