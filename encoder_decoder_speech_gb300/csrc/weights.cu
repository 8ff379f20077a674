// Dispatch of the gathered attention weights.
#include "weights.cuh"

namespace cxa {
namespace {

// A tile of 128 rows holds whole tokens, so G query heads have to fit into it.
bool on_tiles(int G, bool bf16) { return bf16 && G <= 128; }
// The room for scores that an fp32 call of few rows takes; 0: it goes the way of many. (16 single tokens over up to
// 4000 keys of 8 heads of 64: 194 us that way, 27 this.)
size_t few_scores(int B, int width, int page_shift, int Hkv, int G, int max_new, bool bf16) {
  return bf16 || static_cast<long long>(G) * max_new > 16 ? 0 : weights_score_bytes(B, width, page_shift, Hkv, G * max_new);
}

}  // namespace

size_t weights_workspace(int B, int n_tokens, int width, int page_shift, int Hq, int Hkv, int max_new, bool bf16) {
  const int G = Hq / Hkv;
  size_t n = kPagedCounterBytes + weights_ref_bytes(static_cast<long long>(n_tokens) * Hq) + kWeightsPartBytes;
  if (on_tiles(G, bf16)) return n + weights_split(B, width, page_shift, Hkv, G, max_new).score_bytes;
  return n + few_scores(B, width, page_shift, Hkv, G, max_new, bf16);
}

cudaError_t launch_weights(const WeightsLaunch& a, const DeviceInfo& dev, cudaStream_t stream, std::string* msg) {
  if (on_tiles(a.Hq / a.layer.Hkv, a.bf16)) return launch_weights_tile(a, dev, stream, msg);
  if (few_scores(a.batch.B, a.batch.width, a.layer.page_shift, a.layer.Hkv, a.Hq / a.layer.Hkv, a.max_new, a.bf16) != 0)
    return launch_weights_few_rows(a, dev, stream);
  return launch_weights_rows(a, dev, stream);
}

}  // namespace cxa
