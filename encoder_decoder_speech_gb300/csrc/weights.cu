// Dispatch of the gathered attention weights.
#include "weights.cuh"

namespace cxa {
namespace {

// A tile of 128 rows holds whole tokens, so G query heads have to fit into it.
bool on_tiles(int G, bool bf16) { return bf16 && G <= 128; }

}  // namespace

size_t weights_workspace(int B, int n_tokens, int width, int page_shift, int Hq, int Hkv, int max_new, bool bf16) {
  const int G = Hq / Hkv;
  size_t n = kPagedCounterBytes + weights_ref_bytes(static_cast<long long>(n_tokens) * Hq) + kWeightsPartBytes;
  if (on_tiles(G, bf16)) n += weights_split(B, width, page_shift, Hkv, G, max_new).score_bytes;
  return n;
}

cudaError_t launch_weights(const WeightsLaunch& a, const DeviceInfo& dev, cudaStream_t stream, std::string* msg) {
  if (on_tiles(a.Hq / a.layer.Hkv, a.bf16)) return launch_weights_tile(a, dev, stream, msg);
  return launch_weights_rows(a, dev, stream);
}

}  // namespace cxa
