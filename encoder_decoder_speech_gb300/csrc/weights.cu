// Dispatch of the gathered attention weights.
#include "weights.cuh"

namespace cxa {

size_t weights_workspace(int n_tokens, int Hq, int, int, int, bool) {
  return kPagedCounterBytes + weights_ref_bytes(static_cast<long long>(n_tokens) * Hq) + kWeightsPartBytes;
}

cudaError_t launch_weights(const WeightsLaunch& a, const DeviceInfo& dev, cudaStream_t stream, std::string*) {
  return launch_weights_rows(a, dev, stream);
}

}  // namespace cxa
