// What the expansion's kernels share.
#pragma once

#include "latent.cuh"

namespace cxa {

// fp32, on the CUDA cores (expand_rows.cu; bf16 goes to expand_tile.cu).
cudaError_t launch_expand_rows(const LatentExpandLaunch& a, const DeviceInfo& dev, cudaStream_t stream);

// Positions of sequence b that are expanded: [lo, hi).
struct ExpandSpan {
  int lo, hi;
};
__host__ __device__ inline ExpandSpan expand_span(const int* from, const int* kv_len, int cap, int b) {
  ExpandSpan s;
  const int kv = kv_len[b];
  s.hi = kv < 0 ? 0 : kv > cap ? cap : kv;
  const int f = from != nullptr ? from[b] : 0;
  s.lo = f < 0 ? 0 : f > s.hi ? s.hi : f;
  return s;
}
// Whether some positions of sequence b that are to be expanded lie behind its row of the table.
__host__ __device__ inline bool expand_passes(const int* from, const int* kv_len, int cap, int b) {
  return kv_len[b] > cap && (from == nullptr || from[b] < kv_len[b]);
}

}  // namespace cxa
