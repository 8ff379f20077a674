// What the two kernels of the latent attention leave for the merge of items that were cut between
// blocks, and the workspace that holds it.
//
// Work is dealt out as in paged_work.cuh. An item cut by a block boundary leaves one partial state
// per block that holds a part of it: block c's slot 2c if the item began before its range, 2c + 1 if
// it goes on behind. The block in which a cut item begins says so in cut[c]; a second kernel merges
// the parts, whose rows and channels it deals out over the whole GPU. (Merging in the last block to
// arrive, as the few-rows kernel of the K/V pages does, would leave one block with 64 rows of 512
// channels of up to 152 parts: 20 MB.)
#pragma once

#include "latent.cuh"

namespace cxa {

constexpr int kLatentMaxBlocks = 320;      // two an SM, where rows are narrow (latent_rows.cu)

struct LatentCut {
  int q0, rt, parts, rows;     // of the item: first token row, tile, parts (0: none), rows of the tile
};

// In the workspace: room that stands for the counters of the paged attention's, which must stay as they are where a
// caller has one buffer for both, the cuts, and the partial states.
constexpr size_t kLatentCutBytes = kLatentMaxBlocks * sizeof(LatentCut);
static_assert((kPagedCounterBytes + kLatentCutBytes) % 256 == 0, "the partial states behind are aligned");
inline LatentCut* latent_cuts(void* workspace) {
  return reinterpret_cast<LatentCut*>(static_cast<uint8_t*>(workspace) + kPagedCounterBytes);
}
inline float* latent_part(void* workspace) {
  return reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kPagedCounterBytes + kLatentCutBytes);
}

// A partial state: [R][latent] sums, then R references (base 2) and R sums of weights.
__host__ __device__ constexpr size_t latent_slot(int R, int latent) { return static_cast<size_t>(R) * (latent + 2); }

inline size_t latent_parts_bytes(int R, int latent, int blocks) {
  return kPagedCounterBytes + kLatentCutBytes + 2 * static_cast<size_t>(blocks) * latent_slot(R, latent) * 4;
}
// Blocks an SM of the fp32 kernel, and the most that a kernel of so many an SM runs.
constexpr int latent_rows_blocks(int latent) { return latent <= 256 ? 2 : 1; }
constexpr int latent_max_blocks(int per_sm) { return 160 * per_sm; }

// Enqueues the merge behind a kernel of `blocks` blocks (latent_merge.cu).
cudaError_t launch_latent_merge(const LatentAttnLaunch& a, int R, int blocks, const DeviceInfo& dev,
                                cudaStream_t stream);

// latent_rows.cu: fp32; latent_tile.cu: bf16.
constexpr int kLatentRowsF32 = 16;
cudaError_t launch_latent_rows(const LatentAttnLaunch& a, const DeviceInfo& dev, cudaStream_t stream);

}  // namespace cxa
