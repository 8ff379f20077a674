// What the kernels of the latent cache, and those of the gathered weights and the eviction, take
// from the C-ABI layer.
#pragma once

#include "paged.cuh"

namespace cxa {

// One layer of a latent pool: [num_pages][1 << page_shift][latent + rope].
struct LatentLayer {
  void* C;
  int num_pages, page_shift, latent, rope;
};

struct LatentAppendLaunch {
  const void *c, *kr;               // kr may be null
  long long c_stride, kr_stride;    // elements from one token's row to the next
  const float* weight;              // [latent] or null (1)
  float eps;
  bool norm, act_bf16, pool_bf16;
  RotaryArg rot;
  PagedBatch batch;
  LatentLayer layer;
};
cudaError_t launch_latent_append(const LatentAppendLaunch& a, const DeviceInfo& dev, cudaStream_t stream);

struct LatentAttnLaunch {
  const void* q;
  void* out;
  long long q_stride, o_stride;     // elements
  int H, max_new;
  float scale;
  bool bf16;
  PagedBatch batch;
  LatentLayer layer;
  void* workspace;
};
size_t latent_attention_workspace(int H, int latent, int max_new, bool bf16);
cudaError_t launch_latent_attention(const LatentAttnLaunch& a, const DeviceInfo& dev, cudaStream_t stream,
                                    std::string* msg);

struct LatentExpandLaunch {
  LatentLayer layer;
  PagedLayer to;
  int dh;
  bool bf16;
  int B;
  const int *from, *kv_len, *table, *to_table;
  int width, to_width;
  const void *WK, *WV;
};
cudaError_t launch_latent_expand(const LatentExpandLaunch& a, const DeviceInfo& dev, cudaStream_t stream,
                                 std::string* msg);

struct WeightsLaunch {
  const void* q;
  long long q_stride;
  int Hq, dh, max_new;
  float* weights;                   // of the layer: [num_pages][Hkv][1 << page_shift]
  float decay, scale;
  bool bf16;
  PagedBatch batch;
  PagedLayer layer;
  void* workspace;
  size_t workspace_bytes;
};
// The least that a call needs, and the most that it makes use of.
struct WeightsWorkspace {
  size_t least, most;
};
WeightsWorkspace weights_workspace(int B, int n_tokens, int width, int page_shift, int num_pages, int Hq, int Hkv,
                                   int max_new, bool bf16);
// Whether the work of all its kernels can be numbered in 31 bits.
bool weights_countable(const PagedBatch& bt, int page_shift, int Hkv, int G, bool bf16);
cudaError_t launch_weights(const WeightsLaunch& a, const DeviceInfo& dev, cudaStream_t stream, std::string* msg);

struct EvictLaunch {
  void *K, *V;                      // of layer l0
  float* W;
  size_t layer_bytes;               // of K or V
  int num_pages, Hkv, page_shift, row_bytes, nl;
  int B, keep, first, recent;
  const int *kv_len, *table, *out_table;
  int width, out_width;
  int *kept, *out_len;
};
cudaError_t launch_evict(const EvictLaunch& a, const DeviceInfo& dev, cudaStream_t stream);

}  // namespace cxa
