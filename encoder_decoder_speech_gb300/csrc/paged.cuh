// What the paged self-attention kernels share: the batch of new tokens, the pages of
// a layer, and the look-up of a key's row (also run on the host by cxa_paged_check).
#pragma once

#include <cstddef>
#include <cstdint>
#include <string>

#include <cuda.h>
#include <cuda_runtime.h>

#include "internal.h"

namespace cxa {

constexpr int kMaxRotaryPairs = 64;

// A rotation, passed by value as a kernel parameter. step[i] is the turn of pair i per
// position in units of 2^-64 turns: position * step modulo 2^64 is the pair's phase with
// whole turns dropped exactly, so a far position costs no precision (an error of at most
// |position| * 2^-65 turns), where position * frequency in fp32 would lose it all.
struct RotaryArg {
  unsigned long long step[kMaxRotaryPairs];
  float factor;       // multiplies the rotated values
  int pairs;          // rotated pairs; 0: no rotation
  int interleaved;    // pair i is (2i, 2i + 1); otherwise (i, i + pairs)
};

// The new tokens of a batch, packed: sequence b owns rows q_start[b] .. q_start[b + 1),
// the last of them at position kv_len[b] - 1. All pointers are device pointers.
struct PagedBatch {
  const int* q_start;
  const int* kv_len;
  const int* table;      // [B][width] page numbers
  int B, n_tokens, width;
};

// One layer of the pool: [num_pages][Hkv][1 << page_shift][dh].
struct PagedLayer {
  void* K;
  void* V;
  int num_pages, Hkv, page_shift;
};

struct PagedSeq {
  int q0, n;     // first row and number of new tokens
  int kv;        // keys after them
};

__host__ __device__ inline PagedSeq paged_seq(const int* q_start, const int* kv_len, int b, int n_tokens) {
  PagedSeq s;
  const int lo = q_start[b], hi = q_start[b + 1];
  s.q0 = lo < 0 ? 0 : lo > n_tokens ? n_tokens : lo;
  const int q1 = hi < 0 ? 0 : hi > n_tokens ? n_tokens : hi;
  s.n = q1 > s.q0 ? q1 - s.q0 : 0;
  s.kv = kv_len[b] > 0 ? kv_len[b] : 0;
  return s;
}

// The page that holds position t of a sequence, or -1 if t lies outside the table's
// row or the entry outside the pool.
__host__ __device__ inline int paged_lookup(const int* table_row, int width, int page_shift, int num_pages, int t) {
  if (t < 0 || (t >> page_shift) >= width) return -1;
  const int page = table_row[t >> page_shift];
  return page >= 0 && page < num_pages ? page : -1;
}

// Bits of the device status word.
constexpr unsigned int kStatusTimeout = 1u, kStatusBadPage = 2u, kStatusBadBatch = 4u;

struct NormRopeLaunch {
  const void *q, *k, *v;            // k, v may be null; v only with pages
  long long q_stride, k_stride, v_stride;      // elements from one token's row to the next
  void *q_out, *k_out;              // k_out unused with pages
  long long qo_stride, ko_stride;
  int Hq, Hk, dh, n_tokens;
  const int* pos;                   // [n_tokens], without pages
  const float *wq, *wk;             // [dh] or NULL (1)
  float eps;
  bool norm;
  bool act_bf16, pool_bf16;
  RotaryArg rot;
  bool append;                      // write k and v into the layer's pages
  PagedBatch batch;
  PagedLayer layer;
};

struct PagedAttnLaunch {
  const void* q;
  void* out;
  long long q_stride, o_stride;     // elements
  int Hq, dh, max_new;
  float scale;
  bool act_bf16, pool_bf16;
  PagedBatch batch;
  PagedLayer layer;
  void* workspace;
};

// Lets a kernel use `bytes` of dynamic shared memory, as much of it on an SM as there is;
// once a device (done: a static of the caller's, one a kernel).
struct SmemOnce {
  unsigned char done[128];
};
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, int device, SmemOnce* once) {
  const bool known = device >= 0 && device < 128;
  if (known && once->done[device]) return cudaSuccess;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  if (e == cudaSuccess && known) once->done[device] = 1;    // (two threads may both come here: no harm)
  return e;
}

cudaError_t launch_norm_rope(const NormRopeLaunch& a, const DeviceInfo& dev, cudaStream_t stream);

// Attention, one kernel or two: sequences of up to kFewRows query rows a K/V head go to
// paged_rows.cu, the others, where paged_tile_takes(), to paged_tile.cu; the first kernel
// takes all of them otherwise. Both sides of the border, in us for 16 sequences, 8 K/V heads of
// 64 channels, bf16 (few-rows kernel / tile kernel): over 32768 keys 16 rows 173 / 247, 20 rows
// 323 / 249, 64 rows 637 / 248; 128 channels 326 / 436, 630 / 439, 1216 / 438: from 17 rows on the
// few-rows kernel reads the keys once more. Over 1024 keys, which L2 holds, it stays ahead to some
// 40 rows (25 / 27; 128 channels 32 rows 29 / 34), one sequence over 32768 keys to 40 (37 / 41).
constexpr int kFewRows = 16;
// The workspace: both kernels' arrival counters, at places that no argument moves (so that calls
// of different shapes may share it), then the partial states of the first and of the second.
constexpr int kRowsMaxBlocks = 160 * 4, kTileMaxBlocks = 160;
constexpr size_t kRowsCounters = kRowsMaxBlocks * 3, kTileCounters = kTileMaxBlocks * 2 * 3;
constexpr size_t kPagedCounterBytes = (kRowsCounters + kTileCounters) * 4;
static_assert(kPagedCounterBytes % 256 == 0, "the partial states behind the counters are aligned");
size_t paged_rows_part_bytes(int dh);
// Whether the work of each kernel can be numbered in 31 bits.
bool paged_rows_countable(const PagedAttnLaunch& a, int max_rows);
bool paged_tile_countable(const PagedAttnLaunch& a);
cudaError_t launch_paged_rows(const PagedAttnLaunch& a, int max_rows, const DeviceInfo& dev, cudaStream_t stream);
bool paged_tile_takes(int G, bool act_bf16, int max_new);
size_t paged_tile_part_bytes(int dh);
// The tensor maps of q and of the layer's pages, made before anything of the call is enqueued.
struct PagedTileMaps {
  CUtensorMap q, k, v;
};
cudaError_t prepare_paged_tile(const PagedAttnLaunch& a, const DeviceInfo& dev, PagedTileMaps* maps, std::string* msg);
cudaError_t launch_paged_tile(const PagedAttnLaunch& a, const PagedTileMaps& maps, const DeviceInfo& dev,
                              cudaStream_t stream);

}  // namespace cxa
