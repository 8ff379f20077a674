// What the C-ABI files of the paged caches share: the handles behind the descriptors, errors, and
// the checks of arguments that every call makes before it enqueues anything.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>
#include <string>

#include "cxa.h"
#include "internal.h"
#include "paged.cuh"

struct cxa_rotary {
  cxa::RotaryArg arg;
};

struct cxa_pages {
  void* Kp;
  void* Vp;
  int num_pages, page_size, page_shift, L, Hkv, dh;
  int dtype;
};

namespace cxa {
namespace api {

inline int fail(int code, const std::string& msg) {
  cxa::set_last_error(msg);
  return code;
}

inline int fail_cuda(cudaError_t e, const std::string& what) {
  cxa::set_last_error(what + ": " + cudaGetErrorName(e) + " (" + cudaGetErrorString(e) + ")");
  return CXA_ECUDA;
}

// Runs a call's body; nothing thrown in it (host memory for a message or a list) leaves the
// C entry point.
template <typename F>
int guarded(F body) noexcept {
  try {
    return body();
  } catch (...) {
    return CXA_EINVAL;
  }
}

// Held while a call of several kernels, or of one that works on a workspace, is enqueued, so that nothing of
// another thread's call on the same stream comes between its kernels: they hand scratch to each other in a workspace
// that calls of one stream may share, and the second kernel of the paged attention starts without waiting for
// anything but the first (paged_tile.cu). One lock for the streams whose handles fall together.
std::mutex& stream_lock(cudaStream_t s);

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool valid_dtype(int t) { return t == CXA_F32 || t == CXA_BF16; }
inline int elt(int t) { return t == CXA_BF16 ? 2 : 4; }

// A packed tensor of rows: one token's heads contiguous, tokens `stride` elements apart. A
// tensor map's strides are below 2^40 bytes, whichever kernel a call goes to.
inline int check_rows(const std::string& w, const char* name, const void* p, long long stride, int rows, int H,
                      int dh, int dtype) {
  if (p == nullptr) return fail(CXA_EINVAL, w + ": " + name + " is NULL");
  if (!aligned(p, 16)) return fail(CXA_EINVAL, w + ": " + name + " must be 16-byte aligned");
  if (stride < static_cast<long long>(H) * dh || stride >= (1LL << 40) / elt(dtype) || stride * elt(dtype) % 16 != 0)
    return fail(CXA_EINVAL, w + ": the row stride of " + name +
                                " must hold its heads, be a multiple of 16 bytes and below 2^40 bytes");
  if (static_cast<double>(rows) * static_cast<double>(stride) * elt(dtype) > 72057594037927936.0)
    return fail(CXA_EINVAL, w + ": the rows of " + name + " span more than 2^56 bytes");
  return CXA_OK;
}

// Whether the spans of two packed tensors, first row to last, meet.
inline bool overlap(const void* a, long long sa, const void* b, long long sb, long long rows, int Ha, int Hb, int dh,
                    int es) {
  if (rows <= 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  const uintptr_t a1 = a0 + static_cast<uintptr_t>(((rows - 1) * sa + static_cast<long long>(Ha) * dh) * es);
  const uintptr_t b1 = b0 + static_cast<uintptr_t>(((rows - 1) * sb + static_cast<long long>(Hb) * dh) * es);
  return a0 < b1 && b0 < a1;
}

inline int check_norm(const std::string& w, int norm, float eps, const float* wq, const float* wk) {
  if (norm != CXA_NORM_NONE && norm != CXA_NORM_RMS)
    return fail(CXA_EINVAL, w + ": norm must be CXA_NORM_NONE or CXA_NORM_RMS");
  if (norm == CXA_NORM_RMS && (!std::isfinite(eps) || eps < 0.f))
    return fail(CXA_EINVAL, w + ": eps must be finite and >= 0");
  if (!aligned(wq, 4) || !aligned(wk, 4)) return fail(CXA_EINVAL, w + ": the norm weights must be 4-byte aligned");
  return CXA_OK;
}

inline int check_rotary(const std::string& w, const cxa_rotary* rot, int dh) {
  if (rot != nullptr && 2 * rot->arg.pairs > dh)
    return fail(CXA_EINVAL, w + ": the rotation turns more channels than a head has");
  return CXA_OK;
}

// A batch over the pages of a pool of L layers.
inline int check_table(const std::string& w, int L, int page_shift, int layer, int B, int n_tokens, const int* q_start,
                       const int* kv_len, const int* page_table, int max_pages) {
  if (layer < 0 || layer >= L) return fail(CXA_EINVAL, w + ": layer out of range");
  if (B < 1 || n_tokens < 0 || max_pages < 1)
    return fail(CXA_EINVAL, w + ": B and max_pages must be positive, n_tokens not negative");
  if (B > 1 << 30) return fail(CXA_EINVAL, w + ": B must be at most 2^30");
  if (static_cast<long long>(max_pages) << page_shift > (1LL << 30))
    return fail(CXA_EINVAL, w + ": a table row may span at most 2^30 positions");
  if (q_start == nullptr || kv_len == nullptr || page_table == nullptr)
    return fail(CXA_EINVAL, w + ": a pointer argument is NULL");
  if (!aligned(q_start, 4) || !aligned(kv_len, 4) || !aligned(page_table, 4))
    return fail(CXA_EINVAL, w + ": q_start, kv_len and page_table must be 4-byte aligned");
  return CXA_OK;
}

inline int check_batch(const std::string& w, const cxa_pages* pages, int layer, int B, int n_tokens,
                       const int* q_start, const int* kv_len, const int* page_table, int max_pages) {
  if (pages == nullptr) return fail(CXA_EINVAL, w + ": page descriptor is NULL");
  return check_table(w, pages->L, pages->page_shift, layer, B, n_tokens, q_start, kv_len, page_table, max_pages);
}

// A batch on the host, sound or not (cxa_paged_check).
int check_host_batch(const std::string& w, int num_pages, int page_shift, int B, int n_tokens, const int* q_start,
                     const int* kv_len, const int* page_table, int max_pages);

inline cxa::PagedLayer layer_of(const cxa_pages* pages, int layer) {
  const size_t bytes = static_cast<size_t>(pages->num_pages) * pages->Hkv * pages->page_size * pages->dh *
                       elt(pages->dtype) * layer;
  cxa::PagedLayer l;
  l.K = static_cast<uint8_t*>(pages->Kp) + bytes;
  l.V = static_cast<uint8_t*>(pages->Vp) + bytes;
  l.num_pages = pages->num_pages;
  l.Hkv = pages->Hkv;
  l.page_shift = pages->page_shift;
  return l;
}

inline cxa::RotaryArg rotary_arg(const cxa_rotary* rot) {
  if (rot != nullptr) return rot->arg;
  cxa::RotaryArg none = {};
  none.factor = 1.f;
  return none;
}

}  // namespace api
}  // namespace cxa
