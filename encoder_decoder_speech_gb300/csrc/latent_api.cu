// The C ABI of the latent cache, of the gathered attention weights and of the eviction by them
// (declared in include/cxa.h): descriptors, argument validation and dispatch. Every check runs
// before any device work is enqueued.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>
#include <new>
#include <string>
#include <vector>

#include "cxa.h"
#include "internal.h"
#include "latent.cuh"
#include "paged_handles.h"

using namespace cxa::api;

struct cxa_latent {
  void* Cp;
  int num_pages, page_size, page_shift, L, latent, rope;
  int dtype;
};

namespace {

int check_latent_batch(const std::string& w, const cxa_latent* c, int layer, int B, int n_tokens, const int* q_start,
                       const int* kv_len, const int* page_table, int max_pages) {
  if (c == nullptr) return fail(CXA_EINVAL, w + ": latent descriptor is NULL");
  return check_table(w, c->L, c->page_shift, layer, B, n_tokens, q_start, kv_len, page_table, max_pages);
}

cxa::LatentLayer latent_layer(const cxa_latent* c, int layer) {
  const size_t bytes = static_cast<size_t>(c->num_pages) * c->page_size * (c->latent + c->rope) * elt(c->dtype);
  cxa::LatentLayer l;
  l.C = static_cast<uint8_t*>(c->Cp) + bytes * layer;
  l.num_pages = c->num_pages;
  l.page_shift = c->page_shift;
  l.latent = c->latent;
  l.rope = c->rope;
  return l;
}

bool valid_page_size(int n) { return n >= 16 && n <= 256 && (n & (n - 1)) == 0; }
bool valid_latent(int n) { return n >= 128 && n <= 512 && n % 128 == 0; }

int check_scale(const std::string& w, float scale) {
  if (!std::isfinite(scale) || (scale > 0.f && !std::isfinite(scale * 1.4426950408889634f)))
    return fail(CXA_EINVAL, w + ": scale must be finite, log2(e) times it too");
  return CXA_OK;
}

int check_workspace(const std::string& w, const void* p, size_t bytes, size_t need) {
  if (p == nullptr || !aligned(p, 256))
    return fail(CXA_EINVAL, w + ": the workspace is NULL or not 256-byte aligned");
  if (bytes < need) return fail(CXA_EINVAL, w + ": workspace smaller than " + w + "_workspace_bytes()");
  return CXA_OK;
}

cxa::WeightsWorkspace weights_workspace_of(const cxa_pages* pages, int B, int n_tokens, int max_new, int max_pages,
                                           int Hq) {
  if (pages == nullptr || B < 1 || B > 1 << 30 || n_tokens < 0 || max_new < 1 || max_pages < 1 ||
      static_cast<long long>(max_pages) << pages->page_shift > (1LL << 30) || Hq < 1 || Hq > 65535 ||
      Hq % pages->Hkv != 0)
    return {0, 0};
  return cxa::weights_workspace(B, n_tokens, max_pages, pages->page_shift, pages->num_pages, Hq, pages->Hkv, max_new,
                                pages->dtype == CXA_BF16);
}

}  // namespace

extern "C" {

int cxa_latent_create(cxa_latent** out, void* Cp, int num_pages, int page_size, int L, int latent, int rope,
                      int cache_dtype) {
  return guarded([&]() -> int {
    const std::string w = "cxa_latent_create";
    if (out == nullptr) return fail(CXA_EINVAL, w + ": out is NULL");
    *out = nullptr;
    if (Cp == nullptr || !aligned(Cp, 16)) return fail(CXA_EINVAL, w + ": Cp is NULL or not 16-byte aligned");
    if (!valid_page_size(page_size)) return fail(CXA_EINVAL, w + ": page_size must be 16, 32, 64, 128 or 256");
    if (num_pages < 1 || L < 1 || L > 65535)
      return fail(CXA_EINVAL, w + ": num_pages and L must be positive, L at most 65535");
    if (!valid_latent(latent)) return fail(CXA_EINVAL, w + ": latent must be 128, 256, 384 or 512");
    if (rope < 0 || rope > 64 || rope % 16 != 0) return fail(CXA_EINVAL, w + ": rope must be 0, 16, 32, 48 or 64");
    if (!valid_dtype(cache_dtype)) return fail(CXA_EINVAL, w + ": cache_dtype must be CXA_F32 or CXA_BF16");
    cxa_latent* c = new (std::nothrow) cxa_latent;
    if (c == nullptr) return fail(CXA_EINVAL, w + ": out of host memory");
    c->Cp = Cp;
    c->num_pages = num_pages;
    c->page_size = page_size;
    c->page_shift = 0;
    while ((1 << c->page_shift) < page_size) ++c->page_shift;
    c->L = L;
    c->latent = latent;
    c->rope = rope;
    c->dtype = cache_dtype;
    *out = c;
    return CXA_OK;
  });
}

void cxa_latent_destroy(cxa_latent* c) { delete c; }

int cxa_latent_check(const cxa_latent* c, int B, int n_tokens, const int* q_start, const int* kv_len,
                     const int* page_table, int max_pages) {
  return guarded([&]() -> int {
    const std::string w = "cxa_latent_check";
    const int rc = check_latent_batch(w, c, 0, B, n_tokens, q_start, kv_len, page_table, max_pages);
    if (rc != CXA_OK) return rc;
    return check_host_batch(w, c->num_pages, c->page_shift, B, n_tokens, q_start, kv_len, page_table, max_pages);
  });
}

int cxa_latent_append(const cxa_latent* cache, int layer, int B, int n_tokens, const int* q_start, const int* kv_len,
                      const int* page_table, int max_pages, const void* c, long long c_stride, const void* kr,
                      long long kr_stride, int norm, float eps, const float* weight, const cxa_rotary* rot, int dtype,
                      void* stream) {
  return guarded([&]() -> int {
    const std::string w = "cxa_latent_append";
    int rc = check_latent_batch(w, cache, layer, B, n_tokens, q_start, kv_len, page_table, max_pages);
    if (rc != CXA_OK) return rc;
    if (!valid_dtype(dtype)) return fail(CXA_EINVAL, w + ": dtype must be CXA_F32 or CXA_BF16");
    if (dtype == CXA_BF16 && cache->dtype == CXA_F32)
      return fail(CXA_EINVAL, w + ": bf16 activations need a bf16 pool");
    rc = check_norm(w, norm, eps, weight, nullptr);
    if (rc != CXA_OK) return rc;
    if (rot != nullptr && 2 * rot->arg.pairs > cache->rope)
      return fail(CXA_EINVAL, w + ": the rotation turns more channels than the rotated part has");
    if (n_tokens == 0) return CXA_OK;
    rc = check_rows(w, "c", c, c_stride, n_tokens, 1, cache->latent, dtype);
    if (rc == CXA_OK && cache->rope > 0) rc = check_rows(w, "kr", kr, kr_stride, n_tokens, 1, cache->rope, dtype);
    if (rc != CXA_OK) return rc;
    std::string msg;
    cxa::DeviceInfo dev;
    cudaError_t e = cxa::current_device_info(&dev, &msg);
    if (e != cudaSuccess) return fail_cuda(e, w + ": " + msg);
    cxa::LatentAppendLaunch a = {};
    a.c = c;
    a.kr = cache->rope > 0 ? kr : nullptr;
    a.c_stride = c_stride;
    a.kr_stride = kr_stride;
    a.weight = weight;
    a.eps = eps;
    a.norm = norm == CXA_NORM_RMS;
    a.act_bf16 = dtype == CXA_BF16;
    a.pool_bf16 = cache->dtype == CXA_BF16;
    a.rot = rotary_arg(rot);
    a.batch = {q_start, kv_len, page_table, B, n_tokens, max_pages};
    a.layer = latent_layer(cache, layer);
    e = cxa::launch_latent_append(a, dev, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail_cuda(e, w + ": launch");
    return CXA_OK;
  });
}

size_t cxa_latent_attention_workspace_bytes(int H, int latent, int max_new, int dtype) {
  if (H < 1 || H > 65535 || !valid_latent(latent) || max_new < 1 || !valid_dtype(dtype)) return 0;
  return cxa::latent_attention_workspace(H, latent, max_new, dtype == CXA_BF16);
}

int cxa_latent_attention(const cxa_latent* cache, int layer, int B, int n_tokens, int max_new, const int* q_start,
                         const int* kv_len, const int* page_table, int max_pages, const void* q, long long q_stride,
                         int H, void* out, long long o_stride, float scale, int dtype, void* workspace,
                         size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    const std::string w = "cxa_latent_attention";
    int rc = check_latent_batch(w, cache, layer, B, n_tokens, q_start, kv_len, page_table, max_pages);
    if (rc != CXA_OK) return rc;
    if (!valid_dtype(dtype) || dtype != cache->dtype)
      return fail(CXA_EINVAL, w + ": dtype must be CXA_F32 or CXA_BF16, and the pool's");
    if (H < 1 || H > 65535) return fail(CXA_EINVAL, w + ": H must lie in [1, 65535]");
    if (max_new < 1) return fail(CXA_EINVAL, w + ": max_new must be positive");
    if (!(scale > 0.f)) return fail(CXA_EINVAL, w + ": scale must be positive");
    rc = check_scale(w, scale);
    if (rc != CXA_OK) return rc;
    if (static_cast<long long>(n_tokens) * H > 0x7FFFFFFFLL - 256)
      return fail(CXA_EINVAL, w + ": too many query rows");
    if (n_tokens == 0) return CXA_OK;
    const int width = cache->latent + cache->rope;
    rc = check_rows(w, "q", q, q_stride, n_tokens, H, width, dtype);
    if (rc == CXA_OK) rc = check_rows(w, "out", out, o_stride, n_tokens, H, cache->latent, dtype);
    if (rc != CXA_OK) return rc;
    // (spans: a row of q holds H * width elements, one of out H * latent)
    const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(out);
    const uintptr_t q1 =
        q0 + static_cast<uintptr_t>(((n_tokens - 1) * q_stride + static_cast<long long>(H) * width) * elt(dtype));
    const uintptr_t o1 = o0 + static_cast<uintptr_t>(
                                  ((n_tokens - 1) * o_stride + static_cast<long long>(H) * cache->latent) * elt(dtype));
    if (q0 < o1 && o0 < q1) return fail(CXA_EINVAL, w + ": out must not overlap q");
    rc = check_workspace(w, workspace, workspace_bytes,
                         cxa_latent_attention_workspace_bytes(H, cache->latent, max_new, dtype));
    if (rc != CXA_OK) return rc;
    const double tiles = static_cast<double>(B) + static_cast<double>(n_tokens) * H / 16.0;
    const double chunks = static_cast<double>((static_cast<long long>(max_pages) << cache->page_shift) / 32 + 1);
    if (tiles * chunks >= 2147483647.0)
      return fail(CXA_EINVAL, w + ": the chunks of keys of all tiles of query rows (see cxa.h) must be below 2^31");
    std::string msg;
    cxa::DeviceInfo dev;
    cudaError_t e = cxa::current_device_info(&dev, &msg);
    if (e != cudaSuccess) return fail_cuda(e, w + ": " + msg);
    cxa::LatentAttnLaunch a = {};
    a.q = q;
    a.out = out;
    a.q_stride = q_stride;
    a.o_stride = o_stride;
    a.H = H;
    a.max_new = max_new;
    a.scale = scale;
    a.bf16 = dtype == CXA_BF16;
    a.batch = {q_start, kv_len, page_table, B, n_tokens, max_pages};
    a.layer = latent_layer(cache, layer);
    a.workspace = workspace;
    const std::lock_guard<std::mutex> together(stream_lock(static_cast<cudaStream_t>(stream)));
    e = cxa::launch_latent_attention(a, dev, static_cast<cudaStream_t>(stream), &msg);
    if (e != cudaSuccess) return fail_cuda(e, w + ": launch " + msg);
    return CXA_OK;
  });
}

int cxa_latent_expand(const cxa_latent* cache, int layer, const cxa_pages* to, int to_layer, int B, const int* from,
                      const int* kv_len, const int* page_table, int max_pages, const int* to_table, int to_max_pages,
                      const void* WK, const void* WV, void* stream) {
  return guarded([&]() -> int {
    const std::string w = "cxa_latent_expand";
    if (to == nullptr) return fail(CXA_EINVAL, w + ": page descriptor is NULL");
    int rc = check_latent_batch(w, cache, layer, B, 0, kv_len, kv_len, page_table, max_pages);
    if (rc == CXA_OK) rc = check_batch(w, to, to_layer, B, 0, kv_len, kv_len, to_table, to_max_pages);
    if (rc != CXA_OK) return rc;
    if (!aligned(from, 4)) return fail(CXA_EINVAL, w + ": from must be 4-byte aligned");
    if (to->dtype != cache->dtype) return fail(CXA_EINVAL, w + ": both pools must be of one type");
    if (cache->rope >= to->dh) return fail(CXA_EINVAL, w + ": rope must be less than the head dim");
    if (WK == nullptr || WV == nullptr || !aligned(WK, 16) || !aligned(WV, 16))
      return fail(CXA_EINVAL, w + ": WK or WV is NULL or not 16-byte aligned");
    const double tiles = static_cast<double>((static_cast<long long>(max_pages) << cache->page_shift) / 64 + 1) * B;
    if (tiles >= 2147483647.0)
      return fail(CXA_EINVAL, w + ": B * (max_pages * page_size / 64 + 1) must be below 2^31");
    std::string msg;
    cxa::DeviceInfo dev;
    cudaError_t e = cxa::current_device_info(&dev, &msg);
    if (e != cudaSuccess) return fail_cuda(e, w + ": " + msg);
    cxa::LatentExpandLaunch a = {};
    a.layer = latent_layer(cache, layer);
    a.to = layer_of(to, to_layer);
    a.dh = to->dh;
    a.bf16 = to->dtype == CXA_BF16;
    a.B = B;
    a.from = from;
    a.kv_len = kv_len;
    a.table = page_table;
    a.to_table = to_table;
    a.width = max_pages;
    a.to_width = to_max_pages;
    a.WK = WK;
    a.WV = WV;
    e = cxa::launch_latent_expand(a, dev, static_cast<cudaStream_t>(stream), &msg);
    if (e != cudaSuccess) return fail_cuda(e, w + ": launch " + msg);
    return CXA_OK;
  });
}

size_t cxa_paged_weights_workspace_bytes(const cxa_pages* pages, int B, int n_tokens, int max_new, int max_pages,
                                         int Hq) {
  return weights_workspace_of(pages, B, n_tokens, max_new, max_pages, Hq).least;
}

size_t cxa_paged_weights_room_bytes(const cxa_pages* pages, int B, int n_tokens, int max_new, int max_pages, int Hq) {
  return weights_workspace_of(pages, B, n_tokens, max_new, max_pages, Hq).most;
}

int cxa_paged_weights(const cxa_pages* pages, int layer, int B, int n_tokens, int max_new, const int* q_start,
                      const int* kv_len, const int* page_table, int max_pages, const void* q, long long q_stride,
                      int Hq, float* weights, float decay, float scale, int dtype, void* workspace,
                      size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    const std::string w = "cxa_paged_weights";
    int rc = check_batch(w, pages, layer, B, n_tokens, q_start, kv_len, page_table, max_pages);
    if (rc != CXA_OK) return rc;
    if (!valid_dtype(dtype) || dtype != pages->dtype)
      return fail(CXA_EINVAL, w + ": dtype must be CXA_F32 or CXA_BF16, and the pool's");
    if (Hq < 1 || Hq > 65535 || Hq % pages->Hkv != 0)
      return fail(CXA_EINVAL, w + ": Hq must be a positive multiple of the pool's K/V heads, at most 65535");
    if (max_new < 1) return fail(CXA_EINVAL, w + ": max_new must be positive");
    if (static_cast<long long>(n_tokens) * (Hq / pages->Hkv) > 0x7FFFFFFFLL - 256)
      return fail(CXA_EINVAL, w + ": too many query rows");
    if (!std::isfinite(decay) || decay < 0.f) return fail(CXA_EINVAL, w + ": decay must be finite and >= 0");
    rc = check_scale(w, scale);
    if (rc != CXA_OK) return rc;
    if (n_tokens == 0) return CXA_OK;
    rc = check_rows(w, "q", q, q_stride, n_tokens, Hq, pages->dh, dtype);
    if (rc != CXA_OK) return rc;
    if (weights == nullptr || !aligned(weights, 4))
      return fail(CXA_EINVAL, w + ": weights is NULL or not 4-byte aligned");
    rc = check_workspace(w, workspace, workspace_bytes,
                         cxa_paged_weights_workspace_bytes(pages, B, n_tokens, max_new, max_pages, Hq));
    if (rc != CXA_OK) return rc;
    const cxa::PagedBatch batch = {q_start, kv_len, page_table, B, n_tokens, max_pages};
    if (!cxa::weights_countable(batch, pages->page_shift, pages->Hkv, Hq / pages->Hkv, dtype == CXA_BF16))
      return fail(CXA_EINVAL, w + ": the chunks of keys of all tiles of query rows (see cxa.h) must be below 2^31");
    std::string msg;
    cxa::DeviceInfo dev;
    cudaError_t e = cxa::current_device_info(&dev, &msg);
    if (e != cudaSuccess) return fail_cuda(e, w + ": " + msg);
    cxa::WeightsLaunch a = {};
    a.q = q;
    a.q_stride = q_stride;
    a.Hq = Hq;
    a.dh = pages->dh;
    a.max_new = max_new;
    a.weights = weights + static_cast<size_t>(layer) * pages->num_pages * pages->Hkv * pages->page_size;
    a.decay = decay;
    a.scale = scale > 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(pages->dh));
    a.bf16 = dtype == CXA_BF16;
    a.batch = batch;
    a.layer = layer_of(pages, layer);
    a.workspace = workspace;
    a.workspace_bytes = workspace_bytes;
    const std::lock_guard<std::mutex> together(stream_lock(static_cast<cudaStream_t>(stream)));
    e = cxa::launch_weights(a, dev, static_cast<cudaStream_t>(stream), &msg);
    if (e != cudaSuccess) return fail_cuda(e, w + ": launch " + msg);
    return CXA_OK;
  });
}

int cxa_paged_evict(const cxa_pages* pages, int l0, int nl, float* weights, int B, int keep, int first, int recent,
                    const int* kv_len, const int* page_table, int max_pages, const int* out_table, int out_max_pages,
                    int* kept, int* out_len, void* stream) {
  return guarded([&]() -> int {
    const std::string w = "cxa_paged_evict";
    int rc = check_batch(w, pages, l0, B, 0, kv_len, kv_len, page_table, max_pages);
    if (rc == CXA_OK) rc = check_batch(w, pages, l0, B, 0, kv_len, kv_len, out_table, out_max_pages);
    if (rc != CXA_OK) return rc;
    if (nl < 1 || nl > pages->L - l0) return fail(CXA_EINVAL, w + ": layers out of range");
    if (keep < 1 || first < 0 || recent < 0 || static_cast<long long>(first) + recent > keep)
      return fail(CXA_EINVAL, w + ": keep must be positive and hold first and recent, which must not be negative");
    if (weights == nullptr || kept == nullptr || out_len == nullptr || !aligned(weights, 4) || !aligned(kept, 4) ||
        !aligned(out_len, 4))
      return fail(CXA_EINVAL, w + ": weights, kept or out_len is NULL or not 4-byte aligned");
    const uintptr_t o0 = reinterpret_cast<uintptr_t>(out_len), k0 = reinterpret_cast<uintptr_t>(kv_len);
    if (o0 < k0 + static_cast<uintptr_t>(B) * 4 && k0 < o0 + static_cast<uintptr_t>(B) * 4)
      return fail(CXA_EINVAL, w + ": out_len must not overlap kv_len");
    const double rows = static_cast<double>(nl) * B * pages->Hkv;
    if (rows * (static_cast<double>(keep) / 32.0 + 8.0) >= 2147483647.0)
      return fail(CXA_EINVAL, w + ": nl * B * Hkv * (keep / 32 + 8) must be below 2^31");
    std::string msg;
    cxa::DeviceInfo dev;
    cudaError_t e = cxa::current_device_info(&dev, &msg);
    if (e != cudaSuccess) return fail_cuda(e, w + ": " + msg);
    const cxa::PagedLayer l = layer_of(pages, l0);
    cxa::EvictLaunch a = {};
    a.K = l.K;
    a.V = l.V;
    a.W = weights + static_cast<size_t>(l0) * pages->num_pages * pages->Hkv * pages->page_size;
    a.row_bytes = pages->dh * elt(pages->dtype);
    a.layer_bytes = static_cast<size_t>(pages->num_pages) * pages->Hkv * pages->page_size * a.row_bytes;
    a.num_pages = pages->num_pages;
    a.Hkv = pages->Hkv;
    a.page_shift = pages->page_shift;
    a.nl = nl;
    a.B = B;
    a.keep = keep;
    a.first = first;
    a.recent = recent;
    a.kv_len = kv_len;
    a.table = page_table;
    a.out_table = out_table;
    a.width = max_pages;
    a.out_width = out_max_pages;
    a.kept = kept;
    a.out_len = out_len;
    const std::lock_guard<std::mutex> together(stream_lock(static_cast<cudaStream_t>(stream)));
    e = cxa::launch_evict(a, dev, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail_cuda(e, w + ": launch");
    return CXA_OK;
  });
}

int cxa_paged_evict_check(const cxa_pages* pages, int B, int keep, const int* kv_len, const int* page_table,
                          int max_pages, const int* out_table, int out_max_pages) {
  return guarded([&]() -> int {
    const std::string w = "cxa_paged_evict_check";
    int rc = check_batch(w, pages, 0, B, 0, kv_len, kv_len, page_table, max_pages);
    if (rc == CXA_OK) rc = check_batch(w, pages, 0, B, 0, kv_len, kv_len, out_table, out_max_pages);
    if (rc != CXA_OK) return rc;
    if (keep < 1) return fail(CXA_EINVAL, w + ": keep must be positive");
    const int shift = pages->page_shift;
    std::vector<char> use(static_cast<size_t>(pages->num_pages), 0);     // 1: read, 2: written
    for (int pass = 0; pass < 2; ++pass)
      for (int b = 0; b < B; ++b) {
        const std::string at = " (sequence " + std::to_string(b) + ")";
        if (kv_len[b] < 0 || kv_len[b] > max_pages << shift)
          return fail(CXA_EINVAL, w + ": kv_len is negative or passes the table's row" + at);
        const int n = pass == 0 || kv_len[b] < keep ? kv_len[b] : keep, width = pass == 0 ? max_pages : out_max_pages;
        if (n > width << shift) return fail(CXA_EINVAL, w + ": what stays passes the row of out_table" + at);
        const int* row = (pass == 0 ? page_table : out_table) + static_cast<size_t>(b) * width;
        for (int t = 0; t < n; t += 1 << shift) {
          const int page = cxa::paged_lookup(row, width, shift, pages->num_pages, t);
          if (page < 0)
            return fail(CXA_EINVAL, w + (pass == 0 ? ": page_table entry " : ": out_table entry ") +
                                        std::to_string(t >> shift) + " is not a page of the pool" + at);
          char& u = use[static_cast<size_t>(page)];
          if (pass == 1 && u == 1) return fail(CXA_EINVAL, w + ": a page of out_table is still read" + at);
          if (pass == 1 && u == 2) return fail(CXA_EINVAL, w + ": a page of out_table is written twice" + at);
          u = pass == 0 ? 1 : 2;
        }
      }
    return CXA_OK;
  });
}

}  // extern "C"
