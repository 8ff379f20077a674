// The C ABI of the paged self-attention cache (declared in include/cxa.h): rotations, the
// page-pool descriptor, argument validation, and dispatch to the kernel files. Every
// check runs before any device work is enqueued.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <exception>
#include <mutex>
#include <new>
#include <string>
#include <vector>

#include "cxa.h"
#include "internal.h"
#include "paged.cuh"
#include "paged_handles.h"

static_assert(cxa::kPagedCounterBytes == CXA_PAGED_COUNTER_BYTES, "what a caller has to clear");

using namespace cxa::api;

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

}  // namespace

namespace cxa {
namespace api {

std::mutex& stream_lock(cudaStream_t s) {
  static std::mutex locks[61];
  return locks[reinterpret_cast<uintptr_t>(s) / 16 % 61];
}

int check_host_batch(const std::string& w, int num_pages, int page_shift, int B, int n_tokens, const int* q_start,
                     const int* kv_len, const int* page_table, int max_pages) {
  if (q_start[0] != 0) return fail(CXA_EINVAL, w + ": q_start[0] must be 0");
  for (int b = 0; b < B; ++b)
    if (q_start[b + 1] < q_start[b] || q_start[b + 1] > n_tokens)
      return fail(CXA_EINVAL, w + ": q_start must not decrease or pass n_tokens (sequence " + std::to_string(b) + ")");
  std::vector<int> writer(static_cast<size_t>(num_pages), -1);
  for (int pass = 0; pass < 2; ++pass)
    for (int b = 0; b < B; ++b) {
      const std::string at = " (sequence " + std::to_string(b) + ")";
      const cxa::PagedSeq s = cxa::paged_seq(q_start, kv_len, b, n_tokens);
      if (s.n == 0) continue;
      if (kv_len[b] < s.n) return fail(CXA_EINVAL, w + ": kv_len is less than the new tokens" + at);
      if (s.kv > max_pages << page_shift)
        return fail(CXA_EINVAL, w + ": kv_len passes the table's row" + at);
      const int* row = page_table + static_cast<size_t>(b) * max_pages;
      const int first_new = (s.kv - s.n) >> page_shift;
      for (int t = 0; t < s.kv; t += 1 << page_shift) {
        const int page = cxa::paged_lookup(row, max_pages, page_shift, num_pages, t);
        if (page < 0)
          return fail(CXA_EINVAL, w + ": page_table entry " + std::to_string(t >> page_shift) +
                                      " is not a page of the pool" + at);
        int& who = writer[static_cast<size_t>(page)];
        if (pass == 0 && (t >> page_shift) >= first_new) {
          if (who != -1) return fail(CXA_EINVAL, w + ": two sequences or positions write one page" + at);
          who = b;
        }
        if (pass == 1 && who != -1 && (who != b || (t >> page_shift) < first_new))
          return fail(CXA_EINVAL, w + ": a page that holds one sequence's new tokens is another's" + at);
      }
    }
  return CXA_OK;
}

}  // namespace api
}  // namespace cxa

extern "C" {

int cxa_rotary_frequencies(int rot_dim, double base, int scaling, double factor, double orig_len, double alpha,
                           double beta, double* freq, double* attn_factor) {
  return guarded([&]() -> int {
    const std::string w = "cxa_rotary_frequencies";
    if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > 2 * cxa::kMaxRotaryPairs)
      return fail(CXA_EINVAL, w + ": rot_dim must be even, 2 .. 128");
    if (freq == nullptr || attn_factor == nullptr) return fail(CXA_EINVAL, w + ": a pointer argument is NULL");
    if (!std::isfinite(base) || base <= 1.0) return fail(CXA_EINVAL, w + ": base must be finite and > 1");
    if (scaling < CXA_ROTARY_PLAIN || scaling > CXA_ROTARY_WAVELENGTH)
      return fail(CXA_EINVAL, w + ": unknown scaling");
    if (scaling != CXA_ROTARY_PLAIN && (!std::isfinite(factor) || factor < 1.0))
      return fail(CXA_EINVAL, w + ": factor must be finite and >= 1");
    if (scaling == CXA_ROTARY_WAVELENGTH &&
        (!std::isfinite(orig_len) || orig_len <= 0.0 || !std::isfinite(alpha) || !std::isfinite(beta) ||
         alpha < 0.0 || beta <= alpha))
      return fail(CXA_EINVAL, w + ": needs orig_len > 0 and 0 <= alpha < beta");
    double b = base;
    if (scaling == CXA_ROTARY_NTK && rot_dim > 2) b = base * std::pow(factor, rot_dim / (rot_dim - 2.0));
    for (int i = 0; i < rot_dim / 2; ++i) {
      double f = std::pow(b, -2.0 * i / rot_dim);
      if (scaling == CXA_ROTARY_LINEAR) f /= factor;
      if (scaling == CXA_ROTARY_WAVELENGTH) {
        const double turns = orig_len * f / kTwoPi;
        double keep = (turns - alpha) / (beta - alpha);
        keep = keep < 0.0 ? 0.0 : keep > 1.0 ? 1.0 : keep;
        f = f * keep + f / factor * (1.0 - keep);
      }
      freq[i] = f;
    }
    *attn_factor = scaling == CXA_ROTARY_WAVELENGTH ? 0.1 * std::log(factor) + 1.0 : 1.0;
    return CXA_OK;
  });
}

int cxa_rotary_create(cxa_rotary** out, int rot_dim, int layout, const double* freq, double attn_factor) {
  return guarded([&]() -> int {
    const std::string w = "cxa_rotary_create";
    if (out == nullptr) return fail(CXA_EINVAL, w + ": out is NULL");
    *out = nullptr;
    if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > 2 * cxa::kMaxRotaryPairs)
      return fail(CXA_EINVAL, w + ": rot_dim must be even, 2 .. 128");
    if (layout != CXA_ROTARY_HALF && layout != CXA_ROTARY_INTERLEAVED)
      return fail(CXA_EINVAL, w + ": layout must be CXA_ROTARY_HALF or CXA_ROTARY_INTERLEAVED");
    if (freq == nullptr) return fail(CXA_EINVAL, w + ": freq is NULL");
    if (!std::isfinite(attn_factor) || !std::isfinite(static_cast<float>(attn_factor)))
      return fail(CXA_EINVAL, w + ": attn_factor must be finite in fp32");
    for (int i = 0; i < rot_dim / 2; ++i)
      if (!std::isfinite(freq[i]) || freq[i] < 0.0)
        return fail(CXA_EINVAL, w + ": frequencies must be finite and >= 0");
    cxa_rotary* r = new (std::nothrow) cxa_rotary;
    if (r == nullptr) return fail(CXA_EINVAL, w + ": out of host memory");
    r->arg = cxa::RotaryArg{};
    for (int i = 0; i < rot_dim / 2; ++i) {
      // whole turns a position do not show; the rest in units of 2^-64 turns
      double turns = freq[i] / kTwoPi;
      turns -= std::floor(turns);
      const double units = std::nearbyint(std::ldexp(turns, 64));
      r->arg.step[i] = units >= 18446744073709551616.0 ? 0ull : static_cast<unsigned long long>(units);
    }
    r->arg.factor = static_cast<float>(attn_factor);
    r->arg.pairs = rot_dim / 2;
    r->arg.interleaved = layout == CXA_ROTARY_INTERLEAVED;
    *out = r;
    return CXA_OK;
  });
}

void cxa_rotary_destroy(cxa_rotary* r) { delete r; }

int cxa_qk_norm_rope(const void* q, long long q_stride, int Hq, const void* k, long long k_stride, int Hk, int dh,
                     int n_tokens, const int* pos, int norm, float eps, const float* q_weight, const float* k_weight,
                     const cxa_rotary* rot, void* q_out, long long qo_stride, void* k_out, long long ko_stride,
                     int dtype, void* stream) {
  return guarded([&]() -> int {
    const std::string w = "cxa_qk_norm_rope";
    if (dh != 64 && dh != 128) return fail(CXA_EINVAL, w + ": head_dim must be 64 or 128");
    if (!valid_dtype(dtype)) return fail(CXA_EINVAL, w + ": dtype must be CXA_F32 or CXA_BF16");
    if (Hq < 0 || Hk < 0 || Hq > 65535 || Hk > 65535 || Hq + Hk == 0 || n_tokens < 0)
      return fail(CXA_EINVAL, w + ": Hq and Hk must lie in [0, 65535], not both 0, and n_tokens not be negative");
    int rc = check_norm(w, norm, eps, q_weight, k_weight);
    if (rc == CXA_OK) rc = check_rotary(w, rot, dh);
    if (rc != CXA_OK) return rc;
    if (n_tokens == 0) return CXA_OK;
    if (pos == nullptr || !aligned(pos, 4)) return fail(CXA_EINVAL, w + ": pos is NULL or misaligned");
    if (Hq > 0) rc = check_rows(w, "q", q, q_stride, n_tokens, Hq, dh, dtype);
    if (rc == CXA_OK && Hq > 0) rc = check_rows(w, "q_out", q_out, qo_stride, n_tokens, Hq, dh, dtype);
    if (rc == CXA_OK && Hk > 0) rc = check_rows(w, "k", k, k_stride, n_tokens, Hk, dh, dtype);
    if (rc == CXA_OK && Hk > 0) rc = check_rows(w, "k_out", k_out, ko_stride, n_tokens, Hk, dh, dtype);
    if (rc != CXA_OK) return rc;
    std::string msg;
    cxa::DeviceInfo dev;
    cudaError_t e = cxa::current_device_info(&dev, &msg);
    if (e != cudaSuccess) return fail_cuda(e, w + ": " + msg);
    cxa::NormRopeLaunch a = {};
    a.q = q;
    a.k = k;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.q_out = q_out;
    a.k_out = k_out;
    a.qo_stride = qo_stride;
    a.ko_stride = ko_stride;
    a.Hq = Hq;
    a.Hk = Hk;
    a.dh = dh;
    a.n_tokens = n_tokens;
    a.pos = pos;
    a.wq = q_weight;
    a.wk = k_weight;
    a.eps = eps;
    a.norm = norm == CXA_NORM_RMS;
    a.act_bf16 = a.pool_bf16 = dtype == CXA_BF16;
    a.rot = rotary_arg(rot);
    e = cxa::launch_norm_rope(a, dev, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail_cuda(e, w + ": launch");
    return CXA_OK;
  });
}

int cxa_pages_create(cxa_pages** out, void* Kp, void* Vp, int num_pages, int page_size, int L, int Hkv, int dh,
                     int cache_dtype) {
  return guarded([&]() -> int {
    const std::string w = "cxa_pages_create";
    if (out == nullptr) return fail(CXA_EINVAL, w + ": out is NULL");
    *out = nullptr;
    if (Kp == nullptr || Vp == nullptr) return fail(CXA_EINVAL, w + ": Kp or Vp is NULL");
    if (!aligned(Kp, 16) || !aligned(Vp, 16)) return fail(CXA_EINVAL, w + ": Kp and Vp must be 16-byte aligned");
    if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)) != 0)
      return fail(CXA_EINVAL, w + ": page_size must be 16, 32, 64, 128 or 256");
    if (num_pages < 1 || L < 1 || Hkv < 1 || L > 65535 || Hkv > 65535)
      return fail(CXA_EINVAL, w + ": num_pages, L and Hkv must be positive, L and Hkv at most 65535");
    if (static_cast<long long>(num_pages) * Hkv > 0x7FFFFFFFLL)
      return fail(CXA_EINVAL, w + ": num_pages * Hkv must be below 2^31");
    if (dh != 64 && dh != 128) return fail(CXA_EINVAL, w + ": head_dim must be 64 or 128");
    if (!valid_dtype(cache_dtype)) return fail(CXA_EINVAL, w + ": cache_dtype must be CXA_F32 or CXA_BF16");
    cxa_pages* c = new (std::nothrow) cxa_pages;
    if (c == nullptr) return fail(CXA_EINVAL, w + ": out of host memory");
    c->Kp = Kp;
    c->Vp = Vp;
    c->num_pages = num_pages;
    c->page_size = page_size;
    c->page_shift = 0;
    while ((1 << c->page_shift) < page_size) ++c->page_shift;
    c->L = L;
    c->Hkv = Hkv;
    c->dh = dh;
    c->dtype = cache_dtype;
    *out = c;
    return CXA_OK;
  });
}

void cxa_pages_destroy(cxa_pages* c) { delete c; }

int cxa_paged_check(const cxa_pages* pages, int B, int n_tokens, const int* q_start, const int* kv_len,
                    const int* page_table, int max_pages) {
  return guarded([&]() -> int {
    const std::string w = "cxa_paged_check";
    int rc = check_batch(w, pages, 0, B, n_tokens, q_start, kv_len, page_table, max_pages);
    if (rc != CXA_OK) return rc;
    return check_host_batch(w, pages->num_pages, pages->page_shift, B, n_tokens, q_start, kv_len, page_table, max_pages);
  });
}

int cxa_paged_append(const cxa_pages* pages, int layer, int B, int n_tokens, const int* q_start, const int* kv_len,
                     const int* page_table, int max_pages, const void* k, long long k_stride, const void* v,
                     long long v_stride, const void* q, long long q_stride, int Hq, void* q_out, long long qo_stride,
                     int norm, float eps, const float* q_weight, const float* k_weight, const cxa_rotary* rot,
                     int dtype, void* stream) {
  return guarded([&]() -> int {
    const std::string w = "cxa_paged_append";
    int rc = check_batch(w, pages, layer, B, n_tokens, q_start, kv_len, page_table, max_pages);
    if (rc != CXA_OK) return rc;
    if (!valid_dtype(dtype)) return fail(CXA_EINVAL, w + ": dtype must be CXA_F32 or CXA_BF16");
    if (dtype == CXA_BF16 && pages->dtype == CXA_F32)
      return fail(CXA_EINVAL, w + ": bf16 activations need a bf16 pool");
    if (q == nullptr) Hq = 0;
    if (q != nullptr && (Hq < 1 || Hq > 65535)) return fail(CXA_EINVAL, w + ": Hq must lie in [1, 65535]");
    rc = check_norm(w, norm, eps, q_weight, k_weight);
    if (rc == CXA_OK) rc = check_rotary(w, rot, pages->dh);
    if (rc != CXA_OK) return rc;
    if (n_tokens == 0) return CXA_OK;
    rc = check_rows(w, "k", k, k_stride, n_tokens, pages->Hkv, pages->dh, dtype);
    if (rc == CXA_OK) rc = check_rows(w, "v", v, v_stride, n_tokens, pages->Hkv, pages->dh, dtype);
    if (rc == CXA_OK && Hq > 0) rc = check_rows(w, "q", q, q_stride, n_tokens, Hq, pages->dh, dtype);
    if (rc == CXA_OK && Hq > 0) rc = check_rows(w, "q_out", q_out, qo_stride, n_tokens, Hq, pages->dh, dtype);
    if (rc != CXA_OK) return rc;
    std::string msg;
    cxa::DeviceInfo dev;
    cudaError_t e = cxa::current_device_info(&dev, &msg);
    if (e != cudaSuccess) return fail_cuda(e, w + ": " + msg);
    cxa::NormRopeLaunch a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_out = q_out;
    a.qo_stride = qo_stride;
    a.Hq = Hq;
    a.Hk = pages->Hkv;
    a.dh = pages->dh;
    a.n_tokens = n_tokens;
    a.wq = q_weight;
    a.wk = k_weight;
    a.eps = eps;
    a.norm = norm == CXA_NORM_RMS;
    a.act_bf16 = dtype == CXA_BF16;
    a.pool_bf16 = pages->dtype == CXA_BF16;
    a.rot = rotary_arg(rot);
    a.append = true;
    a.batch = {q_start, kv_len, page_table, B, n_tokens, max_pages};
    a.layer = layer_of(pages, layer);
    e = cxa::launch_norm_rope(a, dev, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return fail_cuda(e, w + ": launch");
    return CXA_OK;
  });
}

size_t cxa_paged_attention_workspace_bytes(int Hq, int Hkv, int dh, int max_new) {
  if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || (dh != 64 && dh != 128) || max_new < 1) return 0;
  size_t n = cxa::kPagedCounterBytes + cxa::paged_rows_part_bytes(dh);
  if (cxa::paged_tile_takes(Hq / Hkv, true, max_new)) n += cxa::paged_tile_part_bytes(dh);
  return n;
}

int cxa_paged_attention(const cxa_pages* pages, int layer, int B, int n_tokens, int max_new, const int* q_start,
                        const int* kv_len, const int* page_table, int max_pages, const void* q, long long q_stride,
                        int Hq, void* out, long long o_stride, float scale, int dtype, void* workspace,
                        size_t workspace_bytes, void* stream) {
  return guarded([&]() -> int {
    const std::string w = "cxa_paged_attention";
    int rc = check_batch(w, pages, layer, B, n_tokens, q_start, kv_len, page_table, max_pages);
    if (rc != CXA_OK) return rc;
    if (!valid_dtype(dtype)) return fail(CXA_EINVAL, w + ": dtype must be CXA_F32 or CXA_BF16");
    if (dtype == CXA_BF16 && pages->dtype == CXA_F32)
      return fail(CXA_EINVAL, w + ": bf16 queries need a bf16 pool");
    if (Hq < 1 || Hq > 65535 || Hq % pages->Hkv != 0)
      return fail(CXA_EINVAL, w + ": Hq must be a positive multiple of the pool's K/V heads, at most 65535");
    if (max_new < 1) return fail(CXA_EINVAL, w + ": max_new must be positive");
    if (static_cast<long long>(n_tokens) * (Hq / pages->Hkv) > 0x7FFFFFFFLL - 256)
      return fail(CXA_EINVAL, w + ": too many query rows");
    if (!std::isfinite(scale) || (scale > 0.f && !std::isfinite(scale * 1.4426950408889634f)))
      return fail(CXA_EINVAL, w + ": scale must be finite, log2(e) times it too");
    if (n_tokens == 0) return CXA_OK;
    rc = check_rows(w, "q", q, q_stride, n_tokens, Hq, pages->dh, dtype);
    if (rc == CXA_OK) rc = check_rows(w, "out", out, o_stride, n_tokens, Hq, pages->dh, dtype);
    if (rc != CXA_OK) return rc;
    if (overlap(q, q_stride, out, o_stride, n_tokens, Hq, Hq, pages->dh, elt(dtype)))
      return fail(CXA_EINVAL, w + ": out must not overlap q");
    if (workspace == nullptr || !aligned(workspace, 256))
      return fail(CXA_EINVAL, w + ": the workspace is NULL or not 256-byte aligned");
    if (workspace_bytes < cxa_paged_attention_workspace_bytes(Hq, pages->Hkv, pages->dh, max_new))
      return fail(CXA_EINVAL, w + ": workspace smaller than cxa_paged_attention_workspace_bytes()");
    cxa::PagedAttnLaunch a = {};
    a.q = q;
    a.out = out;
    a.q_stride = q_stride;
    a.o_stride = o_stride;
    a.Hq = Hq;
    a.dh = pages->dh;
    a.max_new = max_new;
    a.scale = scale > 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(pages->dh));
    a.act_bf16 = dtype == CXA_BF16;
    a.pool_bf16 = pages->dtype == CXA_BF16;
    a.batch = {q_start, kv_len, page_table, B, n_tokens, max_pages};
    a.layer = layer_of(pages, layer);
    a.workspace = workspace;
    const bool tiles = cxa::paged_tile_takes(Hq / pages->Hkv, a.act_bf16, max_new);
    const int max_rows = tiles ? cxa::kFewRows : 0x7FFFFFFF;
    if (!cxa::paged_rows_countable(a, max_rows) || (tiles && !cxa::paged_tile_countable(a)))
      return fail(CXA_EINVAL, w + ": the chunks of keys of all tiles of query rows (see cxa.h) must be below 2^31");
    std::string msg;
    cxa::DeviceInfo dev;
    cudaError_t e = cxa::current_device_info(&dev, &msg);
    if (e != cudaSuccess) return fail_cuda(e, w + ": " + msg);
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    cxa::PagedTileMaps maps;
    // whatever can fail does before the first kernel is enqueued
    if (tiles && (e = cxa::prepare_paged_tile(a, dev, &maps, &msg)) != cudaSuccess) return fail_cuda(e, w + ": " + msg);
    const std::lock_guard<std::mutex> together(stream_lock(s));      // (of one kernel too: its workspace may be another call's)
    e = cxa::launch_paged_rows(a, max_rows, dev, s);
    if (e == cudaSuccess && tiles) e = cxa::launch_paged_tile(a, maps, dev, s);
    if (e != cudaSuccess) return fail_cuda(e, w + ": launch");
    return CXA_OK;
  });
}

}  // extern "C"
