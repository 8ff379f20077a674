"""Python binding of libcxa (include/cxa.h): argument marshalling only.

The C-named functions (``cxa_populate``, ``cxa_decode``, ``cxa_invalidate``, ...)
take raw device pointers or torch tensors (their ``data_ptr()`` is passed) and
return the C status code. ``CrossAttentionCache`` is a convenience owner of the
cache, workspaces and descriptor that raises ``CxaError`` on a non-zero status.
PyTorch is used for device memory and streams only; every step of populate and
decode runs in libcxa's CUDA kernels. There is no fallback: if the library is
not built, loading it raises.
"""
from __future__ import annotations

import ctypes
import os

from . import _build

CXA_OK, CXA_EINVAL, CXA_ENOTREADY, CXA_ECUDA, CXA_ETIMEOUT, CXA_EPAGE = 0, -1, -2, -3, -4, -5
CXA_F32, CXA_BF16 = 0, 1
CXA_DECODE_AUTO, CXA_DECODE_STREAM, CXA_DECODE_ROWS = 0, 1, 2
CXA_POPULATE_AUTO, CXA_POPULATE_PAIR, CXA_POPULATE_SINGLE = 0, 1, 2
CXA_ROTARY_HALF, CXA_ROTARY_INTERLEAVED = 0, 1
CXA_ROTARY_PLAIN, CXA_ROTARY_LINEAR, CXA_ROTARY_NTK, CXA_ROTARY_WAVELENGTH = 0, 1, 2, 3
CXA_NORM_NONE, CXA_NORM_RMS = 0, 1

# every symbol include/cxa.h declares: name -> (restype, argtypes)
_c_void_pp = ctypes.POINTER(ctypes.c_void_p)
SIGNATURES = {
    "cxa_cache_create": (ctypes.c_int, [_c_void_pp, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "cxa_cache_destroy": (None, [ctypes.c_void_p]),
    "cxa_populate_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "cxa_decode_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int] * 5),
    "cxa_populate": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                    ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                    ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "cxa_pack_weights": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "cxa_populate_packed": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_int,
                                           ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]),
    "cxa_convert_bf16": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "cxa_decode": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float,
                                  ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "cxa_invalidate": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int]),
    "cxa_is_ready": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int]),
    "cxa_strerror": (ctypes.c_char_p, [ctypes.c_int]),
    "cxa_last_error_message": (ctypes.c_char_p, []),
    "cxa_launch_count": (ctypes.c_ulonglong, []),
    "cxa_device_status": (ctypes.c_int, [ctypes.c_int]),
    "cxa_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_uint, ctypes.c_void_p]),
    "cxa_set_decode_policy": (ctypes.c_int, [ctypes.c_int]),
    "cxa_set_populate_policy": (ctypes.c_int, [ctypes.c_int]),
    "cxa_decode_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_float, ctypes.c_void_p]),
    "cxa_decode_shared_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int] * 6),
    "cxa_decode_shared": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t,
                                         ctypes.c_void_p]),
    "cxa_decode_layers": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p,
                                         ctypes.c_size_t, ctypes.c_void_p]),
    "cxa_cross_block_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int] * 5),
    "cxa_cross_block": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float,
                                       ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "cxa_cache_append": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p]),
    "cxa_self_attention_step": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                               ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p,
                                               ctypes.c_size_t, ctypes.c_void_p]),
    "cxa_alignment_weights": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_float,
                                             ctypes.c_void_p]),
    "cxa_rotary_frequencies": (ctypes.c_int, [ctypes.c_int, ctypes.c_double, ctypes.c_int, ctypes.c_double,
                                              ctypes.c_double, ctypes.c_double, ctypes.c_double, ctypes.c_void_p,
                                              ctypes.c_void_p]),
    "cxa_rotary_create": (ctypes.c_int, [_c_void_pp, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_double]),
    "cxa_rotary_destroy": (None, [ctypes.c_void_p]),
    "cxa_qk_norm_rope": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_longlong, ctypes.c_int, ctypes.c_void_p,
                                        ctypes.c_longlong, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                        ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_longlong, ctypes.c_void_p,
                                        ctypes.c_longlong, ctypes.c_int, ctypes.c_void_p]),
    "cxa_pages_create": (ctypes.c_int, [_c_void_pp, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_int,
                                        ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int]),
    "cxa_pages_destroy": (None, [ctypes.c_void_p]),
    "cxa_paged_check": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_int]),
    "cxa_paged_append": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                        ctypes.c_longlong, ctypes.c_void_p, ctypes.c_longlong, ctypes.c_void_p,
                                        ctypes.c_longlong, ctypes.c_int, ctypes.c_void_p, ctypes.c_longlong,
                                        ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p]),
    "cxa_paged_attention_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int] * 4),
    "cxa_paged_attention": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                           ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int,
                                           ctypes.c_void_p, ctypes.c_longlong, ctypes.c_int, ctypes.c_void_p,
                                           ctypes.c_longlong, ctypes.c_float, ctypes.c_int, ctypes.c_void_p,
                                           ctypes.c_size_t, ctypes.c_void_p]),
}

# most query rows cxa_decode_shared takes per cache row (CXA_MAX_SHARED_QUERIES)
CXA_MAX_SHARED_QUERIES = 16

# bytes of the fixed device scratch behind cxa_decode_noalloc (CXA_NOALLOC_SCRATCH_BYTES)
CXA_NOALLOC_SCRATCH_BYTES = 8 << 20
# bytes at the start of a cxa_paged_attention workspace to clear before its first use
CXA_PAGED_COUNTER_BYTES = 11520

_lib = None


def load(path: str | None = None):
    """Load libcxa.so (once) and declare its signatures."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or _build.LIB
    if not os.path.exists(path):
        raise RuntimeError(f"libcxa is not built ({path} is missing); build it with "
                           "encoder_decoder_speech_gb300._build.build_library()")
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


class CxaError(RuntimeError):
    def __init__(self, code: int, where: str):
        lib = load()
        self.code = code
        super().__init__(f"{where}: {lib.cxa_strerror(code).decode()}: {lib.cxa_last_error_message().decode()}")


def check(code: int, where: str = "cxa") -> None:
    if code != CXA_OK:
        raise CxaError(code, where)


def _ptr(x) -> int | None:
    if x is None:
        return None
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    return int(x)


def _stream(s) -> int | None:
    if s is None:
        import torch
        # the current stream's handle without building a Stream object (a few
        # microseconds per call on the host otherwise)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:
            return raw(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if hasattr(s, "cuda_stream"):
        return s.cuda_stream
    return int(s)


# ---------------------------------------------------------------- C-named calls
def cxa_cache_create(Kc, Vc, B, T, L, H, dh, cache_dtype):
    """Returns (status, handle); handle is None unless status == CXA_OK."""
    h = ctypes.c_void_p()
    rc = load().cxa_cache_create(ctypes.byref(h), _ptr(Kc), _ptr(Vc), B, T, L, H, dh, cache_dtype)
    return rc, (h.value if rc == CXA_OK else None)


def cxa_cache_destroy(handle) -> None:
    load().cxa_cache_destroy(handle)


def cxa_populate_workspace_bytes(d, L, in_dtype) -> int:
    return load().cxa_populate_workspace_bytes(d, L, in_dtype)


def cxa_decode_workspace_bytes(B, T, L, H, dh=64) -> int:
    return load().cxa_decode_workspace_bytes(B, T, L, H, dh)


def cxa_populate(handle, b0, nb, E, WK, WV, bV, T, d, L, H, in_dtype, workspace, workspace_bytes, stream=None) -> int:
    return load().cxa_populate(handle, b0, nb, _ptr(E), _ptr(WK), _ptr(WV), _ptr(bV), T, d, L, H, in_dtype,
                               _ptr(workspace), workspace_bytes, _stream(stream))


def cxa_pack_weights(WK, WV, d, L, in_dtype, packed, packed_bytes, stream=None) -> int:
    return load().cxa_pack_weights(_ptr(WK), _ptr(WV), d, L, in_dtype, _ptr(packed), packed_bytes, _stream(stream))


def cxa_populate_packed(handle, b0, nb, E, packed, packed_bytes, bV, T, d, L, H, in_dtype, stream=None) -> int:
    return load().cxa_populate_packed(handle, b0, nb, _ptr(E), _ptr(packed), packed_bytes, _ptr(bV), T, d, L, H,
                                      in_dtype, _stream(stream))


def cxa_convert_bf16(src, dst, n, stream=None) -> int:
    return load().cxa_convert_bf16(_ptr(src), _ptr(dst), n, _stream(stream))


def to_bf16(x, out=None, stream=None):
    """fp32 device tensor -> bf16 device tensor of the same shape (cxa_convert_bf16)."""
    import torch
    if x.dtype != torch.float32 or not x.is_contiguous():
        raise ValueError("to_bf16 takes a contiguous float32 tensor")
    if out is None:
        out = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    check(cxa_convert_bf16(x, out, x.numel(), stream), "cxa_convert_bf16")
    return out


def cxa_decode(handle, Q, key_len, out, scale, workspace, workspace_bytes, stream=None) -> int:
    return load().cxa_decode(handle, _ptr(Q), _ptr(key_len), _ptr(out), float(scale), _ptr(workspace),
                             workspace_bytes, _stream(stream))


def cxa_decode_shared_workspace_bytes(B, T, L, H, dh=64, nq=1) -> int:
    return load().cxa_decode_shared_workspace_bytes(B, T, L, H, dh, nq)


def cxa_decode_shared(handle, nq, Q, key_len, out, scale, workspace, workspace_bytes, stream=None) -> int:
    return load().cxa_decode_shared(handle, nq, _ptr(Q), _ptr(key_len), _ptr(out), float(scale), _ptr(workspace),
                                    workspace_bytes, _stream(stream))


def cxa_decode_layers(handle, l0, nl, Q, key_len, out, scale, workspace, workspace_bytes, stream=None) -> int:
    return load().cxa_decode_layers(handle, l0, nl, _ptr(Q), _ptr(key_len), _ptr(out), float(scale),
                                    _ptr(workspace), workspace_bytes, _stream(stream))


def cxa_cross_block_workspace_bytes(B, T, L, H, dh=64) -> int:
    return load().cxa_cross_block_workspace_bytes(B, T, L, H, dh)


def cxa_cross_block(handle, layer, x, ln_gamma, ln_beta, ln_eps, WQ, bQ, WO, bO, key_len, scale, workspace,
                    workspace_bytes, stream=None) -> int:
    return load().cxa_cross_block(handle, layer, _ptr(x), _ptr(ln_gamma), _ptr(ln_beta), float(ln_eps), _ptr(WQ),
                                  _ptr(bQ), _ptr(WO), _ptr(bO), _ptr(key_len), float(scale), _ptr(workspace),
                                  workspace_bytes, _stream(stream))


def cxa_cache_append(handle, pos, K_new, V_new, stream=None) -> int:
    return load().cxa_cache_append(handle, _ptr(pos), _ptr(K_new), _ptr(V_new), _stream(stream))


def cxa_self_attention_step(handle, pos, Q, K_new, V_new, out, scale, workspace, workspace_bytes, stream=None) -> int:
    return load().cxa_self_attention_step(handle, _ptr(pos), _ptr(Q), _ptr(K_new), _ptr(V_new), _ptr(out), float(scale),
                                          _ptr(workspace), workspace_bytes, _stream(stream))


_HEADS_ARRAYS: dict = {}


def _heads_array(heads):
    """The (layer, head) pairs as a C int array, kept per distinct head list (a call
    site passes the same list every step)."""
    key = tuple((int(l), int(h)) for l, h in heads)
    arr = _HEADS_ARRAYS.get(key)
    if arr is None:
        flat = [v for pair in key for v in pair]
        arr = (ctypes.c_int * max(len(flat), 1))(*flat)
        if len(_HEADS_ARRAYS) < 256:
            _HEADS_ARRAYS[key] = arr
    return arr, len(key)


def cxa_alignment_weights(handle, Q, key_len, heads, weights, mean, scale, stream=None) -> int:
    """heads: host sequence of (layer, head) pairs."""
    arr, n = _heads_array(heads)
    return load().cxa_alignment_weights(handle, _ptr(Q), _ptr(key_len), ctypes.cast(arr, ctypes.c_void_p), n,
                                        _ptr(weights), _ptr(mean), float(scale), _stream(stream))


def cxa_decode_noalloc(handle, Q, key_len, out, scale, stream=None) -> int:
    """cxa_decode with its scratch in libcxa's fixed device array: for callers
    that cannot allocate device memory. Calls must be ordered on one stream."""
    return load().cxa_decode_noalloc(handle, _ptr(Q), _ptr(key_len), _ptr(out), float(scale), _stream(stream))


def cxa_rotary_frequencies(rot_dim, base, scaling, factor=1.0, orig_len=0.0, alpha=1.0, beta=32.0):
    """Returns (status, frequencies, attn_factor): radians a position of each rotated pair."""
    freq, att = (ctypes.c_double * max(rot_dim // 2, 1))(), ctypes.c_double()
    rc = load().cxa_rotary_frequencies(rot_dim, base, scaling, factor, orig_len, alpha, beta, freq, ctypes.byref(att))
    return rc, list(freq), att.value


def cxa_rotary_create(rot_dim, layout, freq, attn_factor=1.0):
    """freq: host sequence of rot_dim / 2 numbers. Returns (status, handle)."""
    if freq is not None and len(freq) < rot_dim // 2:
        raise ValueError("freq must have rot_dim / 2 entries")
    h = ctypes.c_void_p()
    arr = None if freq is None else (ctypes.c_double * max(len(freq), 1))(*freq)
    rc = load().cxa_rotary_create(ctypes.byref(h), rot_dim, layout, arr, attn_factor)
    return rc, (h.value if rc == CXA_OK else None)


def cxa_rotary_destroy(handle) -> None:
    load().cxa_rotary_destroy(handle)


def cxa_qk_norm_rope(q, q_stride, Hq, k, k_stride, Hk, dh, n_tokens, pos, norm, eps, q_weight, k_weight, rot, q_out,
                     qo_stride, k_out, ko_stride, dtype, stream=None) -> int:
    return load().cxa_qk_norm_rope(_ptr(q), q_stride, Hq, _ptr(k), k_stride, Hk, dh, n_tokens, _ptr(pos), norm, eps,
                                   _ptr(q_weight), _ptr(k_weight), rot, _ptr(q_out), qo_stride, _ptr(k_out), ko_stride,
                                   dtype, _stream(stream))


def cxa_pages_create(Kp, Vp, num_pages, page_size, L, Hkv, dh, cache_dtype):
    """Returns (status, handle); handle is None unless status == CXA_OK."""
    h = ctypes.c_void_p()
    rc = load().cxa_pages_create(ctypes.byref(h), _ptr(Kp), _ptr(Vp), num_pages, page_size, L, Hkv, dh, cache_dtype)
    return rc, (h.value if rc == CXA_OK else None)


def cxa_pages_destroy(handle) -> None:
    load().cxa_pages_destroy(handle)


def cxa_paged_check(handle, B, n_tokens, q_start, kv_len, page_table, max_pages) -> int:
    """q_start [B + 1], kv_len [B], page_table [B * max_pages]: host sequences of ints."""
    def ints(x):
        x = [int(v) for v in x]
        if any(v < -2 ** 31 or v >= 2 ** 31 for v in x):
            raise ValueError("q_start, kv_len and page_table must hold 32-bit integers")
        return (ctypes.c_int * max(len(x), 1))(*x)
    if len(q_start) != B + 1 or len(kv_len) != B or len(page_table) != B * max_pages:
        raise ValueError("q_start, kv_len and page_table must have B + 1, B and B * max_pages entries")
    return load().cxa_paged_check(handle, B, n_tokens, ints(q_start), ints(kv_len), ints(page_table), max_pages)


def cxa_paged_append(handle, layer, B, n_tokens, q_start, kv_len, page_table, max_pages, k, k_stride, v, v_stride, q,
                     q_stride, Hq, q_out, qo_stride, norm, eps, q_weight, k_weight, rot, dtype, stream=None) -> int:
    return load().cxa_paged_append(handle, layer, B, n_tokens, _ptr(q_start), _ptr(kv_len), _ptr(page_table), max_pages,
                                   _ptr(k), k_stride, _ptr(v), v_stride, _ptr(q), q_stride, Hq, _ptr(q_out), qo_stride,
                                   norm, eps, _ptr(q_weight), _ptr(k_weight), rot, dtype, _stream(stream))


def cxa_paged_attention_workspace_bytes(Hq, Hkv, dh, max_new) -> int:
    return load().cxa_paged_attention_workspace_bytes(Hq, Hkv, dh, max_new)


def cxa_paged_attention(handle, layer, B, n_tokens, max_new, q_start, kv_len, page_table, max_pages, q, q_stride, Hq,
                        out, o_stride, scale, dtype, workspace, workspace_bytes, stream=None) -> int:
    return load().cxa_paged_attention(handle, layer, B, n_tokens, max_new, _ptr(q_start), _ptr(kv_len),
                                      _ptr(page_table), max_pages, _ptr(q), q_stride, Hq, _ptr(out), o_stride, scale,
                                      dtype, _ptr(workspace), workspace_bytes, _stream(stream))


def cxa_invalidate(handle, b=-1) -> int:
    return load().cxa_invalidate(handle, b)


def cxa_is_ready(handle, b) -> int:
    return load().cxa_is_ready(handle, b)


def cxa_strerror(code) -> str:
    return load().cxa_strerror(code).decode()


def cxa_last_error_message() -> str:
    return load().cxa_last_error_message().decode()


def cxa_launch_count() -> int:
    return load().cxa_launch_count()


def cxa_device_status(clear=0) -> int:
    return load().cxa_device_status(clear)


def cxa_set_decode_policy(policy: int) -> int:
    """Process-wide choice of the one-query decode kernel shape (CXA_DECODE_*)."""
    return load().cxa_set_decode_policy(policy)


def cxa_set_populate_policy(policy: int) -> int:
    """Process-wide choice of the populate GEMM shape (CXA_POPULATE_*)."""
    return load().cxa_set_populate_policy(policy)


def cxa_selftest_wait_timeout(limit_us: int, stream=None) -> int:
    """Enqueue the bounded-wait self-test kernel (its wait expires after limit_us)."""
    return load().cxa_selftest_wait_timeout(limit_us, _stream(stream))


# ---------------------------------------------------------------- owner object
_DTYPES = {"f32": CXA_F32, "bf16": CXA_BF16}


def _dtype_code(t) -> int:
    import torch
    if t == torch.float32:
        return CXA_F32
    if t == torch.bfloat16:
        return CXA_BF16
    raise TypeError(f"unsupported dtype {t}; expected float32 or bfloat16")


class CrossAttentionCache:
    """Owns a [B][L][H][T][64] K/V projection cache, its decode workspace and
    the libcxa descriptor; allocation goes through torch on ``device``."""

    def __init__(self, B: int, T: int, L: int, H: int, dh: int = 64, cache_dtype: str = "f32", device="cuda"):
        import torch
        self.B, self.T, self.L, self.H, self.dh = B, T, L, H, dh
        self.d = H * dh
        self.cache_dtype = cache_dtype
        tdt = torch.float32 if cache_dtype == "f32" else torch.bfloat16
        self.Kc = torch.empty((B, L, H, T, dh), dtype=tdt, device=device)
        self.Vc = torch.empty((B, L, H, T, dh), dtype=tdt, device=device)
        self.decode_ws_bytes = cxa_decode_workspace_bytes(B, T, L, H, dh)
        self.decode_ws = torch.zeros(max(self.decode_ws_bytes, 256), dtype=torch.uint8, device=device)
        self._pop_ws = {}
        self._shared_ws = None
        self._block_ws = None
        rc, h = cxa_cache_create(self.Kc, self.Vc, B, T, L, H, dh, _DTYPES[cache_dtype])
        check(rc, "cxa_cache_create")
        self.handle = h

    def populate_workspace(self, in_dtype: int):
        import torch
        if in_dtype not in self._pop_ws:
            n = cxa_populate_workspace_bytes(self.d, self.L, in_dtype)
            self._pop_ws[in_dtype] = torch.empty(n, dtype=torch.uint8, device=self.Kc.device)
        return self._pop_ws[in_dtype]

    def populate(self, E, WK, WV, bV, b0: int = 0, stream=None) -> None:
        """E [nb, T, d]; WK, WV [L, d, d] (d_in, d_out), same dtype as E; bV [L, d] fp32."""
        in_dtype = _dtype_code(E.dtype)
        for name, t in (("E", E), ("WK", WK), ("WV", WV), ("bV", bV)):
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
        if WK.dtype != E.dtype or WV.dtype != E.dtype:
            raise TypeError("WK and WV must have E's dtype")
        nb = E.shape[0] if E.dim() == 3 else 1
        ws = self.populate_workspace(in_dtype)
        check(cxa_populate(self.handle, b0, nb, E, WK, WV, bV, E.shape[-2], E.shape[-1], WK.shape[0],
                           self.H, in_dtype, ws, ws.numel(), stream), "cxa_populate")

    def pack_weights(self, WK, WV, stream=None):
        """Pack WK, WV [L, d, d] (d_in, d_out) once for populate_packed; returns the
        packed buffer (a uint8 device tensor owned by the caller)."""
        import torch
        in_dtype = _dtype_code(WK.dtype)
        if WV.dtype != WK.dtype or not WK.is_contiguous() or not WV.is_contiguous():
            raise ValueError("WK and WV must be contiguous and of one dtype")
        n = cxa_populate_workspace_bytes(self.d, self.L, in_dtype)
        packed = torch.empty(n, dtype=torch.uint8, device=self.Kc.device)
        check(cxa_pack_weights(WK, WV, self.d, self.L, in_dtype, packed, n, stream), "cxa_pack_weights")
        return packed

    def populate_packed(self, E, packed, bV, b0: int = 0, stream=None) -> None:
        """E [nb, T, d] (fp32 or bf16, the dtype the weights were packed in); bV [L, d] fp32."""
        in_dtype = _dtype_code(E.dtype)
        if not E.is_contiguous() or not bV.is_contiguous():
            raise ValueError("E and bV must be contiguous")
        nb = E.shape[0] if E.dim() == 3 else 1
        check(cxa_populate_packed(self.handle, b0, nb, E, packed, packed.numel(), bV, E.shape[-2], E.shape[-1],
                                  self.L, self.H, in_dtype, stream), "cxa_populate_packed")

    def decode(self, Q, key_len, out=None, scale: float = 0.0, stream=None):
        """Q [B, L, H, 64] fp32, key_len [B] int32 (device). Returns out [B, L, H, 64] fp32."""
        import torch
        if out is None:
            out = torch.empty_like(Q)
        check(cxa_decode(self.handle, Q, key_len, out, scale, self.decode_ws, self.decode_ws_bytes, stream),
              "cxa_decode")
        return out

    def decode_shared(self, Q, key_len, out=None, scale: float = 0.0, stream=None):
        """Q [B, nq, L, H, 64] fp32: nq hypotheses per slot sharing the slot's cache.
        Returns out [B, nq, L, H, 64] fp32."""
        import torch
        nq = Q.shape[1]
        need = cxa_decode_shared_workspace_bytes(self.B, self.T, self.L, self.H, self.dh, nq)
        if self._shared_ws is None or self._shared_ws.numel() < need:
            self._shared_ws = torch.zeros(max(need, 256), dtype=torch.uint8, device=self.Kc.device)
        if out is None:
            out = torch.empty_like(Q)
        check(cxa_decode_shared(self.handle, nq, Q, key_len, out, scale, self._shared_ws, self._shared_ws.numel(),
                                stream), "cxa_decode_shared")
        return out

    def decode_layers(self, l0: int, Q, key_len, out=None, scale: float = 0.0, stream=None):
        """Q [B, nl, H, 64] fp32 for layers [l0, l0+nl). Returns out of the same shape."""
        import torch
        if out is None:
            out = torch.empty_like(Q)
        check(cxa_decode_layers(self.handle, l0, Q.shape[1], Q, key_len, out, scale, self.decode_ws,
                                self.decode_ws_bytes, stream), "cxa_decode_layers")
        return out

    def cross_block(self, layer: int, x, WQ, WO, key_len, ln_gamma=None, ln_beta=None, ln_eps: float = 1e-5,
                    bQ=None, bO=None, scale: float = 0.0, stream=None):
        """One decoder layer's cross-attention block, in place on x [B, d] fp32."""
        import torch
        need = cxa_cross_block_workspace_bytes(self.B, self.T, self.L, self.H, self.dh)
        if self._block_ws is None or self._block_ws.numel() < need:
            self._block_ws = torch.zeros(max(need, 256), dtype=torch.uint8, device=self.Kc.device)
        check(cxa_cross_block(self.handle, layer, x, ln_gamma, ln_beta, ln_eps, WQ, bQ, WO, bO, key_len, scale,
                              self._block_ws, self._block_ws.numel(), stream), "cxa_cross_block")
        return x

    def append(self, pos, K_new, V_new, stream=None) -> None:
        """Write K_new/V_new [B, L, H, 64] fp32 at position pos[b] (device int32 [B])."""
        check(cxa_cache_append(self.handle, pos, K_new, V_new, stream), "cxa_cache_append")

    def self_attention_step(self, pos, Q, K_new, V_new, out=None, scale: float = 0.0, stream=None):
        """Append the new rows at pos, then decode Q over positions 0 .. pos[b]."""
        import torch
        if out is None:
            out = torch.empty_like(Q)
        check(cxa_self_attention_step(self.handle, pos, Q, K_new, V_new, out, scale, self.decode_ws,
                                      self.decode_ws_bytes, stream), "cxa_self_attention_step")
        return out

    def alignment_weights(self, Q, key_len, heads, scale: float = 0.0, with_mean: bool = True, stream=None):
        """Softmax rows [B, nsel, T] of the (layer, head) pairs in `heads` for queries
        Q [B, L, H, 64], and their mean over heads [B, T] (or None)."""
        import torch
        w = torch.empty((self.B, len(heads), self.T), dtype=torch.float32, device=self.Kc.device)
        m = torch.empty((self.B, self.T), dtype=torch.float32, device=self.Kc.device) if with_mean else None
        check(cxa_alignment_weights(self.handle, Q, key_len, heads, w, m, scale, stream), "cxa_alignment_weights")
        return w, m

    def invalidate(self, b: int = -1) -> None:
        check(cxa_invalidate(self.handle, b), "cxa_invalidate")

    def is_ready(self, b: int) -> bool:
        return cxa_is_ready(self.handle, b) == 1

    def close(self) -> None:
        if getattr(self, "handle", None):
            cxa_cache_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------- paged self-attention
# A decoding step makes these calls once a layer, with kernels of a few microseconds: their
# checks are written to cost little (together with the call, 8 us of the host's time).
class _TorchCalls:
    """torch's types and its shortest ways to the current device, stream and capture state."""

    def __init__(self):
        import torch
        c = torch._C
        self.torch, self.i32, self.f32 = torch, torch.int32, torch.float32
        self.code = {torch.float32: CXA_F32, torch.bfloat16: CXA_BF16}
        self.device = getattr(c, "_cuda_getDevice", torch.cuda.current_device)
        self.stream = getattr(c, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)
        self.capturing = getattr(c, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)


_torch_calls = None


def _calls():
    global _torch_calls
    if _torch_calls is None:
        _torch_calls = _TorchCalls()
    return _torch_calls


def _rows(name, t, H, dh, n, dtype, index):
    """Check a packed [n tokens, H heads, dh] tensor; returns its row stride."""
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [tokens, heads, head dim]")
    if shape != (n, H, dh):
        raise ValueError(f"{name} is {tuple(shape)}, expected {(n, H, dh)}")
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != dh and H > 1):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    if n <= 1:
        s0 = H * dh
    elif s0 < H * dh:
        raise ValueError(f"{name}: the rows of different tokens must not overlap")
    if t.dtype is not dtype:
        raise TypeError(f"{name}: {t.dtype}, expected {dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    return s0


def _heads(name, t):
    """The tokens and heads of a packed tensor."""
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [tokens, heads, head dim]")
    return shape[0], shape[1]


def _ints(name, t, shape, index, i32):
    if t.dtype is not i32 or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {shape} on cuda:{index}")


def _weight(name, t, dh, index, f32):
    if t.dtype is not f32 or t.shape != (dh,) or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape ({dh},) on cuda:{index}")
    return t.data_ptr()


def _code(tc, dtype):
    code = tc.code.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}; expected float32 or bfloat16")
    return code


def _run(tc, index, where, call, args):
    """call(*args) with the device current that the tensors are on; raises on a non-zero status."""
    if tc.device() == index:
        rc = call(*args)
    else:
        with tc.torch.cuda.device(index):
            rc = call(*args)
    if rc != CXA_OK:
        raise CxaError(rc, where)


def _capturing(tc, index, stream, raw):
    """Whether the call's stream (handle raw, of device index) is being captured."""
    if stream is None and tc.device() == index:
        return tc.capturing()
    with tc.torch.cuda.stream(tc.torch.cuda.ExternalStream(raw, device=index)):
        return tc.capturing()


# cudaStreamPerThread: one handle for every thread's own default stream. The allocator takes
# them for one stream, so memory of theirs may be handed from one thread to another while the
# first one's work is still using it.
_PER_THREAD = 2


def _own_handle(raw, what):
    if raw == _PER_THREAD:
        raise ValueError(f"memory cannot be kept apart for threads' own default streams: pass {what}, or name "
                         "another stream")


def _new(tc, q, stream, index):
    """An empty tensor like q for the result of a call on `stream`, in that stream's memory."""
    if stream is None:
        return q.new_empty(q.shape)
    _own_handle(_stream(stream), "the tensors for the results")
    with tc.torch.cuda.stream(tc.torch.cuda.ExternalStream(_stream(stream), device=index)):
        return q.new_empty(q.shape)


_LAYOUTS = {"half": CXA_ROTARY_HALF, "interleaved": CXA_ROTARY_INTERLEAVED}
_SCALINGS = {"none": CXA_ROTARY_PLAIN, "linear": CXA_ROTARY_LINEAR, "ntk": CXA_ROTARY_NTK,
             "wavelength": CXA_ROTARY_WAVELENGTH}


class Rotary:
    """A position rotation of the first ``rot_dim`` channels of a head (cxa_rotary): layout
    "half" pairs channels (i, i + rot_dim / 2), "interleaved" (2i, 2i + 1); scaling "none",
    "linear", "ntk" or "wavelength" (the YaRN paper's ramp in turns; checkpoints that ramp by
    pair number pass ``freq``) for contexts longer than the trained one. ``freq``
    (rot_dim / 2 radians a position) replaces the frequencies that base and scaling give,
    ``attn_factor`` the factor of the rotated values."""

    def __init__(self, rot_dim: int, base: float = 10000.0, layout: str = "half", scaling: str = "none",
                 factor: float = 1.0, orig_len: float = 0.0, alpha: float = 1.0, beta: float = 32.0, freq=None,
                 attn_factor: float | None = None):
        self.handle = None
        if layout not in _LAYOUTS or scaling not in _SCALINGS:
            raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}, scaling one of {sorted(_SCALINGS)}")
        if freq is None:
            rc, freq, att = cxa_rotary_frequencies(rot_dim, base, _SCALINGS[scaling], factor, orig_len, alpha, beta)
            check(rc, "cxa_rotary_frequencies")
        else:
            freq, att = [float(f) for f in freq], 1.0
            if len(freq) * 2 != rot_dim:
                raise ValueError("freq must have rot_dim / 2 entries")
        self.rot_dim, self.freq = rot_dim, freq
        self.attn_factor = att if attn_factor is None else attn_factor
        rc, self.handle = cxa_rotary_create(rot_dim, _LAYOUTS[layout], freq, self.attn_factor)
        check(rc, "cxa_rotary_create")

    def __del__(self):
        try:
            if self.handle:
                cxa_rotary_destroy(self.handle)
                self.handle = None
        except Exception:
            pass


def qk_norm_rope(q, k, pos, rotary: Rotary | None = None, norm_eps: float | None = None, q_weight=None, k_weight=None,
                 q_out=None, k_out=None, stream=None):
    """Head norms (RMS, if norm_eps is given) and rotation of q [N, Hq, dh] and k [N, Hk, dh]
    (or None), float32 or bfloat16, at positions pos [N] int32. Token rows may be strided
    slices; q_out and k_out may be q and k. Without norm_eps, or without k for k's, weights
    have no effect. Returns (q_out, k_out)."""
    tc = _torch_calls or _calls()
    n, Hq = _heads("q", q)
    dh, dt, at = q.shape[2], q.dtype, q.get_device()
    if at < 0:
        raise ValueError("the tensors must be on a CUDA device")
    qs = _rows("q", q, Hq, dh, n, dt, at)
    _ints("pos", pos, (n,), at, tc.i32)
    if q_out is None:
        q_out = _new(tc, q, stream, at)
    qos = _rows("q_out", q_out, Hq, dh, n, dt, at)
    Hk = ks = kos = 0
    kp = kop = None
    if k is not None:
        Hk = _heads("k", k)[1]
        ks = _rows("k", k, Hk, dh, n, dt, at)
        if k_out is None:
            k_out = _new(tc, k, stream, at)
        kos = _rows("k_out", k_out, Hk, dh, n, dt, at)
        kp, kop = k.data_ptr(), k_out.data_ptr()
    else:
        k_out = None
    norm, eps = (CXA_NORM_NONE, 0.0) if norm_eps is None else (CXA_NORM_RMS, norm_eps)
    _run(tc, at, "cxa_qk_norm_rope", load().cxa_qk_norm_rope, (
        q.data_ptr(), qs, Hq, kp, ks, Hk, dh, n, pos.data_ptr(), norm, eps,
        None if q_weight is None else _weight("q_weight", q_weight, dh, at, tc.f32),
        None if k_weight is None else _weight("k_weight", k_weight, dh, at, tc.f32),
        None if rotary is None else rotary.handle, q_out.data_ptr(), qos, kop, kos, _code(tc, dt),
        tc.stream(at) if stream is None else _stream(stream)))
    return q_out, k_out


class PagedCache:
    """Owns a [L][num_pages][Hkv][page_size][dh] pool of K/V pages (``Kp``, ``Vp``, zeroed),
    its descriptor, and the attention's workspaces: one per stream, so that calls on
    different streams do not share one (of more than 64 the oldest are dropped; a stream's
    calls must be done before it is destroyed, as its handle may come back as another's).
    Calls on a thread's own default stream (cudaStreamPerThread) need a workspace and an
    out of the caller's. The batch of a call is q_start [B + 1], kv_len [B]
    and page_table [B, max_pages], int32 on the device (see include/cxa.h)."""

    KEPT_WORKSPACES = 64

    def __init__(self, num_pages: int, page_size: int, L: int, Hkv: int, dh: int = 64, cache_dtype: str = "bf16",
                 device="cuda"):
        import torch
        self.handle = None
        self.num_pages, self.page_size, self.L, self.Hkv, self.dh = num_pages, page_size, L, Hkv, dh
        self.cache_dtype = cache_dtype
        tdt = torch.float32 if _DTYPES[cache_dtype] == CXA_F32 else torch.bfloat16
        self.Kp = torch.zeros((L, num_pages, Hkv, page_size, dh), dtype=tdt, device=device)
        self.Vp = torch.zeros((L, num_pages, Hkv, page_size, dh), dtype=tdt, device=device)
        self._ws, self._ws_bytes = {}, {}
        self._at = self.Kp.get_device()
        rc, self.handle = cxa_pages_create(self.Kp, self.Vp, num_pages, page_size, L, Hkv, dh, _DTYPES[cache_dtype])
        check(rc, "cxa_pages_create")

    def _batch(self, q_start, kv_len, page_table, i32):
        shape, at = page_table.shape, self._at
        if at < 0:
            raise ValueError("the tensors must be on a CUDA device")
        if len(shape) != 2:
            raise ValueError("page_table must be [sequences, pages]")
        B = shape[0]
        _ints("q_start", q_start, (B + 1,), at, i32)
        _ints("kv_len", kv_len, (B,), at, i32)
        _ints("page_table", page_table, shape, at, i32)
        return B, shape[1]

    def _scratch(self, tc, Hq, max_new, stream, raw):
        """The workspace of a call on the stream with handle raw: the tensor, its address and bytes."""
        need = self._ws_bytes.get((Hq, max_new))
        if need is None:
            if len(self._ws_bytes) > 4096:
                self._ws_bytes.clear()
            need = cxa_paged_attention_workspace_bytes(Hq, self.Hkv, self.dh, max_new)
            self._ws_bytes[Hq, max_new] = need
        _own_handle(raw, "a workspace")
        kept = self._ws.get(raw)
        capturing = _capturing(tc, self._at, stream, raw)
        if kept is not None and kept[2] >= need and not capturing:
            return kept
        torch = tc.torch
        with torch.cuda.stream(torch.cuda.ExternalStream(raw, device=self._at)):
            ws = torch.empty(max(need, CXA_PAGED_COUNTER_BYTES), dtype=torch.uint8, device=self.Kp.device)
            ws[:CXA_PAGED_COUNTER_BYTES].zero_()
        new = (ws, ws.data_ptr(), ws.numel())
        if not capturing:
            self._ws.pop(raw, None)
            self._ws[raw] = new                # the newest last
            while len(self._ws) > self.KEPT_WORKSPACES:
                self._ws.pop(next(iter(self._ws), None), None)     # its memory goes back to its stream's
        return new

    def workspace(self, Hq: int, max_new: int, stream=None):
        """An attention workspace (its counters zeroed), kept per stream. While a graph is captured
        it is a new one (cleared in the graph), as replays may run beside anything else."""
        tc = _calls()
        return self._scratch(tc, Hq, max_new, stream, tc.stream(self._at) if stream is None else _stream(stream))[0]

    def append(self, layer: int, k, v, q_start, kv_len, page_table, q=None, q_out=None, rotary: Rotary | None = None,
               norm_eps: float | None = None, q_weight=None, k_weight=None, stream=None):
        """Write k, v [N, Hkv, dh] of the new tokens into their pages, k normalised (RMS, if
        norm_eps is given: without it weights have no effect) and rotated; with q [N, Hq, dh]
        also return q_out, the queries normalised and rotated (rows behind the batch's last
        token are left as they are)."""
        tc = _torch_calls or _calls()
        at, dh, dt, n = self._at, self.dh, k.dtype, _heads("k", k)[0]
        B, width = self._batch(q_start, kv_len, page_table, tc.i32)
        ks = _rows("k", k, self.Hkv, dh, n, dt, at)
        vs = _rows("v", v, self.Hkv, dh, n, dt, at)
        Hq = qs = qos = 0
        qp = qop = None
        if q is not None:
            Hq = _heads("q", q)[1]
            qs = _rows("q", q, Hq, dh, n, dt, at)
            if q_out is None:
                q_out = _new(tc, q, stream, at)
            qos = _rows("q_out", q_out, Hq, dh, n, dt, at)
            qp, qop = q.data_ptr(), q_out.data_ptr()
        norm, eps = (CXA_NORM_NONE, 0.0) if norm_eps is None else (CXA_NORM_RMS, norm_eps)
        _run(tc, at, "cxa_paged_append", load().cxa_paged_append, (
            self.handle, layer, B, n, q_start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), width,
            k.data_ptr(), ks, v.data_ptr(), vs, qp, qs, Hq, qop, qos, norm, eps,
            None if q_weight is None else _weight("q_weight", q_weight, dh, at, tc.f32),
            None if k_weight is None else _weight("k_weight", k_weight, dh, at, tc.f32),
            None if rotary is None else rotary.handle, _code(tc, dt),
            tc.stream(at) if stream is None else _stream(stream)))
        return q_out if q is not None else None

    def attend(self, layer: int, q, q_start, kv_len, page_table, max_new: int, out=None, scale: float = 0.0,
               workspace=None, stream=None):
        """Attention of the new tokens' queries q [N, Hq, dh] over their sequences' keys up to
        each token's own. max_new: an upper bound of the new tokens of one sequence; workspace:
        a tensor, its counters zeroed, to use instead of the cache's own. Returns out [N, Hq, dh] (rows behind
        the batch's last token are left as they are)."""
        tc = _torch_calls or _calls()
        at, dh, dt = self._at, self.dh, q.dtype
        B, width = self._batch(q_start, kv_len, page_table, tc.i32)
        n, Hq = _heads("q", q)
        qs = _rows("q", q, Hq, dh, n, dt, at)
        if out is None:
            out = _new(tc, q, stream, at)
        os_ = _rows("out", out, Hq, dh, n, dt, at)
        raw = tc.stream(at) if stream is None else _stream(stream)
        if workspace is None:
            ws = self._scratch(tc, Hq, max_new, stream, raw)
        else:
            if workspace.get_device() != at or not workspace.is_contiguous():
                raise ValueError(f"workspace must be a contiguous tensor on cuda:{at}")
            ws = workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()
        _run(tc, at, "cxa_paged_attention", load().cxa_paged_attention, (
            self.handle, layer, B, n, max_new, q_start.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), width,
            q.data_ptr(), qs, Hq, out.data_ptr(), os_, scale, _code(tc, dt), ws[1], ws[2], raw))
        return out

    def check(self, q_start, kv_len, page_table, n_tokens: int) -> None:
        """Raise CxaError if the batch (host or device tensors) is not sound (cxa_paged_check)."""
        check(cxa_paged_check(self.handle, page_table.shape[0], n_tokens, q_start.tolist(), kv_len.tolist(),
                              page_table.reshape(-1).tolist(), page_table.shape[1]), "cxa_paged_check")

    def drop_workspaces(self) -> None:
        """Give the kept workspaces back: the next calls get new ones, with counters of zero. To be
        called after a CXA_ETIMEOUT, which may leave counters behind."""
        self._ws.clear()

    def close(self) -> None:
        if getattr(self, "handle", None):
            cxa_pages_destroy(self.handle)
            self.handle = None
            self.drop_workspaces()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
