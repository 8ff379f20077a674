"""Failure detection on the GPU without a fault: a kernel's bounded wait on a
barrier that nothing completes gives up after a short limit, sets the device
status word and returns; the host reads CXA_ETIMEOUT, clears it, and the context
goes on working (a decode right after still matches the oracle)."""
import threading
import time

import numpy as np
import pytest
import torch

from _gpu_common import DECODE_F32_MAX_ABS, cache_for, dev, host, inputs_on_device
from encoder_decoder_speech_gb300 import cxa
from encoder_decoder_speech_gb300 import workloads as W
from oracle import cross_attention as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib(cxa_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    torch.cuda.synchronize()
    assert cxa.cxa_device_status(1) == cxa.CXA_OK


def test_bounded_wait_expires_and_is_reported():
    assert cxa.cxa_device_status(1) == cxa.CXA_OK          # start clean
    t0 = time.perf_counter()
    assert cxa.cxa_selftest_wait_timeout(20000) == cxa.CXA_OK   # a 20 ms limit
    torch.cuda.synchronize()
    waited = time.perf_counter() - t0
    assert 0.015 <= waited < 5.0                           # it waited, and it came back
    assert cxa.cxa_device_status(1) == cxa.CXA_ETIMEOUT    # reported, and cleared
    assert cxa.cxa_device_status(0) == cxa.CXA_OK
    # the context is still usable
    w = W.custom("after_timeout", B=2, T=100, d=128, L=1, H=2, index=990)
    d, h = inputs_on_device(w)
    c = cache_for(w, "f32")
    c.populate(d["E"], d["WK"], d["WV"], d["bV"])
    Q = W.make_Q(w, 0)
    out = host(c.decode(dev(Q), d["key_len"]))
    ref = O.decode(Q, host(c.Kc), host(c.Vc), h["key_len"])
    assert np.abs(out - ref).max() <= DECODE_F32_MAX_ABS
    assert cxa.cxa_device_status(0) == cxa.CXA_OK


def test_selftest_rejects_bad_limits():
    assert cxa.cxa_selftest_wait_timeout(0) == cxa.CXA_EINVAL
    assert cxa.cxa_selftest_wait_timeout(1000001) == cxa.CXA_EINVAL


@pytest.mark.parametrize("what", ["decode_shared", "attend", "populate"])
def test_calls_from_a_thread_that_has_used_no_cuda_yet(what):
    """Tensor maps are encoded in the calling thread, which then needs a current context: the
    library binds it, whatever the thread has called before."""
    w = W.custom("fresh_thread", B=2, T=100, d=128, L=1, H=2, index=991)
    d, _ = inputs_on_device(w)
    c = cache_for(w, "bf16")
    c.populate(d["E"], d["WK"], d["WV"], d["bV"])
    stream = torch.cuda.current_stream().cuda_stream
    if what == "attend":
        p = cxa.PagedCache(8, 16, 1, 2, 64)
        q = torch.ones(40, 2, 64, dtype=torch.bfloat16, device="cuda")
        at = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 40], [40], [[0, 1, 2]])]
        ws, out = p.workspace(2, 40), torch.empty_like(q)
        rc = lambda: cxa.cxa_paged_attention(p.handle, 0, 1, 40, 40, *at, 3, q, 128, 2, out, 128, 0.0, cxa.CXA_BF16, ws,
                                             ws.numel(), stream)
    elif what == "decode_shared":
        Q = torch.ones(2, 3, 1, 2, 64, device="cuda")
        out = torch.empty_like(Q)
        n = cxa.cxa_decode_shared_workspace_bytes(2, 100, 1, 2, 64, 3)
        ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
        rc = lambda: cxa.cxa_decode_shared(c.handle, 3, Q, d["key_len"], out, 0.0, ws, n, stream)
    else:
        rc = lambda: c.populate(d["E"], d["WK"], d["WV"], d["bV"], stream=stream) or cxa.CXA_OK
    assert rc() == cxa.CXA_OK                               # here, where a context is current
    torch.cuda.synchronize()
    got = []
    t = threading.Thread(target=lambda: got.append((rc(), cxa.cxa_last_error_message())))
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert got and got[0][0] == cxa.CXA_OK, got
