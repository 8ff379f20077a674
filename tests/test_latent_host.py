"""Host side of the latent cache's, the gathered weights' and the eviction's calls: refusals, sizes and
the checks of batches. No GPU is needed: every call here returns before any CUDA call, and the device
pointers handed over are never dereferenced."""
import math
import os
import subprocess
import sys

import pytest

from encoder_decoder_speech_gb300 import cxa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7f0000000000          # 256-byte aligned, never dereferenced
BIG = 1 << 40


@pytest.fixture(autouse=True)
def _lib(cxa_lib):
    yield


def make_latent(Cp=FAKE, num_pages=10, page_size=16, L=2, latent=256, rope=32, dtype=cxa.CXA_BF16):
    return cxa.cxa_latent_create(Cp, num_pages, page_size, L, latent, rope, dtype)


def make_pages(num_pages=10, page_size=16, L=2, Hkv=4, dh=64, dtype=cxa.CXA_BF16):
    return cxa.cxa_pages_create(FAKE, FAKE + (1 << 32), num_pages, page_size, L, Hkv, dh, dtype)


@pytest.fixture
def latent():
    rc, h = make_latent()
    assert rc == cxa.CXA_OK
    yield h
    cxa.cxa_latent_destroy(h)


@pytest.fixture
def pages():
    rc, h = make_pages()
    assert rc == cxa.CXA_OK
    yield h
    cxa.cxa_pages_destroy(h)


def refused(rc, text):
    assert rc == cxa.CXA_EINVAL
    assert text in cxa.cxa_last_error_message()


BATCH = [(dict(layer=2), "layer"), (dict(layer=-1), "layer"), (dict(B=0), "B and max_pages"),
         (dict(B=(1 << 30) + 1), "2^30"), (dict(max_pages=0), "max_pages"), (dict(max_pages=1 << 27), "2^30"),
         (dict(kv_len=0), "NULL"), (dict(page_table=0), "NULL"), (dict(kv_len=FAKE + 2), "4-byte")]
TOKENS = [(dict(n_tokens=-1), "n_tokens"), (dict(q_start=0), "NULL"), (dict(q_start=FAKE + 1), "4-byte")]


def test_latent_create_refusals():
    refused(make_latent(Cp=0)[0], "NULL")
    refused(make_latent(Cp=FAKE + 8)[0], "aligned")
    for size in (0, 8, 24, 512, -16):
        refused(make_latent(page_size=size)[0], "page_size")
    for n in (0, 64, 192, 640, -128):
        refused(make_latent(latent=n)[0], "latent must be")
    for n in (-16, 8, 80, 24):
        refused(make_latent(rope=n)[0], "rope must be")
    refused(make_latent(num_pages=0)[0], "num_pages")
    refused(make_latent(L=0)[0], "L")
    refused(make_latent(L=65536)[0], "L")
    refused(make_latent(dtype=2)[0], "cache_dtype")


def append(h, **kw):
    a = dict(layer=0, B=2, n_tokens=5, q_start=FAKE, kv_len=FAKE, page_table=FAKE, max_pages=3, c=FAKE, c_stride=288,
             kr=FAKE + 512, kr_stride=288, norm=cxa.CXA_NORM_RMS, eps=1e-6, weight=None, rot=None,
             dtype=cxa.CXA_BF16, stream=0)
    a.update(kw)
    return cxa.cxa_latent_append(h, **a)


def test_append_refusals(latent):
    for kw, text in BATCH + TOKENS:
        refused(append(latent, **kw), text)
    refused(append(None), "descriptor is NULL")
    refused(append(latent, dtype=7), "dtype")
    refused(append(latent, norm=3), "norm")
    refused(append(latent, eps=-1.0), "eps")
    refused(append(latent, weight=FAKE + 2), "norm weights")
    refused(append(latent, c=0), "c is NULL")
    refused(append(latent, c=FAKE + 8), "c must be 16-byte aligned")
    refused(append(latent, c_stride=255), "row stride of c")
    refused(append(latent, c_stride=260), "row stride of c")
    refused(append(latent, kr=0), "kr is NULL")
    refused(append(latent, kr_stride=24), "row stride of kr")
    rc, rot = cxa.cxa_rotary_create(48, 0, [0.1] * 24)
    refused(append(latent, rot=rot), "more channels")
    cxa.cxa_rotary_destroy(rot)
    rc, f32 = make_latent(dtype=cxa.CXA_F32)
    refused(append(f32), "bf16 activations")
    cxa.cxa_latent_destroy(f32)
    before = cxa.cxa_launch_count()
    assert append(latent, n_tokens=0) == cxa.CXA_OK
    assert cxa.cxa_launch_count() == before


def attend(h, **kw):
    a = dict(layer=0, B=2, n_tokens=5, max_new=3, q_start=FAKE, kv_len=FAKE, page_table=FAKE, max_pages=3, q=FAKE,
             q_stride=8 * 288, H=8, out=FAKE + (1 << 30), o_stride=8 * 256, scale=0.1, dtype=cxa.CXA_BF16,
             workspace=FAKE + (1 << 31), workspace_bytes=BIG, stream=0)
    a.update(kw)
    return cxa.cxa_latent_attention(h, **a)


def test_attention_refusals(latent):
    for kw, text in BATCH + TOKENS:
        refused(attend(latent, **kw), text)
    refused(attend(None), "descriptor is NULL")
    for dtype in (cxa.CXA_F32, 9):
        refused(attend(latent, dtype=dtype), "the pool's")
    for H in (0, -1, 65536):
        refused(attend(latent, H=H), "H must")
    refused(attend(latent, max_new=0), "max_new")
    for scale in (0.0, -1.0, math.nan):
        refused(attend(latent, scale=scale), "scale must be positive")
    for scale in (math.inf, 3e38):
        refused(attend(latent, scale=scale), "scale must be finite")
    refused(attend(latent, q=0), "q is NULL")
    refused(attend(latent, q_stride=8 * 288 - 8), "row stride of q")
    refused(attend(latent, out=FAKE + (1 << 30) + 2), "out must be 16-byte aligned")
    refused(attend(latent, o_stride=8), "row stride of out")
    refused(attend(latent, out=FAKE + 5 * 8 * 288 * 2 - 16), "overlap")
    refused(attend(latent, q=FAKE + 5 * 8 * 256 * 2 - 16, out=FAKE), "overlap")
    refused(attend(latent, workspace=0), "workspace")
    refused(attend(latent, workspace=FAKE + 128), "256-byte")
    need = cxa.cxa_latent_attention_workspace_bytes(8, 256, 3, cxa.CXA_BF16)
    refused(attend(latent, workspace_bytes=need - 1), "workspace smaller")
    refused(attend(latent, n_tokens=1 << 28, H=8), "too many query rows")
    refused(attend(latent, B=1 << 20, max_pages=1 << 20), "below 2^31")
    assert attend(latent, n_tokens=0) == cxa.CXA_OK


def test_workspace_sizes(pages):
    size = cxa.cxa_latent_attention_workspace_bytes
    assert size(8, 256, 1, cxa.CXA_BF16) > 2 * 152 * 16 * 256 * 4
    assert size(8, 256, 1, cxa.CXA_BF16) < size(8, 256, 4, cxa.CXA_BF16) < size(8, 512, 4, cxa.CXA_BF16)
    for bad in ((0, 256, 1, 0), (8, 100, 1, 0), (8, 256, 0, 0), (8, 256, 1, 5), (70000, 256, 1, 0)):
        assert size(*bad) == 0
    size = cxa.cxa_paged_weights_workspace_bytes
    base = size(pages, 2, 100, 50, 3, 8)
    assert base >= cxa.CXA_PAGED_COUNTER_BYTES + 100 * 8 * 4
    # the scores of single tokens, unless they take more than 256 MB
    assert size(pages, 2, 2, 1, 80, 8) >= 2 * 4 * 80 * 16 * 2 * 4 + cxa.CXA_PAGED_COUNTER_BYTES
    assert size(pages, 64, 64, 1, 1 << 16, 8) < base + (1 << 20)
    for bad in ((None, 2, 100, 3, 3, 8), (pages, 0, 1, 1, 3, 8), (pages, 1, -1, 1, 3, 8), (pages, 1, 1, 0, 3, 8),
                (pages, 1, 1, 1, 0, 8), (pages, 1, 1, 1, 1 << 27, 8), (pages, 1, 1, 1, 3, 6), (pages, 1, 1, 1, 3, 0)):
        assert size(*bad) == 0


def expand(h, to, **kw):
    a = dict(layer=0, to=to, to_layer=0, B=2, from_=None, kv_len=FAKE, page_table=FAKE, max_pages=3, to_table=FAKE,
             to_max_pages=3, WK=FAKE, WV=FAKE, stream=0)
    a.update(kw)
    return cxa.cxa_latent_expand(h, **a)


def test_expand_refusals(latent, pages):
    for kw, text in BATCH:
        refused(expand(latent, pages, **kw), text)
    refused(expand(None, pages), "descriptor is NULL")
    refused(expand(latent, None), "descriptor is NULL")
    refused(expand(latent, pages, to_layer=2), "layer")
    refused(expand(latent, pages, to_max_pages=0), "max_pages")
    refused(expand(latent, pages, to_table=0), "NULL")
    refused(expand(latent, pages, from_=FAKE + 1), "from")
    refused(expand(latent, pages, WK=0), "WK or WV")
    refused(expand(latent, pages, WV=FAKE + 8), "WK or WV")
    refused(expand(latent, pages, B=1 << 24, max_pages=1 << 20), "below 2^31")
    rc, wide = make_latent(rope=64)
    refused(expand(wide, pages), "rope must be less")
    cxa.cxa_latent_destroy(wide)
    rc, f32 = make_pages(dtype=cxa.CXA_F32)
    refused(expand(latent, f32), "one type")
    cxa.cxa_pages_destroy(f32)


def weights(h, **kw):
    a = dict(layer=0, B=2, n_tokens=5, max_new=3, q_start=FAKE, kv_len=FAKE, page_table=FAKE, max_pages=3, q=FAKE,
             q_stride=512, Hq=8, weights=FAKE, decay=1.0, scale=0.0, dtype=cxa.CXA_BF16, workspace=FAKE,
             workspace_bytes=BIG, stream=0)
    a.update(kw)
    return cxa.cxa_paged_weights(h, **a)


def test_weights_refusals(pages):
    for kw, text in BATCH + TOKENS:
        refused(weights(pages, **kw), text)
    refused(weights(None), "descriptor is NULL")
    for dtype in (cxa.CXA_F32, 9):
        refused(weights(pages, dtype=dtype), "the pool's")
    for Hq in (0, 6, 65540):
        refused(weights(pages, Hq=Hq), "Hq must")
    refused(weights(pages, max_new=0), "max_new")
    for decay in (-0.5, math.nan, math.inf):
        refused(weights(pages, decay=decay), "decay")
    refused(weights(pages, scale=math.nan), "scale")
    refused(weights(pages, scale=3e38), "scale")
    refused(weights(pages, q=0), "q is NULL")
    refused(weights(pages, q_stride=500), "row stride of q")
    refused(weights(pages, weights=0), "weights is NULL")
    refused(weights(pages, weights=FAKE + 2), "weights")
    refused(weights(pages, workspace=FAKE + 64), "256-byte")
    refused(weights(pages, workspace_bytes=1000), "workspace smaller")
    refused(weights(pages, n_tokens=1 << 30), "too many query rows")
    refused(weights(pages, B=1 << 20, max_pages=1 << 20), "below 2^31")
    assert weights(pages, n_tokens=0) == cxa.CXA_OK


def evict(h, **kw):
    a = dict(l0=0, nl=2, weights=FAKE, B=2, keep=20, first=2, recent=4, kv_len=FAKE, page_table=FAKE, max_pages=3,
             out_table=FAKE, out_max_pages=2, kept=FAKE, out_len=FAKE + 64, stream=0)
    a.update(kw)
    return cxa.cxa_paged_evict(h, **a)


def test_evict_refusals(pages):
    for kw, text in BATCH:
        kw = {("l0" if k == "layer" else k): v for k, v in kw.items()}
        refused(evict(pages, **kw), text)
    refused(evict(None), "descriptor is NULL")
    refused(evict(pages, nl=0), "layers")
    refused(evict(pages, l0=1, nl=2), "layers")
    for kw in (dict(keep=0), dict(first=-1), dict(recent=-1), dict(first=17), dict(first=2 ** 31 - 1, recent=2 ** 31 - 1)):
        refused(evict(pages, **kw), "keep must be positive")
    refused(evict(pages, out_max_pages=0), "max_pages")
    refused(evict(pages, out_table=0), "NULL")
    refused(evict(pages, weights=0), "weights, kept or out_len")
    refused(evict(pages, kept=0), "weights, kept or out_len")
    refused(evict(pages, out_len=FAKE + 66), "weights, kept or out_len")
    refused(evict(pages, out_len=FAKE + 4), "overlap kv_len")
    refused(evict(pages, B=1 << 28, out_len=FAKE + BIG), "below 2^31")


def test_evict_check(pages):
    ok = dict(B=2, keep=20, kv_len=[40, 10], page_table=[0, 1, 2, 3, -1, -1], max_pages=3, out_table=[4, 5, 6, 99],
              out_max_pages=2)
    call = lambda **kw: cxa.cxa_paged_evict_check(pages, **dict(ok, **kw))
    assert call() == cxa.CXA_OK
    assert call(kv_len=[40, 0], out_table=[4, 5, -1, -1]) == cxa.CXA_OK
    refused(call(kv_len=[49, 10]), "passes the table's row")
    refused(call(kv_len=[-1, 10]), "negative")
    refused(call(page_table=[0, 1, 10, 3, -1, -1]), "page_table entry 2")
    refused(call(out_table=[4, -1, 6, 99]), "out_table entry 1")
    refused(call(out_table=[4, 3, 6, 99]), "still read")
    refused(call(out_table=[4, 5, 5, 99]), "written twice")
    refused(call(keep=0), "keep")
    refused(call(keep=33, kv_len=[40, 10]), "row of out_table")
    with pytest.raises(ValueError):
        call(kv_len=[2 ** 31, 1])
    with pytest.raises(ValueError):
        call(out_table=[1])


def test_latent_check(latent):
    call = lambda qs, kv, table: cxa.cxa_latent_check(latent, len(kv), 5, qs, kv, table, 2)
    assert call([0, 3, 5], [3, 20], [0, -1, 1, 2]) == cxa.CXA_OK
    refused(call([0, 3, 2], [3, 20], [0, -1, 1, 2]), "decrease")
    refused(call([0, 3, 5], [2, 20], [0, -1, 1, 2]), "less than the new tokens")
    refused(call([0, 3, 5], [3, 33], [0, -1, 1, 2]), "passes the table's row")
    refused(call([0, 3, 5], [3, 20], [0, -1, 1, 10]), "not a page")
    refused(call([0, 3, 5], [3, 20], [0, -1, 0, 2]), "another's")


def test_python_refusals_without_a_device():
    """What the Python classes refuse themselves, on tensors of the host."""
    import torch
    c = cxa.LatentCache(4, 16, 1, 128, 16, "f32", device="cpu")
    with pytest.raises(ValueError):
        c.attend(0, torch.zeros(1, 2, 144), torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32),
                 torch.zeros(1, 1, dtype=torch.int32), max_new=1, scale=1.0)
    for kw in (dict(latent=100), dict(rope=8), dict(page_size=20)):
        with pytest.raises(cxa.CxaError):
            cxa.LatentCache(**dict(dict(num_pages=4, page_size=16, L=1, latent=128, rope=16, device="cpu"), **kw))


def test_room_for_scores(pages):
    """The least workspace has room for the scores of tables that can need 256 MB; in wider ones room is the caller's."""
    least, room = cxa.cxa_paged_weights_workspace_bytes, cxa.cxa_paged_weights_room_bytes
    assert room(pages, 2, 2, 1, 80, 8) == least(pages, 2, 2, 1, 80, 8)
    # (160 positions of the pool, in 64 sequences: 66 chunks of 128 keys a head)
    assert room(pages, 64, 64, 1, 1 << 16, 8) == least(pages, 64, 64, 1, 1 << 16, 8) + 66 * 4 * 2 * 512
    big = make_pages(num_pages=1 << 24)[1]
    assert room(big, 64, 64, 1, 1 << 16, 8) == least(big, 64, 64, 1, 1 << 16, 8) + (256 << 20)
    cxa.cxa_pages_destroy(big)
    assert room(pages, 1, 2000, 2000, 1 << 16, 8) == least(pages, 1, 2000, 2000, 1 << 16, 8)      # no sequence of few rows
    assert room(pages, 1, 1, 1, 3, 6) == 0 and room(None, 1, 1, 1, 3, 8) == 0


def test_weights_of_calls_that_can_be_numbered_are_not_refused():
    """65,536 tokens of 4 heads a K/V head, 8 K/V heads, over a table of 2^20 positions: 1,025 tiles of 256 rows a head,
    8,193 chunks each, in bf16. In a process that sees no GPU, where a call that passes every check ends with CXA_ECUDA."""
    code = """if True:
        from encoder_decoder_speech_gb300 import cxa
        rc, p = cxa.cxa_pages_create(1 << 46, 1 << 47, 5000, 256, 1, 8, 64, {t})
        assert rc == cxa.CXA_OK
        rc = cxa.cxa_paged_weights(p, 0, {B}, {n}, {m}, 1 << 40, 1 << 40, 1 << 40, {w}, 1 << 45, 2048, 32, 1 << 48, 1.0, 0.0,
                                   {t}, 1 << 40, 1 << 40, 0)
        print(rc, cxa.cxa_last_error_message())
    """
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")

    def call(**kw):
        a = dict(dict(t=cxa.CXA_BF16, B=1, n=65536, m=65536, w=4096), **kw)
        r = subprocess.run([sys.executable, "-c", code.format(**a)], env=env, cwd=ROOT, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return r.stdout

    for kw in (dict(), dict(t=cxa.CXA_F32), dict(B=1000, m=1), dict(n=1 << 20, m=100, w=4096)):
        assert call(**kw).startswith(str(cxa.CXA_ECUDA)), kw
    for kw in (dict(B=1 << 15), dict(n=1 << 18, t=cxa.CXA_F32), dict(n=1 << 22, m=100)):
        out = call(**kw)
        assert out.startswith(str(cxa.CXA_EINVAL)) and "below 2^31" in out, kw
