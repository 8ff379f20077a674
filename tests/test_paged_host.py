"""Host side of the paged self-attention calls: frequencies, refusals and the batch check.
No GPU is needed: every call here returns before any CUDA call, and the device pointers
handed over are never dereferenced."""
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


def make_pages(num_pages=10, page_size=16, L=2, Hkv=4, dh=64, dtype=cxa.CXA_BF16, Kp=FAKE, Vp=FAKE + (1 << 32)):
    return cxa.cxa_pages_create(Kp, Vp, num_pages, page_size, L, Hkv, dh, dtype)


@pytest.fixture
def pages():
    rc, h = make_pages()
    assert rc == cxa.CXA_OK
    yield h
    cxa.cxa_pages_destroy(h)


def refused(rc, text):
    assert rc == cxa.CXA_EINVAL
    assert text in cxa.cxa_last_error_message()


# ------------------------------------------------------------------ rotations
@pytest.mark.parametrize("rot", [2, 6, 64, 128])
def test_frequencies_follow_their_formulas(rot):
    rc, f, att = cxa.cxa_rotary_frequencies(rot, 10000.0, cxa.CXA_ROTARY_PLAIN)
    assert rc == cxa.CXA_OK and att == 1.0
    plain = [10000.0 ** (-2 * i / rot) for i in range(rot // 2)]
    assert f == pytest.approx(plain, rel=1e-14)
    _, f, att = cxa.cxa_rotary_frequencies(rot, 10000.0, cxa.CXA_ROTARY_LINEAR, 4.0)
    assert f == pytest.approx([x / 4 for x in plain], rel=1e-14) and att == 1.0
    _, f, _ = cxa.cxa_rotary_frequencies(rot, 10000.0, cxa.CXA_ROTARY_NTK, 4.0)
    base = 10000.0 * 4.0 ** (rot / (rot - 2)) if rot > 2 else 10000.0
    assert f == pytest.approx([base ** (-2 * i / rot) for i in range(rot // 2)], rel=1e-13)
    if rot > 2:     # the slowest pair is slowed down by exactly the factor
        assert f[-1] == pytest.approx(plain[-1] / 4, rel=1e-13)
    _, f, att = cxa.cxa_rotary_frequencies(rot, 10000.0, cxa.CXA_ROTARY_WAVELENGTH, 4.0, 2048.0, 1.0, 32.0)
    assert att == pytest.approx(0.1 * math.log(4.0) + 1)
    for x, y in zip(plain, f):
        turns = 2048 * x / (2 * math.pi)
        if turns >= 32:
            assert y == pytest.approx(x, rel=1e-14)
        elif turns <= 1:
            assert y == pytest.approx(x / 4, rel=1e-14)
        else:
            keep = (turns - 1) / 31
            assert y == pytest.approx(keep * x + (1 - keep) * x / 4, rel=1e-14)


def test_frequency_and_rotation_refusals():
    bad = lambda *a: cxa.cxa_rotary_frequencies(*a)[0]
    refused(bad(0, 1e4, 0), "rot_dim")
    refused(bad(7, 1e4, 0), "rot_dim")
    refused(bad(130, 1e4, 0), "rot_dim")
    refused(bad(64, 1.0, 0), "base")
    refused(bad(64, math.nan, 0), "base")
    refused(bad(64, 1e4, 9), "scaling")
    refused(bad(64, 1e4, cxa.CXA_ROTARY_LINEAR, 0.5), "factor")
    refused(bad(64, 1e4, cxa.CXA_ROTARY_WAVELENGTH, 2.0, 0.0), "orig_len")
    refused(bad(64, 1e4, cxa.CXA_ROTARY_WAVELENGTH, 2.0, 100.0, 3.0, 3.0), "alpha")
    mk = lambda *a: cxa.cxa_rotary_create(*a)[0]
    refused(mk(64, 0, None), "freq")
    refused(mk(64, 5, [0.1] * 32), "layout")
    refused(mk(63, 0, [0.1] * 31), "rot_dim")
    refused(mk(4, 0, [0.1, -1.0]), "frequencies")
    refused(mk(4, 0, [0.1, math.inf]), "frequencies")
    refused(mk(4, 0, [0.1, 1.0], math.nan), "attn_factor")
    with pytest.raises(ValueError):
        cxa.Rotary(64, layout="other")
    with pytest.raises(ValueError):
        cxa.Rotary(64, freq=[0.1])
    with pytest.raises(cxa.CxaError):
        cxa.Rotary(66 * 2)


def test_norm_rope_refusals():
    ok = dict(q=FAKE, q_stride=512, Hq=8, k=FAKE + (1 << 20), k_stride=512, Hk=8, dh=64, n_tokens=3, pos=FAKE,
              norm=cxa.CXA_NORM_RMS, eps=1e-6, q_weight=0, k_weight=0, rot=None, q_out=FAKE, qo_stride=512,
              k_out=FAKE, ko_stride=512, dtype=cxa.CXA_BF16, stream=0)
    call = lambda **kw: cxa.cxa_qk_norm_rope(**dict(ok, **kw))
    refused(call(dh=32), "head_dim")
    refused(call(dtype=3), "dtype")
    refused(call(Hq=0, Hk=0), "Hq and Hk")
    refused(call(n_tokens=-1), "n_tokens")
    refused(call(norm=2), "norm")
    refused(call(eps=-1.0), "eps")
    refused(call(eps=math.nan), "eps")
    refused(call(pos=0), "pos")
    refused(call(q=0), "q is NULL")
    refused(call(q=FAKE + 8), "q must be 16-byte aligned")
    refused(call(q_stride=508), "row stride of q")
    refused(call(q_stride=516), "row stride of q")            # not a multiple of 16 bytes
    refused(call(k_stride=256), "row stride of k")
    refused(call(k_out=0), "k_out is NULL")
    refused(call(q_weight=FAKE + 2), "norm weights")
    rc, rot = cxa.cxa_rotary_create(128, 0, [0.1] * 64)
    refused(call(rot=rot), "more channels than a head has")
    cxa.cxa_rotary_destroy(rot)
    before = cxa.cxa_launch_count()
    assert call(n_tokens=0) == cxa.CXA_OK
    assert cxa.cxa_launch_count() == before


# ------------------------------------------------------------------ pages
def test_pages_create_refusals():
    refused(make_pages(Kp=0)[0], "NULL")
    refused(make_pages(Vp=FAKE + 4)[0], "aligned")
    for size in (0, 8, 24, 512, -16):
        refused(make_pages(page_size=size)[0], "page_size")
    refused(make_pages(num_pages=0)[0], "num_pages")
    refused(make_pages(num_pages=1 << 29)[0], "2^31")
    refused(make_pages(L=0)[0], "positive")
    refused(make_pages(Hkv=70000)[0], "65535")
    refused(make_pages(dh=96)[0], "head_dim")
    refused(make_pages(dtype=2)[0], "cache_dtype")


def append(pages, **kw):
    a = dict(layer=0, B=2, n_tokens=5, q_start=FAKE, kv_len=FAKE, page_table=FAKE, max_pages=3, k=FAKE, k_stride=256,
             v=FAKE, v_stride=256, q=None, q_stride=0, Hq=0, q_out=None, qo_stride=0, norm=0, eps=0.0, q_weight=None,
             k_weight=None, rot=None, dtype=cxa.CXA_BF16, stream=0)
    a.update(kw)
    return cxa.cxa_paged_append(pages, **a)


def attention(pages, **kw):
    a = dict(layer=0, B=2, n_tokens=5, max_new=4, q_start=FAKE, kv_len=FAKE, page_table=FAKE, max_pages=3, q=FAKE,
             q_stride=512, Hq=8, out=FAKE + (1 << 20), o_stride=512, scale=0.0, dtype=cxa.CXA_BF16, workspace=FAKE,
             workspace_bytes=BIG, stream=0)
    a.update(kw)
    return cxa.cxa_paged_attention(pages, **a)


@pytest.mark.parametrize("call", [append, attention])
def test_batch_refusals(pages, call):
    refused(call(None), "descriptor is NULL")
    refused(call(pages, layer=2), "layer")
    refused(call(pages, layer=-1), "layer")
    refused(call(pages, B=0), "B and max_pages")
    refused(call(pages, n_tokens=-1), "n_tokens")
    refused(call(pages, max_pages=0), "max_pages")
    refused(call(pages, max_pages=(1 << 26) + 1), "2^30")
    refused(call(pages, q_start=0), "NULL")
    refused(call(pages, kv_len=FAKE + 1), "aligned")
    refused(call(pages, dtype=9), "dtype")
    rc, f32 = make_pages(dtype=cxa.CXA_F32)
    refused(call(f32), "bf16 pool")
    cxa.cxa_pages_destroy(f32)
    before = cxa.cxa_launch_count()
    assert call(pages, n_tokens=0) == cxa.CXA_OK
    assert cxa.cxa_launch_count() == before


def test_append_refusals(pages):
    refused(append(pages, k=0), "k is NULL")
    refused(append(pages, v=FAKE + 2), "v must be 16-byte aligned")
    refused(append(pages, v_stride=64), "row stride of v")
    refused(append(pages, q=FAKE, Hq=0), "Hq")
    refused(append(pages, q=FAKE, Hq=8, q_stride=512, q_out=None), "q_out is NULL")
    refused(append(pages, norm=1, eps=-1.0), "eps")


def test_attention_refusals(pages):
    refused(attention(pages, Hq=6), "multiple")
    refused(attention(pages, Hq=0), "multiple")
    refused(attention(pages, max_new=0), "max_new")
    refused(attention(pages, scale=math.inf), "scale")
    refused(attention(pages, out=FAKE), "overlap")
    refused(attention(pages, out=FAKE + 512), "overlap")
    refused(attention(pages, workspace=0), "workspace")
    refused(attention(pages, workspace=FAKE + 16), "256-byte")
    need = cxa.cxa_paged_attention_workspace_bytes(8, 4, 64, 4)
    assert need > 0
    refused(attention(pages, workspace_bytes=need - 1), "workspace smaller")
    refused(attention(pages, n_tokens=1 << 30, Hq=8), "too many query rows")
    refused(attention(pages, B=1 << 17, max_pages=1 << 18), "below 2^31")
    for args in [(8, 3, 64, 1), (8, 4, 32, 1), (8, 4, 64, 0), (0, 4, 64, 1), (8, 0, 64, 1)]:
        assert cxa.cxa_paged_attention_workspace_bytes(*args) == 0


def test_batch_check_finds_what_the_kernels_would_leave_out(pages):
    good = dict(B=2, n_tokens=6, q_start=[0, 1, 5], kv_len=[17, 40], page_table=[3, 4, -1, 9, 0, 7], max_pages=3)
    chk = lambda **kw: cxa.cxa_paged_check(pages, **dict(good, **kw))
    assert chk() == cxa.CXA_OK
    refused(chk(page_table=[3, -1, -1, 9, 0, 7]), "entry 1 is not a page of the pool (sequence 0)")
    refused(chk(page_table=[3, 10, -1, 9, 0, 7]), "entry 1 is not a page")
    refused(chk(page_table=[3, 4, -1, 9, 0, -5]), "entry 2 is not a page of the pool (sequence 1)")
    refused(chk(q_start=[1, 1, 5]), "q_start[0]")
    refused(chk(q_start=[0, 3, 2]), "must not decrease")
    refused(chk(q_start=[0, 1, 7]), "pass n_tokens")
    refused(chk(kv_len=[0, 40]), "less than the new tokens")
    refused(chk(kv_len=[-3, 40]), "less than the new tokens")
    refused(chk(kv_len=[17, 49]), "passes the table's row")
    refused(chk(page_table=[3, 7, -1, 9, 0, 7]), "two sequences or positions write one page")
    refused(chk(page_table=[7, 4, -1, 9, 0, 7]), "is another's")
    refused(chk(page_table=[3, 4, -1, 9, 7, 7]), "is another's")
    assert chk(page_table=[9, 4, -1, 9, 0, 7]) == cxa.CXA_OK           # a shared prefix page
    assert chk(q_start=[0, 0, 4], page_table=[-1, -1, -1, 9, 0, 7]) == cxa.CXA_OK   # nothing new: not looked at
    assert cxa.cxa_strerror(cxa.CXA_EPAGE).startswith("CXA_EPAGE")


def test_workspace_holds_its_counters_and_a_part_for_each_kernel():
    import pathlib
    import re
    header = (pathlib.Path(__file__).parents[1] / "include" / "cxa.h").read_text()
    assert int(re.search(r"#define CXA_PAGED_COUNTER_BYTES (\d+)", header)[1]) == cxa.CXA_PAGED_COUNTER_BYTES
    few = cxa.cxa_paged_attention_workspace_bytes(8, 8, 64, 16)
    many = cxa.cxa_paged_attention_workspace_bytes(8, 8, 64, 17)
    assert cxa.CXA_PAGED_COUNTER_BYTES < few < many
    assert many == cxa.cxa_paged_attention_workspace_bytes(16, 8, 64, 9)
    assert many < cxa.cxa_paged_attention_workspace_bytes(8, 8, 128, 17)
    for bad in ((0, 1, 64, 1), (8, 3, 64, 1), (8, 8, 32, 1), (8, 8, 64, 0)):
        assert cxa.cxa_paged_attention_workspace_bytes(*bad) == 0


def test_strides_that_no_tensor_map_holds_are_refused_before_anything_is_enqueued(pages):
    """Strides stay below 2^40 bytes, even where one token makes them unused, and rows times
    stride below what 64 bits of address hold. (The calls that pass stop at their workspace.)"""
    before = cxa.cxa_launch_count()
    for n in (1, 5):
        kw = dict(n_tokens=n, workspace=0)
        refused(attention(pages, q_stride=1 << 39, **kw), "row stride of q must")
        refused(attention(pages, q_stride=1 << 40, **kw), "row stride of q must")
        refused(attention(pages, o_stride=1 << 39, **kw), "row stride of out must")
        refused(attention(pages, q_stride=(1 << 39) - 8, out=FAKE - (1 << 20), **kw), "workspace")
        refused(append(pages, n_tokens=n, k_stride=1 << 39), "row stride of k must")
        refused(append(pages, n_tokens=n, v_stride=1 << 39), "row stride of v must")
    rc, f32 = make_pages(dtype=cxa.CXA_F32)
    refused(attention(f32, dtype=cxa.CXA_F32, q_stride=1 << 38, workspace=0), "row stride of q must")
    cxa.cxa_pages_destroy(f32)
    for n, stride in ((1 << 26, 1 << 31), (1 << 18, (1 << 39) - 8), ((1 << 28), 1 << 38)):
        refused(attention(pages, n_tokens=n, q_stride=stride, workspace=0), "rows of q span")
    assert cxa.cxa_launch_count() == before


def test_calls_that_can_be_numbered_are_not_refused():
    """65,536 tokens of 4 heads a K/V head, 8 K/V heads, over a table of 2^20 positions: 1,025
    tiles of 256 rows a head, 8,193 chunks each. In a process that sees no GPU, where a call that
    passes every check ends with CXA_ECUDA."""
    code = """if True:
        from encoder_decoder_speech_gb300 import cxa
        rc, p = cxa.cxa_pages_create(1 << 46, 1 << 47, 5000, 256, 1, 8, {dh}, cxa.CXA_BF16)
        assert rc == cxa.CXA_OK
        rc = cxa.cxa_paged_attention(p, 0, {B}, {n}, {m}, 1 << 40, 1 << 40, 1 << 40, {w}, 1 << 45, 32 * {dh}, 32, 1 << 48,
                                     32 * {dh}, 0.0, cxa.CXA_BF16, 1 << 40, 1 << 40, 0)
        print(rc, cxa.cxa_last_error_message())
    """
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")

    def call(**kw):
        a = dict(dict(dh=64, B=1, n=65536, m=65536, w=4096), **kw)
        r = subprocess.run([sys.executable, "-c", code.format(**a)], env=env, cwd=ROOT, capture_output=True, text=True)
        assert r.returncode == 0, r.stderr
        return r.stdout

    for kw in (dict(), dict(dh=128), dict(B=1000, m=64), dict(n=1 << 21, m=1 << 21, w=256)):
        assert call(**kw).startswith(str(cxa.CXA_ECUDA)), kw
    for kw in (dict(m=1), dict(B=1 << 14), dict(n=1 << 25, m=100), dict(n=1 << 24, m=100, dh=128)):
        out = call(**kw)
        assert out.startswith(str(cxa.CXA_EINVAL)) and "below 2^31" in out, kw


def test_batch_check_leaves_sequences_without_new_tokens_alone(pages):
    """Their keys and pages are not read by any kernel: a slot that is free may hold anything."""
    for kv in (-1, 0, 49, 2 ** 31 - 1, -2 ** 31):
        assert cxa.cxa_paged_check(pages, 2, 4, [0, 0, 4], [kv, 40], [-1, 99, -7, 9, 0, 7], 3) == cxa.CXA_OK
        assert cxa.cxa_paged_check(pages, 2, 4, [0, 4, 4], [40, kv], [9, 0, 7, 9, 99, 0], 3) == cxa.CXA_OK
        refused(cxa.cxa_paged_check(pages, 2, 4, [0, 1, 4], [kv, 40], [-1, 99, -7, 9, 0, 7], 3), "(sequence 0)")


def test_short_lists_of_frequencies_are_not_read_past_their_end():
    for rot, n in ((64, 0), (64, 1), (64, 31), (2, 0), (128, 63)):
        with pytest.raises(ValueError, match="rot_dim / 2"):
            cxa.cxa_rotary_create(rot, 0, [0.1] * n)


def test_batch_check_does_not_wrap_large_numbers(pages):
    """What 32 bits do not hold is refused, not taken for what its low bits are."""
    good = dict(q_start=[0, 1, 5], kv_len=[17, 40], page_table=[3, 4, -1, 9, 0, 7])
    for name, i, v in (("kv_len", 1, 2 ** 32 + 40), ("page_table", 0, 2 ** 32 + 3), ("q_start", 2, 5 - 2 ** 32)):
        kw = {k: list(x) for k, x in good.items()}
        assert cxa.cxa_paged_check(pages, 2, 6, **kw, max_pages=3) == cxa.CXA_OK
        kw[name][i] = v
        with pytest.raises(ValueError, match="32-bit"):
            cxa.cxa_paged_check(pages, 2, 6, **kw, max_pages=3)


@pytest.mark.parametrize("call", [append, attention])
def test_more_sequences_than_kernels_count_are_refused(pages, call):
    for B in (2 ** 30 + 1, 2 ** 31 - 1):
        refused(call(pages, B=B, workspace=0) if call is attention else call(pages, B=B), "at most 2^30")


def test_scales_that_overflow_in_base_two_are_refused(pages):
    """Scores are taken in powers of two: scale * log2(e) has to be a number."""
    for scale in (3e38, 2.4e38, math.inf, math.nan, -math.inf):
        refused(attention(pages, scale=scale, workspace=0), "scale must be finite")
    for scale in (2.3e38, 1.0, 0.0, -1.0, -3e38):
        refused(attention(pages, scale=scale, workspace=0), "workspace")
