"""The latent cache on the GPU (append, absorbed attention, expansion) against plain fp64 forms written
out here.

Tolerances, per element, count roundings: u is half a step of the output type (bf16 2^-8, fp32 2^-24).

* Append: |got - ref| <= u |ref| + 2^-19 M, M the magnitudes added for an element: fp32 steps of the norm
  (sums of up to 512 squares, 16 a lane and 5 exchanges, rsqrt, weight) and the sine and cosine (a phase
  rounded to 24 bits of half a turn: pi * 2^-24).
* Attention: |got - ref| <= u |ref| + (e_p + e_s) A, A = sum p |c| of the row. e_p: bf16 weights 2^-8, and for
  both types 2^-21 for ex2, one step of 2^-24 an addition (fp32: a key each; bf16: 16 keys each, truncated,
  2^-23) and 64 more for rescaling and merging. e_s is that of the scores, twice (numerator and
  reference) the steps of the sum of latent + rope products, 2^-23 for each of 16 of them (bf16) or 2^-24 for each
  of the 18 of a lane and the 5 exchanges (fp32), times scale * max sum |q||row|.
* Expansion: |got - ref| <= u |ref| + (steps) sum |c||W|: 2^-23 for each 16 channels in bf16, 2^-24 for each
  channel in fp32.
"""
import math
import threading

import pytest
import torch

from encoder_decoder_speech_gb300 import cxa

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
U = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _lib(cxa_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    yield
    torch.cuda.synchronize()
    assert cxa.cxa_device_status(1) == cxa.CXA_OK


def randn(*shape, seed, dtype=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


class Batch:
    """Sequences with n new tokens of kv keys each, in shuffled latent pages."""

    def __init__(self, n, kv, page=16, H=8, latent=128, rope=32, pool="bf16", seed=0, L=1, layer=0, spare=3, pad=0,
                 extra_cols=1):
        self.n, self.kv, self.page, self.H, self.latent, self.rope, self.layer = n, kv, page, H, latent, rope, layer
        self.B, self.width, self.scale = len(n), latent + rope, 1.0 / math.sqrt(latent + rope)
        need = [-(-max(k, 0) // page) for k in kv]
        P = sum(need) + spare
        self.cache = cxa.LatentCache(P, page, L, latent, rope, pool)
        g = torch.Generator().manual_seed(seed + 77)
        perm = torch.randperm(P, generator=g).tolist()
        self.table = torch.full((self.B, max(need + [0]) + extra_cols), -1, dtype=torch.int32)
        for b in range(self.B):
            for i in range(need[b]):
                self.table[b, i] = perm.pop()
        starts = [0]
        for x in n:
            starts.append(starts[-1] + x)
        self.starts, self.N = starts, starts[-1] + pad
        self.q = randn(self.N, H, self.width, seed=seed + 1, dtype=DT[pool])
        self.C = [randn(max(k, 0), self.width, seed=seed + 100 + b, dtype=DT[pool]) for b, k in enumerate(kv)]
        self.d = dict(q_start=torch.tensor(starts, dtype=torch.int32).cuda(),
                      kv_len=torch.tensor(kv, dtype=torch.int32).cuda(), page_table=self.table.cuda())
        self.max_new = max(n + [1])

    def fill(self, rest=None):
        """Write every key's row into its page; all other rows of the pool hold `rest`."""
        Cp = self.cache.Cp[self.layer].cpu()
        if rest is not None:
            Cp.fill_(rest)
        for b in range(self.B):
            for t in range(0, self.kv[b], self.page):
                p, m = int(self.table[b, t // self.page]), min(self.page, self.kv[b] - t)
                Cp[p, :m] = self.C[b][t:t + m]
        self.cache.Cp[self.layer].copy_(Cp)
        return self

    def attend(self, q=None, **kw):
        kw.setdefault("max_new", self.max_new)
        kw.setdefault("scale", self.scale)
        return self.cache.attend(self.layer, (self.q if q is None else q).cuda(), **self.d, **kw)

    def reference(self, scale=None):
        """out, sum p |c|, and the largest scale * sum |q||row|, in fp64."""
        scale = scale or self.scale
        out = torch.zeros(self.N, self.H, self.latent, dtype=torch.float64, device="cuda")
        A = torch.zeros_like(out)
        big = 0.0
        for b in range(self.B):
            n, kv = self.n[b], self.kv[b]
            if n == 0 or kv <= 0:
                continue
            q, C = self.q[self.starts[b]:self.starts[b + 1]].cuda().double(), self.C[b].cuda().double()
            big = max(big, float((q.abs() @ C.abs().T * scale).nan_to_num(0, 0, 0).max()))
            for i in range(n):
                see = max(0, min(kv, kv - n + i + 1))
                if see == 0:
                    continue
                p = torch.softmax(q[i] @ C[:see].T * scale, -1)
                out[self.starts[b] + i] = p @ C[:see, :self.latent]
                A[self.starts[b] + i] = p @ C[:see, :self.latent].abs()
        return out.cpu(), A.cpu(), big

    def close(self, got, scale=None):
        out, A, big = self.reference(scale)
        got = got.detach().cpu()
        keys = max(self.kv + [0])
        if got.dtype == torch.float32:
            e = 2.0 ** -21 + (keys + 64) * 2.0 ** -24 + 2 * 23 * 2.0 ** -24 * big
        else:
            e = 2.0 ** -8 + 2.0 ** -21 + (keys / 16 + 64) * 2.0 ** -23 + 2 * (self.width / 16 + 1) * 2.0 ** -23 * big
        rows = slice(0, self.starts[-1])
        fin = out.isfinite()[rows].all(-1)
        assert bool((got[rows].isfinite().all(-1) == fin).all())
        over = ((got.double() - out).abs() - U[got.dtype] * out.abs() - e * A)[rows][fin]
        assert over.numel() == 0 or float(over.max()) <= 0


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("act, pool", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("latent, rope", [(128, 0), (256, 32), (384, 48), (512, 64)])
@pytest.mark.parametrize("layout, norm", [("half", True), ("interleaved", False)])
def test_append(act, pool, latent, rope, layout, norm):
    n, kv, page = [1, 0, 37, 5], [1, 12, 50, 900], 32
    b = Batch(n, kv, page, 1, latent, rope, pool, seed=latent + rope, L=2, layer=1, pad=2).fill(7.0)
    before = b.cache.Cp.clone()
    row = randn(b.N, 24 + latent + rope, seed=5, dtype=DT[act])      # slices of wider rows
    c, kr = row[:, 8:8 + latent], row[:, 8 + latent:8 + latent + rope] if rope else None
    w = 1 + randn(latent, seed=6, scale=0.2)
    rot_dim = rope - 16 if rope > 32 else rope
    rotary = cxa.Rotary(rot_dim, layout=layout, attn_factor=1.25) if rope else None
    dev = row.cuda()
    b.cache.append(1, dev[:, 8:8 + latent], dev[:, 8 + latent:8 + latent + rope] if rope else None, **b.d,
                   rotary=rotary, norm_eps=1e-5 if norm else None, weight=w.cuda() if norm else None)
    got, want = b.cache.Cp.cpu(), before.cpu().double()
    mag = torch.zeros_like(want)
    for s in range(4):
        for i in range(n[s]):
            t = kv[s] - n[s] + i
            y = c[b.starts[s] + i].double()
            if norm:
                y = y / torch.sqrt((y * y).mean() + 1e-5) * w.double()
            m = y.abs()
            if rope:
                z = kr[b.starts[s] + i].double().clone()
                zm = z.abs()
                h = rot_dim // 2
                ang = t * torch.tensor(rotary.freq, dtype=torch.float64)
                co, si = 1.25 * torch.cos(ang), 1.25 * torch.sin(ang)
                lo, hi = (slice(0, h), slice(h, 2 * h)) if layout == "half" else (slice(0, 2 * h, 2), slice(1, 2 * h, 2))
                x0, x1 = z[lo].clone(), z[hi].clone()
                z[lo], z[hi] = x0 * co - x1 * si, x0 * si + x1 * co
                zm[lo] = zm[hi] = 1.25 * (x0.abs() + x1.abs())
                y, m = torch.cat([y, z]), torch.cat([m, zm])
            p = int(b.table[s, t // page])
            want[1, p, t % page], mag[1, p, t % page] = y, m
    same = mag == 0
    assert torch.equal(got.double()[same], want[same])              # nothing else is touched
    over = (got.double() - want).abs() - U[got.dtype] * want.abs() - 2.0 ** -19 * mag
    assert float(over.max()) <= 0


def test_append_leaves_out_bad_pages_and_rows_of_no_sequence():
    b = Batch([2, 1], [20, 3], 16, 1, 128, 16, "bf16", pad=3)
    b.table[0, 1] = 99
    b.d["page_table"] = b.table.cuda()
    before = b.cache.Cp.clone()
    x = torch.ones(b.N, 144, dtype=torch.bfloat16, device="cuda")
    b.cache.append(0, x[:, :128], x[:, 128:], **b.d)
    assert cxa.cxa_device_status(1) == cxa.CXA_EPAGE
    before[0, int(b.table[1, 0]), 2] = 1
    assert torch.equal(before, b.cache.Cp)


def test_append_with_weights_anywhere():
    """Norm weights need 4 bytes of alignment, no more."""
    b = Batch([1, 3], [20, 3], 16, 1, 384, 0, "bf16")
    b.cache.Cp.zero_()
    c = randn(b.N, 384, seed=3).cuda()
    w = randn(385, seed=4).cuda()
    b.cache.append(0, c, None, **b.d, norm_eps=1e-5, weight=w[1:].clone())
    want = b.cache.Cp.clone()
    b.cache.Cp.zero_()
    b.cache.append(0, c, None, **b.d, norm_eps=1e-5, weight=w[1:])
    assert torch.equal(b.cache.Cp, want) and float(want.float().abs().max()) > 0


# ------------------------------------------------------------------ attention
CASES = [
    dict(n=[1], kv=[1]),
    dict(n=[1], kv=[448], latent=256, rope=0),
    dict(n=[1, 1, 1], kv=[63, 64, 65], H=20, latent=512, rope=64),
    dict(n=[1], kv=[3000], H=128, latent=512, rope=64, page=64),
    dict(n=[1] * 7, kv=[5, 1000, 130, 17, 2049, 64, 700], H=16, latent=384, rope=48, page=32),
    dict(n=[5, 0, 1, 3], kv=[900, 40, 33, 3], H=8, latent=256, rope=16, page=128),
    dict(n=[33], kv=[33], H=20, latent=512, rope=64, page=256),
    dict(n=[40, 1, 7], kv=[300, 700, 7], H=6, latent=128, rope=0, page=64),
    dict(n=[3], kv=[9000], H=40, latent=512, rope=64, page=64),
    dict(n=[2, 1], kv=[70, 129], H=1, latent=512, rope=32, page=16),
    dict(n=[200], kv=[1000], H=3, latent=256, rope=64, page=64),
    dict(n=[1, 2], kv=[777, 65], H=66, latent=128, rope=16, page=32),
]


@pytest.mark.parametrize("pool", ["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_attention(i, pool):
    b = Batch(pool=pool, seed=10 * i, **CASES[i]).fill(float("nan"))
    b.close(b.attend())


@pytest.mark.parametrize("pool", ["bf16", "f32"])
@pytest.mark.parametrize("H, n", [(16, 1), (8, 4), (64, 1), (20, 3)])
def test_attention_over_a_long_context(pool, H, n):
    """Items cut between many blocks."""
    b = Batch([n], [40000], 128, H, 512, 64, pool, seed=H).fill(float("inf"))
    b.close(b.attend())


@pytest.mark.parametrize("pool", ["bf16", "f32"])
@pytest.mark.parametrize("H", [128, 45, 7])
def test_many_tiles_of_a_sequence(pool, H):
    """Tiles of equal numbers of chunks are numbered together: prompts alone, behind context, and cut off by their rows."""
    b = Batch([153, 1, 0, 70, 200], [153, 900, 5, 1500, 190], 32, H, 128, 16, pool, seed=H).fill(float("nan"))
    b.close(b.attend())


@pytest.mark.parametrize("pool", ["bf16", "f32"])
def test_scores_of_growing_size(pool):
    """References that move at every step, and scores far apart."""
    b = Batch([2, 1], [700, 650], 64, 20, 256, 32, pool, seed=3)
    for C in b.C:
        C.mul_(torch.linspace(0.1, 6, len(C))[:, None].to(C.dtype))
    b.fill(float("nan"))
    b.close(b.attend(scale=0.5), scale=0.5)


@pytest.mark.parametrize("pool", ["bf16", "f32"])
def test_a_larger_max_new_and_padding_rows(pool):
    b = Batch([1, 3, 2], [100, 300, 2], 16, 8, 256, 32, pool, pad=5).fill(float("nan"))
    out = torch.full((b.N, b.H, b.latent), 9.0, dtype=DT[pool], device="cuda")
    got = b.attend(max_new=50, out=out)
    assert got is out and bool((out[b.starts[-1]:] == 9.0).all())
    b.close(out)


@pytest.mark.parametrize("pool", ["bf16", "f32"])
def test_rows_that_see_nothing_are_zero(pool):
    """kv_len below the new tokens (against the batch's contract): the first of them see no key."""
    b = Batch([4, 1], [2, 0], 16, 8, 128, 16, pool, extra_cols=2).fill(float("nan"))
    got = b.attend().cpu()
    assert not bool(got[:2].any()) and not bool(got[4].any())
    b.close(got)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("pool", ["bf16", "f32"])
def test_later_tokens_values_do_not_reach_earlier_ones(pool, value):
    b = Batch([6], [70], 64, 8, 256, 32, pool).fill(float("nan"))
    clean = b.attend().cpu()
    b.C[0][67, 5] = value               # seen by the last three tokens
    b.fill(float("nan"))
    got = b.attend().cpu()
    assert torch.equal(got[:3], clean[:3])
    if value != value:                  # (an infinity may leave a weight of 0, and 0 * inf undecided)
        assert not bool(got[3:, :, 5].isfinite().any())


@pytest.mark.parametrize("pool", ["bf16", "f32"])
def test_a_bad_page_is_reported_and_left_out(pool):
    b = Batch([1, 2], [200, 90], 32, 8, 256, 32, pool).fill(float("nan"))
    good = b.attend().cpu()
    b.table[0, 2] = 1000
    b.d["page_table"] = b.table.cuda()
    got = b.attend().cpu()
    assert cxa.cxa_device_status(1) == cxa.CXA_EPAGE
    assert torch.equal(got[1:], good[1:])
    b.C[0] = torch.cat([b.C[0][:64], b.C[0][96:]])
    b.kv[0] = 168                        # the same keys without the page's
    b.close(got)


@pytest.mark.parametrize("pool", ["bf16", "f32"])
def test_strided_queries_and_results(pool):
    b = Batch([3, 1], [90, 300], 64, 5, 128, 48, pool).fill(float("nan"))
    qw = torch.zeros(b.N, 5 * b.width + 16, dtype=DT[pool], device="cuda")
    ow = torch.full((b.N, 5 * 128 + 24), 3.0, dtype=DT[pool], device="cuda")
    q, out = qw[:, 8:8 + 5 * b.width].unflatten(1, (5, b.width)), ow[:, 16:16 + 5 * 128].unflatten(1, (5, 128))
    q.copy_(b.q)
    b.cache.attend(0, q, **b.d, max_new=3, scale=b.scale, out=out)
    b.close(out)
    assert bool((ow[:, :16] == 3.0).all()) and bool((ow[:, 16 + 640:] == 3.0).all())


@pytest.mark.parametrize("pool", ["bf16", "f32"])
def test_results_do_not_change_from_call_to_call(pool):
    b = Batch([1] * 9, [3000, 10, 900, 4000, 77, 2500, 1, 640, 2000], 64, 20, 512, 64, pool).fill(float("nan"))
    first = b.attend()
    for _ in range(5):
        assert torch.equal(b.attend(), first)


@pytest.mark.parametrize("pool", ["bf16", "f32"])
def test_graphs_and_streams_at_once(pool):
    bs = [Batch([1, 2], [5000 + 100 * i, 300], 64, 16, 256, 32, pool, seed=i).fill(float("nan")) for i in range(3)]
    want = [b.attend() for b in bs]
    graphs, outs = [], []
    for b in bs:
        q = b.q.cuda()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(b.cache.attend(0, q, **b.d, max_new=2, scale=b.scale))
        graphs.append((graph, q))
    streams = [torch.cuda.Stream() for _ in bs]
    torch.cuda.synchronize()
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    eager = []
    for b, (graph, _), s in zip(bs, graphs, streams):
        with torch.cuda.stream(s):
            graph.replay()
            eager.append(b.attend())
            graph.replay()
    torch.cuda.synchronize()
    for w, o, e in zip(want, outs, eager):
        assert torch.equal(w, o) and torch.equal(w, e)


def test_calls_from_threads():
    bs = [Batch([1], [3000 + i], 64, 16, 256, 32, "bf16", seed=i).fill() for i in range(4)]
    want = [b.attend() for b in bs]
    got = [None] * 4
    torch.cuda.synchronize()

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got[i] = bs[i].attend()
            torch.cuda.current_stream().synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    for w, g in zip(want, got):
        assert torch.equal(w, g)


def test_one_workspace_for_calls_of_all_shapes():
    a = Batch([1], [9000], 64, 64, 512, 64, "bf16").fill()
    b = Batch([1, 4], [700, 90], 16, 8, 128, 16, "bf16", seed=4).fill()
    c = Batch([2], [1500], 32, 3, 256, 0, "f32", seed=5).fill()
    ws = torch.full((cxa.cxa_latent_attention_workspace_bytes(64, 512, 1, cxa.CXA_BF16),), 255, dtype=torch.uint8,
                    device="cuda")
    for x in (a, b, c, a, c, b):
        x.close(x.attend(workspace=ws))


def test_python_refusals():
    b = Batch([1], [10]).fill()
    q = b.q.cuda()
    call = lambda q=q, **kw: b.cache.attend(0, q, **dict(dict(b.d, max_new=1, scale=1.0), **kw))
    with pytest.raises(cxa.CxaError):
        call(q=q.float())
    with pytest.raises(cxa.CxaError):
        call(scale=0.0)
    with pytest.raises(ValueError):
        call(q=q[..., :128])
    with pytest.raises(ValueError):
        call(kv_len=b.d["kv_len"].long())
    with pytest.raises(ValueError):
        call(out=torch.empty(1, 8, 64, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        call(q=b.q)
    x = torch.zeros(1, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        b.cache.append(0, x, None, **b.d)
    with pytest.raises(ValueError):
        b.cache.append(0, x, x[:, :16], **b.d)


# ------------------------------------------------------------------ expansion
EXPAND = [
    dict(kv=[1], start=None, H=1, dh=64, latent=128, rope=0, page=16, to_page=16),
    dict(kv=[300, 0, 64, 129], start=None, H=8, dh=64, latent=256, rope=32, page=16, to_page=64),
    dict(kv=[700, 65], start=[300, 64], H=20, dh=128, latent=512, rope=64, page=128, to_page=32),
    dict(kv=[40, 90, 7], start=[40, 200, -3], H=5, dh=128, latent=384, rope=16, page=32, to_page=256),
    dict(kv=[1000], start=[17], H=6, dh=64, latent=512, rope=48, page=256, to_page=16),
    dict(kv=[33] * 20, start=None, H=3, dh=64, latent=128, rope=16, page=64, to_page=128),
    dict(kv=[5000], start=None, H=2, dh=128, latent=256, rope=0, page=64, to_page=64),
]


def expand_case(kv, start, H, dh, latent, rope, page, to_page, pool, seed=0):
    b = Batch([0] * len(kv), kv, page, 1, latent, rope, pool, seed=seed).fill(float("nan"))
    need = [-(-k // to_page) for k in kv]
    to = cxa.PagedCache(sum(need) + 2, to_page, 2, H, dh, pool)
    to.Kp.fill_(5.0)
    to.Vp.fill_(6.0)
    perm = torch.randperm(sum(need) + 2, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(kv), max(need) + 1), -1, dtype=torch.int32)
    for s, m in enumerate(need):
        for i in range(m):
            table[s, i] = perm.pop()
    WK = randn(latent, H * (dh - rope), seed=seed + 1, dtype=DT[pool], scale=latent ** -0.5)
    WV = randn(latent, H * dh, seed=seed + 2, dtype=DT[pool], scale=latent ** -0.5)
    return b, to, table, WK, WV


@pytest.mark.parametrize("pool", ["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(EXPAND)))
def test_expand(i, pool):
    kw = EXPAND[i]
    b, to, table, WK, WV = expand_case(pool=pool, seed=i, **kw)
    H, dh, rope, latent, page = kw["H"], kw["dh"], kw["rope"], kw["latent"], kw["to_page"]
    start = None if kw["start"] is None else torch.tensor(kw["start"], dtype=torch.int32).cuda()
    b.cache.expand(0, WK.cuda(), WV.cuda(), b.d["kv_len"], b.d["page_table"], to, 1, table.cuda(), start=start)
    assert bool((to.Kp[0] == 5.0).all()) and bool((to.Vp[0] == 6.0).all())
    K, V = (torch.full(to.Kp[1].shape, x, dtype=torch.float64) for x in (5.0, 6.0))
    MK, MV = torch.zeros_like(K), torch.zeros_like(V)
    step = latent / 16 * 2.0 ** -23 if pool == "bf16" else latent * 2.0 ** -24
    for s, n in enumerate(kw["kv"]):
        c, r = b.C[s][:, :latent].double(), b.C[s][:, latent:].double()
        k, v = (c @ WK.double()).view(n, H, dh - rope), (c @ WV.double()).view(n, H, dh)
        mk, mv = (c.abs() @ WK.double().abs()).view(n, H, dh - rope), (c.abs() @ WV.double().abs()).view(n, H, dh)
        lo = max(0, kw["start"][s]) if kw["start"] else 0
        for t in range(lo, n):
            p, at = int(table[s, t // page]), t % page
            K[p, :, at, :rope], K[p, :, at, rope:], V[p, :, at] = r[t], k[t], v[t]
            MK[p, :, at, rope:], MV[p, :, at] = mk[t], mv[t]
    for got, want, mag in ((to.Kp[1].cpu(), K, MK), (to.Vp[1].cpu(), V, MV)):
        same = mag == 0                 # the rotated part, and all that no position is
        assert torch.equal(got.double()[same], want[same])
        over = (got.double() - want).abs() - U[got.dtype] * want.abs() - step * mag
        assert float(over.max()) <= 0


@pytest.mark.parametrize("pool", ["bf16", "f32"])
def test_expand_leaves_out_bad_pages(pool):
    kw = dict(kv=[100, 50], start=None, H=4, dh=64, latent=128, rope=16, page=32, to_page=16)
    b, to, table, WK, WV = expand_case(pool=pool, **kw)
    call = lambda t, to_t: b.cache.expand(0, WK.cuda(), WV.cuda(), b.d["kv_len"], t.cuda(), to, 1, to_t.cuda())
    call(b.table, table)
    good = to.Kp.clone(), to.Vp.clone()
    for bad_src in (True, False):
        to.Kp.fill_(5.0)
        to.Vp.fill_(6.0)
        t, to_t = b.table.clone(), table.clone()
        (t if bad_src else to_t)[0, 1] = 12345
        call(t, to_t)
        assert cxa.cxa_device_status(1) == cxa.CXA_EPAGE
        gone = [int(table[0, i]) for i in ((2, 3) if bad_src else (1,))]
        kept = [p for p in range(to.num_pages) if p not in gone]
        assert torch.equal(to.Kp[:, kept], good[0][:, kept]) and torch.equal(to.Vp[:, kept], good[1][:, kept])
        assert bool((to.Kp[1, gone] == 5.0).all()) and bool((to.Vp[1, gone] == 6.0).all())


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("pool", ["bf16", "f32"])
def test_both_forms_give_the_same_attention(pool):
    """A prompt, then single tokens, of two sequences in a decoder with latent attention: the new rows
    are appended; the prompt goes the expanded way, the tokens the absorbed one, and each is compared with the
    attention of all heads in 64 bits over the rows as they are stored."""
    H, dh, latent, rope, page = 6, 64, 256, 32, 16
    cache = cxa.LatentCache(40, page, 1, latent, rope, pool)
    to = cxa.PagedCache(20, 64, 1, H, dh, pool)
    dt, scale = DT[pool], 1.0 / math.sqrt(dh)
    WK, WV = (randn(latent, H * w, seed=w, dtype=dt, scale=latent ** -0.5).cuda() for w in (dh - rope, dh))
    rot = cxa.Rotary(rope)
    table = torch.arange(40, dtype=torch.int32).view(2, 20).cuda()
    to_table = torch.arange(20, dtype=torch.int32).view(2, 10).cuda()
    lens = [0, 0]
    for step, n in enumerate(([70, 33], [1, 1], [1, 1])):
        lens = [a + b for a, b in zip(lens, n)]
        N = sum(n)
        q_start = torch.tensor([0, n[0], N], dtype=torch.int32).cuda()
        kv_len = torch.tensor(lens, dtype=torch.int32).cuda()
        pos = torch.cat([torch.arange(k - m, k) for k, m in zip(lens, n)]).int().cuda()
        batch = dict(q_start=q_start, kv_len=kv_len, page_table=table)
        c, kr = (randn(N, w, seed=50 * step + w, dtype=dt).cuda() for w in (latent, rope))
        q = randn(N, H, dh, seed=step, dtype=dt).cuda()
        q, _ = cxa.qk_norm_rope(q, None, pos, rotary=rot)
        cache.check(q_start, kv_len, table, N)
        cache.append(0, c, kr, **batch, rotary=rot, norm_eps=1e-6)
        wk = WK.double().view(latent, H, dh - rope)
        wv = WV.double().view(latent, H, dh)
        if step == 0:
            cache.expand(0, WK, WV, kv_len, table, to, 0, to_table)
            got = to.attend(0, q, q_start, kv_len, to_table, max_new=70).double()
        else:
            qa = torch.cat([torch.einsum("nhd,chd->nhc", q[..., rope:].double(), wk), q[..., :rope].double()], -1).to(dt)
            got = cache.attend(0, qa, **batch, max_new=1, scale=scale).double()
            got = torch.einsum("nhc,chd->nhd", got, wv)
        for s in range(2):
            rows = cache.Cp[0][table[s].long()].reshape(-1, latent + rope)[:lens[s]].double()
            k = torch.cat([rows[:, None, latent:].expand(-1, H, -1), torch.einsum("tc,chd->thd", rows[:, :latent], wk)], -1)
            v = torch.einsum("tc,chd->thd", rows[:, :latent], wv)
            for i in range(n[s]):
                at = int(q_start[s]) + i
                see = lens[s] - n[s] + i + 1
                p = torch.softmax(torch.einsum("hd,thd->ht", q[at].double(), k[:see]) * scale, -1)
                want = torch.einsum("ht,thd->hd", p, v[:see])
                # roundings of K, V or of the absorbed query and the result (u each, through weights
                # of up to big), of the weights (bf16: 2^-8) and of what is returned
                u = U[dt]
                big = float((torch.einsum("hd,thd->ht", q[at].double().abs(), k[:see].abs()) * scale).max())
                big = max(big, float((torch.einsum("hd,chd,tc->ht", q[at, :, rope:].double().abs(), wk.abs(),
                                                   rows[:see, :latent].abs()) * scale).max()))
                A = torch.einsum("ht,thd->hd", p, torch.einsum("tc,chd->thd", rows[:see, :latent].abs(), wv.abs()))
                e = (4 * u + 2 * u * big if pool == "bf16" else 2.0 ** -18 * (1 + big))
                assert float(((got[at] - want).abs() - e * A).max()) <= 0


@pytest.mark.parametrize("pool", ["bf16", "f32"])
def test_threads_share_a_stream_and_its_workspace(pool):
    """Attention is two kernels that hand partial states to one another in the workspace: calls that threads enqueue
    at once on one stream are each enqueued whole."""
    bs = [Batch([1] * 4, [3000, 20, 9000, 77], 64, 20, 512, 64, pool, seed=1).fill(),
          Batch([3, 1], [5000, 700], 64, 8, 128, 16, pool, seed=2).fill(), Batch([40], [900], 32, 6, 256, 0, pool, seed=3).fill()]
    code = {"bf16": cxa.CXA_BF16, "f32": cxa.CXA_F32}[pool]
    need = max(cxa.cxa_latent_attention_workspace_bytes(b.H, b.latent, b.max_new, code) for b in bs)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    want = [b.attend() for b in bs]
    outs = [[torch.zeros_like(w) for _ in range(40)] for w in want]
    qs = [b.q.cuda() for b in bs]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()

    def calls(i):
        for out in outs[i]:
            bs[i].cache.attend(0, qs[i], **bs[i].d, max_new=bs[i].max_new, scale=bs[i].scale, out=out, workspace=ws,
                               stream=stream)

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(3)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, x) for x in o)


@pytest.mark.parametrize("pool", ["bf16", "f32"])
def test_expand_reports_positions_behind_the_row_of_the_table(pool):
    """kv_len past what page_table's row holds: the positions that it does hold are written, the others reported."""
    kw = dict(kv=[100, 50], start=None, H=4, dh=64, latent=128, rope=16, page=32, to_page=16)
    b, to, table, WK, WV = expand_case(pool=pool, **kw)
    wide = torch.cat([table, torch.full((2, 40), to.num_pages - 1, dtype=torch.int32)], 1)     # (no position writes there)

    def call(kv, start=None, t=b.table):
        ints = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32).cuda()
        b.cache.expand(0, WK.cuda(), WV.cuda(), ints(kv), t.cuda(), to, 1, wide.cuda(), start=ints(start))
        return cxa.cxa_device_status(1)

    assert b.table.shape[1] * 32 == 160
    assert call([100, 50]) == cxa.CXA_OK
    good = to.Kp.clone(), to.Vp.clone()
    narrow = b.table[:, :3].contiguous()              # 96 positions
    to.Kp.fill_(5.0)
    to.Vp.fill_(6.0)
    assert call([100, 50], t=narrow) == cxa.CXA_EPAGE
    last = int(table[0, 6])                           # of positions 96 to 99
    kept = [p for p in range(to.num_pages) if p != last]
    assert torch.equal(to.Kp[:, kept], good[0][:, kept]) and torch.equal(to.Vp[:, kept], good[1][:, kept])
    assert bool((to.Kp[1, last] == 5.0).all()) and bool((to.Vp[1, last] == 6.0).all())
    for kv, start, status in (([97, 0], [97, 0], cxa.CXA_OK), ([97, 0], [96, 0], cxa.CXA_EPAGE),
                              ([0, 2 ** 31 - 1], [0, 97], cxa.CXA_EPAGE), ([96, 96], [-5, 500], cxa.CXA_OK)):
        assert call(kv, start, narrow) == status


@pytest.mark.parametrize("H, latent, rope", [(8, 256, 0), (20, 512, 64), (64, 512, 64), (128, 128, 16), (40, 384, 32)])
def test_bf16_weights_are_two_values(H, latent, rope):
    """As in `close`, but for the softmax weights' rounding: to two bf16 values, 2^-8 of 2^-8, whose products add
    2^-23 for each 16 keys of either. (To one, a sum of few values of either sign is off by up to 2^-8 of their magnitudes.)"""
    b = Batch([1, 1, 3, 1], [5, 30, 70, 2000], 64, H, latent, rope, "bf16", seed=H).fill(float("nan"))
    got, (out, A, big) = b.attend().cpu(), b.reference()
    e = 2.0 ** -16 + 2.0 ** -21 + (2 * 2000 / 16 + 64) * 2.0 ** -23 + 2 * (b.width / 16 + 1) * 2.0 ** -23 * big
    over = (got.double() - out).abs() - U[got.dtype] * out.abs() - e * A
    assert float(over.max()) <= 0


@pytest.mark.parametrize("pool", ["bf16", "f32"])
@pytest.mark.parametrize("H, n", [(16, 1), (8, 4), (64, 1), (20, 3)])
def test_every_key_of_a_long_context_counts(pool, H, n):
    """Items cut between many blocks. Each run of 64 keys has a channel of its own (or one of two), and weights rise
    along the context, so that a part that is lost, taken twice or misweighted moves a channel by a large share of it."""
    kv, latent, rope = 40000, 512, 64
    b = Batch([n], [kv], 128, H, latent, rope, pool, seed=H)
    at = torch.arange(kv)
    C = b.C[0].float() * 0.01
    C[at, (at // 64) % latent] += 8.0
    C[:, latent] = torch.linspace(0, 8, kv)
    q = b.q.float() * 0.05
    q[:, :, latent] = 8.0
    b.C[0], b.q = C.to(DT[pool]), q.to(DT[pool])
    b.fill(float("inf"))
    got, (out, A, big) = b.attend().cpu(), b.reference()
    if pool == "f32":
        e = 2.0 ** -21 + (kv + 64) * 2.0 ** -24 + 2 * 23 * 2.0 ** -24 * big
    else:
        e = 2.0 ** -16 + 2.0 ** -21 + (2 * kv / 16 + 64) * 2.0 ** -23 + 2 * (b.width / 16 + 1) * 2.0 ** -23 * big
    bound = U[got.dtype] * out.abs() + e * A
    assert float(((got.double() - out).abs() - bound).max()) <= 0
    # what the bound would see: the result without some run of 64 keys, or with a run twice
    for run in (0, 77, 300, 624):
        keys = b.C[0][64 * run:64 * run + 64].double()
        logits = b.q.double() @ b.C[0].double().T * b.scale
        p = torch.softmax(logits[0], -1)[:, 64 * run:64 * run + 64]          # the first token's
        for times in (-1, 1):
            wrong = (out[0] + times * p @ keys[:, :latent]) / (1 + times * p.sum(-1, keepdim=True))
            assert bool(((wrong - out[0]).abs() > 4 * bound[0]).any(-1).all())


@pytest.mark.parametrize("pool", ["bf16", "f32"])
def test_one_workspace_for_calls_of_both_caches(pool):
    """One buffer, cleared once, for latent attention, paged attention and gathered weights in turn."""
    b = Batch([1, 4], [9000, 700], 64, 20, 512, 64, pool).fill()
    kv = cxa.PagedCache(200, 64, 1, 2, 64, pool)
    for i, x in enumerate((kv.Kp, kv.Vp)):
        x.copy_(randn(*x.shape, seed=i))
    d = dict(b.d, page_table=torch.arange(180, dtype=torch.int32, device="cuda").view(1, 180).repeat(2, 1))
    d["page_table"][1] += 20
    d["kv_len"] = torch.tensor([180 * 64, 300], dtype=torch.int32, device="cuda")
    d["page_table"][1, 5:] = -1
    d["page_table"][1, :5] = torch.arange(190, 195, dtype=torch.int32)
    q = randn(5, 8, 64, seed=3, dtype=DT[pool]).cuda()
    W = kv.new_weights()
    want = kv.attend(0, q, **d, max_new=4), kv.accumulate(0, q, **d, max_new=4, weights=W, decay=0.0).clone(), b.attend()
    code = {"bf16": cxa.CXA_BF16, "f32": cxa.CXA_F32}[pool]
    ws = torch.zeros(max(cxa.cxa_latent_attention_workspace_bytes(20, 512, 4, code),
                         cxa.cxa_paged_attention_workspace_bytes(8, 2, 64, 4),
                         cxa.cxa_paged_weights_workspace_bytes(kv.handle, 2, 5, 4, 180, 8)), dtype=torch.uint8, device="cuda")
    for _ in range(3):
        assert torch.equal(b.attend(workspace=ws), want[2])
        assert torch.equal(kv.attend(0, q, **d, max_new=4, workspace=ws), want[0])
        assert torch.equal(b.attend(workspace=ws), want[2])
        W.fill_(float("nan"))
        kv.accumulate(0, q, **d, max_new=4, weights=W, decay=0.0, workspace=ws)
        assert torch.equal(W.nan_to_num(0), want[1])
    assert not bool(ws[:cxa.CXA_PAGED_COUNTER_BYTES].any())
