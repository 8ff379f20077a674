"""The attention weight that keys gather, and the eviction by it, on the GPU against plain fp64 forms
written out here.

Tolerance of gathered weights, per element: |got - ref| <= 2^-24 |ref| + e S, S the sum of the
magnitudes added (the old number among them). e counts 2^-20 for ex2 and log2 of both passes, one step of 2^-24
for each of the rows added, and twice (numerator and reference) the steps of a sum of dh products, a
reference of up to that size and their difference: 2 (dh + 16) 2^-24 times scale * max sum |q||k|. A row's
weight below the smallest normal number, 2^-126, becomes 0 (ex2 flushes it): 2^-126 more for each row.
Evictions copy: they are compared bit for bit.
"""
import math
import threading

import pytest
import torch

from encoder_decoder_speech_gb300 import cxa

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


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
    """Sequences with n new tokens of kv keys each, in shuffled pages, with weights gathered so far."""

    def __init__(self, n, kv, page=16, Hq=4, Hkv=4, dh=64, pool="bf16", seed=0, L=1, layer=0, spare=3, pad=0):
        self.n, self.kv, self.page, self.Hq, self.Hkv, self.dh, self.layer = n, kv, page, Hq, Hkv, dh, layer
        self.B = len(n)
        need = [-(-max(k, 0) // page) for k in kv]
        P = sum(need) + spare
        self.cache = cxa.PagedCache(P, page, L, Hkv, dh, pool)
        self.cache.Kp.fill_(float("nan"))
        g = torch.Generator().manual_seed(seed + 77)
        perm = torch.randperm(P, generator=g).tolist()
        self.table = torch.full((self.B, max(need + [0]) + 1), -1, dtype=torch.int32)
        for b in range(self.B):
            for i in range(need[b]):
                self.table[b, i] = perm.pop()
        self.starts = [sum(n[:b]) for b in range(self.B + 1)]
        self.N = self.starts[-1] + pad
        self.q = randn(self.N, Hq, dh, seed=seed + 1, dtype=DT[pool])
        self.K = [randn(max(k, 0), Hkv, dh, seed=seed + 100 + b, dtype=DT[pool]) for b, k in enumerate(kv)]
        self.W = self.cache.new_weights()
        self.W.copy_(torch.rand(self.W.shape, generator=g))
        self.d = dict(q_start=torch.tensor(self.starts, dtype=torch.int32).cuda(),
                      kv_len=torch.tensor(kv, dtype=torch.int32).cuda(), page_table=self.table.cuda())
        self.max_new = max(n + [1])

    def places(self, b):
        t = torch.arange(max(self.kv[b], 0))
        return self.table[b][t // self.page].long(), t % self.page

    def fill(self):
        Kp = self.cache.Kp.cpu()
        for b in range(self.B):
            p, s = self.places(b)
            Kp[self.layer][p, :, s] = self.K[b]
        self.cache.Kp.copy_(Kp)
        return self

    def accumulate(self, **kw):
        kw.setdefault("max_new", self.max_new)
        return self.cache.accumulate(self.layer, kw.pop("q", self.q).cuda(), **self.d, weights=self.W, **kw)

    def close(self, before, got, decay=1.0, scale=None):
        scale = scale or 1 / math.sqrt(self.dh)
        G = self.Hq // self.Hkv
        want, mag = before.double().cpu(), torch.zeros(before.shape, dtype=torch.float64)
        big = 0.0
        for b in range(self.B):
            n, kv = self.n[b], self.kv[b]
            if n == 0 or kv <= 0:
                continue
            q = self.q[self.starts[b]:self.starts[b + 1]].cuda().double()
            K = self.K[b].cuda().double()
            seen = torch.arange(kv, device="cuda")[None] <= (kv - n + torch.arange(n, device="cuda"))[:, None]
            add = torch.zeros(kv, self.Hkv, dtype=torch.float64, device="cuda")
            for h in range(self.Hq):
                s = q[:, h] @ K[:, h // G].T * scale
                big = max(big, float((q[:, h].abs() @ K[:, h // G].abs().T * scale).nan_to_num(0, 0, 0).max()))
                s = s.masked_fill(~seen, -math.inf)
                p = torch.softmax(s, -1).masked_fill(~seen.any(-1, keepdim=True), 0.0)
                add[:, h // G] += torch.where(seen, p, 0.0).sum(0)
            p, at = self.places(b)
            old = want[self.layer][p, :, at] * decay
            old[max(0, kv - n):] = 0
            want[self.layer][p, :, at] = old + add.cpu()
            mag[self.layer][p, :, at] = old + add.cpu()
        got = got.cpu().double()
        assert torch.equal(got[mag == 0].nan_to_num(-1), want[mag == 0].nan_to_num(-1))
        e = 2.0 ** -20 + max(self.n) * G * 2.0 ** -24 + 2 * (self.dh + 16) * 2.0 ** -24 * big
        over = (got - want).abs() - 2.0 ** -24 * want.abs() - e * mag - max(self.n) * G * 2.0 ** -126
        fin = want.isfinite()
        assert bool((got.isfinite() == fin).all())
        assert float(over[fin].max()) <= 0


CASES = [
    dict(n=[1], kv=[1]),
    dict(n=[1], kv=[448], Hq=8, Hkv=8),
    dict(n=[1, 1, 1, 1], kv=[63, 64, 65, 700], Hq=32, Hkv=8, dh=128, page=64),
    dict(n=[1] * 9, kv=[5, 1000, 130, 17, 2049, 64, 700, 128, 3], Hq=8, Hkv=1, page=32),
    dict(n=[5, 0, 1, 3], kv=[900, 40, 33, 3], Hq=4, Hkv=2, dh=128, page=128),
    dict(n=[130], kv=[130], Hq=6, Hkv=6, page=256),
    dict(n=[300, 1, 70], kv=[1000, 700, 70], Hq=10, Hkv=2, page=64),
    dict(n=[17], kv=[5000], Hq=20, Hkv=20, page=128),
    dict(n=[257, 64], kv=[3000, 64], Hq=5, Hkv=1, dh=128, page=16),
    dict(n=[2, 1], kv=[129, 256], Hq=40, Hkv=1, page=16),
    dict(n=[3], kv=[200], Hq=200, Hkv=1, page=64),
]


@pytest.mark.parametrize("pool", ["bf16", "f32"])
@pytest.mark.parametrize("decay", [1.0, 0.75, 0.0])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_accumulate(i, decay, pool):
    b = Batch(pool=pool, seed=10 * i, **CASES[i]).fill()
    before = b.W.clone()
    if decay == 0.0:
        b.W.fill_(float("nan"))
        before = torch.where(torch.isnan(b.W), 0.0, 0.0)
        for s in range(b.B):
            if b.n[s] == 0:
                continue
            p, at = b.places(s)
            before[0][p, :, at] = 1.0
        rest = before == 0
        before = torch.where(rest, float("nan"), torch.zeros_like(before))
    assert b.accumulate(decay=decay) is b.W
    b.close(before, b.W, decay=decay)


@pytest.mark.parametrize("pool", ["bf16", "f32"])
@pytest.mark.parametrize("n", [1, 4, 40])
def test_accumulate_over_a_long_context(n, pool):
    b = Batch([n], [40000], 128, 8, 2, 64, pool, seed=n).fill()
    before = b.W.clone()
    b.accumulate()
    b.close(before, b.W)


@pytest.mark.parametrize("pool", ["bf16", "f32"])
@pytest.mark.parametrize("n", [2, 60])
def test_scores_far_apart(n, pool):
    b = Batch([n], [600], 64, 4, 2, 64, pool, seed=3)
    b.K[0].mul_(torch.linspace(0.1, 20, 600)[:, None, None].to(b.K[0].dtype))
    b.fill()
    before = b.W.clone()
    b.accumulate(scale=0.5)
    b.close(before, b.W, scale=0.5)


@pytest.mark.parametrize("pool", ["bf16", "f32"])
def test_padding_rows_max_new_and_other_layers(pool):
    b = Batch([1, 30, 2], [100, 300, 2], 16, 8, 4, 64, pool, L=3, layer=1, pad=5).fill()
    before = b.W.clone()
    b.accumulate(max_new=500)
    b.close(before, b.W)
    assert torch.equal(before[0], b.W[0]) and torch.equal(before[2], b.W[2])


@pytest.mark.parametrize("pool", ["bf16", "f32"])
@pytest.mark.parametrize("n", [4, 40])
def test_rows_that_see_nothing_add_nothing(n, pool):
    b = Batch([n, 1], [2, 0], 16, 4, 4, 64, pool).fill()
    before = b.W.clone()
    b.accumulate()
    b.close(before, b.W)


@pytest.mark.parametrize("pool", ["bf16", "f32"])
@pytest.mark.parametrize("n", [3, 40])
def test_a_bad_page_is_reported_and_left_out(n, pool):
    b = Batch([n, 2], [200, 90], 32, 4, 2, 64, pool).fill()
    before = b.W.clone()
    gone = int(b.table[0, 2])
    b.table[0, 2] = 1000
    b.d["page_table"] = b.table.cuda()
    b.accumulate()
    assert cxa.cxa_device_status(1) == cxa.CXA_EPAGE
    assert torch.equal(before[0, gone], b.W[0, gone])
    b.K[0] = torch.cat([b.K[0][:64], b.K[0][96:]])
    b.table[0, 2:-1] = b.table[0, 3:].clone()
    b.kv[0] = 168                        # the same keys without the page's
    b.close(before, b.W)


@pytest.mark.parametrize("n", [3, 70])
@pytest.mark.parametrize("pool", ["bf16", "f32"])
def test_infinities_reach_only_who_sees_them(n, pool):
    b = Batch([n], [200], 64, 4, 2, 64, pool).fill()
    b.K[0][199, 1, 5] = float("nan")      # seen by the last token alone, in the second K/V head
    b.fill()
    before = b.W.clone()
    b.accumulate()
    p, at = b.places(0)
    got = b.W.cpu()[0][p, :, at]
    assert bool(got[:, 0].isfinite().all()) and bool(got[:, 1].isnan().all())
    first = Batch([n - 1], [199], 64, 4, 2, 64, pool)        # the same without the last token
    first.q, first.K, first.table = b.q[:n - 1], [b.K[0][:199]], b.table
    first.d["page_table"] = b.table.cuda()
    first.fill()
    first.W.copy_(before)
    first.accumulate()
    first.close(before, first.W)


@pytest.mark.parametrize("pool", ["bf16", "f32"])
def test_results_do_not_change_and_strides(pool):
    b = Batch([1] * 5 + [90], [3000, 10, 900, 4000, 77, 2500], 64, 8, 2, 128, pool).fill()
    before = b.W.clone()
    first = b.accumulate().clone()
    wide = torch.zeros(b.N, 8 * 128 + 24, dtype=DT[pool], device="cuda")
    q = wide[:, 16:16 + 1024].unflatten(1, (8, 128))
    q.copy_(b.q)
    for _ in range(4):
        b.W.copy_(before)
        b.cache.accumulate(0, q, **b.d, max_new=b.max_new, weights=b.W)
        assert torch.equal(b.W, first)


@pytest.mark.parametrize("pool", ["bf16", "f32"])
def test_graphs_and_streams_at_once(pool):
    bs = [Batch([1, 30 * i + 1], [5000 + 100 * i, 300], 64, 8, 2, 64, pool, seed=i).fill() for i in range(3)]
    before = [b.W.clone() for b in bs]
    want = [b.accumulate().clone() for b in bs]
    graphs = []
    for b in bs:
        q = b.q.cuda()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b.cache.accumulate(0, q, **b.d, max_new=b.max_new, weights=b.W)
        graphs.append((graph, q))
    other = [w.clone() for w in before]
    for b, w in zip(bs, before):
        b.W.copy_(w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    for b, o, (graph, q), s in zip(bs, other, graphs, streams):
        with torch.cuda.stream(s):
            graph.replay()
            b.cache.accumulate(0, q, **b.d, max_new=b.max_new, weights=o)
    torch.cuda.synchronize()
    for w, b, o in zip(want, bs, other):
        assert torch.equal(w, b.W) and torch.equal(w, o)


# ------------------------------------------------------------------ eviction
def plain_evict(case, weights):
    """kept, by the definition: a list of old positions for every (layer, sequence, head)."""
    kept = {}
    for l in range(case["nl"]):
        for b, kv in enumerate(case["kv"]):
            for h in range(case["Hkv"]):
                w = weights(case["l0"] + l, b, h)
                rank = []
                for t in range(kv):
                    stays = t < case["first"] or t >= kv - case["recent"]
                    x = float(w[t]) + 0.0
                    rank.append((0 if stays else 2 if x != x else 1, 0.0 if stays or x != x else -x, t))
                kept[l, b, h] = sorted(t for _, _, t in sorted(rank)[:min(kv, case["keep"])])
    return kept


EVICT = [
    dict(kv=[1], keep=1, first=0, recent=0),
    dict(kv=[40, 0, 17, 16], keep=16, first=0, recent=0),
    dict(kv=[300, 448, 100], keep=112, first=4, recent=32, L=3, Hkv=8),
    dict(kv=[700], keep=40, first=20, recent=20, Hkv=2, dh=128, page=64),
    dict(kv=[3000, 50], keep=1000, first=1, recent=0, page=128, L=2, l0=1, nl=1),
    dict(kv=[33, 31], keep=32, first=0, recent=7, page=32, dh=128),
    dict(kv=[5000], keep=4999, first=0, recent=1, page=256, Hkv=1),
    dict(kv=[2100, 900], keep=1, first=0, recent=1, page=16),
    dict(kv=[70000], keep=300, first=2, recent=100, page=256, Hkv=2),
]


@pytest.mark.parametrize("kind", ["sums", "ties", "odd"])
@pytest.mark.parametrize("pool", ["bf16", "f32"])
@pytest.mark.parametrize("i", range(len(EVICT)))
def test_evict(i, pool, kind):
    case = dict(dict(L=1, l0=0, Hkv=3, dh=64, page=16), **EVICT[i])
    case.setdefault("nl", case["L"] - case["l0"])
    kv, keep, page, Hkv = case["kv"], case["keep"], case["page"], case["Hkv"]
    need, need_out = [-(-k // page) for k in kv], [-(-min(k, keep) // page) for k in kv]
    P = sum(need) + sum(need_out) + 2
    cache = cxa.PagedCache(P, page, case["L"], Hkv, case["dh"], pool)
    g = torch.Generator().manual_seed(i)
    perm = torch.randperm(P, generator=g).tolist()
    table = torch.full((len(kv), max(need + [1])), -1, dtype=torch.int32)
    out_table = torch.full((len(kv), -(-min(keep, max(need + [1]) * page) // page)), -1, dtype=torch.int32)
    for b in range(len(kv)):
        for t, m in ((table, need[b]), (out_table, need_out[b])):
            for j in range(m):
                t[b, j] = perm.pop()
    for pool_t in (cache.Kp, cache.Vp):
        pool_t.copy_(torch.randn(pool_t.shape, generator=g))
    W = cache.new_weights()
    w = torch.rand(W.shape, generator=g) ** 6
    if kind == "ties":
        w = (w * 4).floor() / 4
    if kind == "odd":
        r = torch.rand(W.shape, generator=g)
        w = torch.where(r < 0.05, float("nan"), torch.where(r < 0.1, -0.0, torch.where(r < 0.12, math.inf, torch.where(
            r < 0.14, -math.inf, torch.where(r < 0.3, -w, torch.where(r < 0.4, 0.0, torch.where(r < 0.45, 1e-41, w)))))))
    W.copy_(w)
    before = [x.cpu().clone() for x in (cache.Kp, cache.Vp, W)]
    kv_len = torch.tensor(kv, dtype=torch.int32).cuda()
    cache.check_evict(keep, kv_len, table, out_table)
    kept, out_len = cache.evict(W, keep, kv_len, table.cuda(), out_table.cuda(), first=case["first"],
                                recent=case["recent"], l0=case["l0"], nl=case["nl"])
    assert out_len.tolist() == [min(k, keep) for k in kv]

    def weights(l, b, h):
        t = torch.arange(kv[b])
        return w[l][table[b][t // page].long(), h, t % page]
    want = [x.clone() for x in before]
    want_kept = torch.full((case["nl"], len(kv), Hkv, keep), -1, dtype=torch.int32)
    for (l, b, h), at in plain_evict(case, weights).items():
        want_kept[l, b, h, :len(at)] = torch.tensor(at, dtype=torch.int32)
        at, to = torch.tensor(at, dtype=torch.long), torch.arange(len(at))
        for x, y in zip(want, before):
            x[case["l0"] + l][out_table[b][to // page].long(), h, to % page] = \
                y[case["l0"] + l][table[b][at // page].long(), h, at % page]
    assert torch.equal(kept.cpu(), want_kept)
    for got, x in zip((cache.Kp, cache.Vp, W), want):
        got = got.cpu()
        assert torch.equal(got.view(torch.int16 if got.dtype == torch.bfloat16 else torch.int32),
                           x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32))


def test_evict_of_shared_pages_and_bad_ones():
    """Two sequences read the same pages; a page outside the pool is left out and reported."""
    cache = cxa.PagedCache(12, 16, 1, 2, 64, "bf16")
    cache.Kp.copy_(torch.randn(cache.Kp.shape))
    W = cache.new_weights()
    W.copy_(torch.rand(W.shape))
    kv_len = torch.tensor([48, 48], dtype=torch.int32).cuda()
    table = torch.tensor([[0, 1, 2], [0, 1, 2]], dtype=torch.int32)
    out = torch.tensor([[4, 5], [6, 7]], dtype=torch.int32)
    cache.check_evict(20, kv_len, table, out)
    kept, _ = cache.evict(W, 20, kv_len, table.cuda(), out.cuda())
    assert torch.equal(kept[:, 0], kept[:, 1])
    assert torch.equal(cache.Kp[0, 4], cache.Kp[0, 6]) and torch.equal(W[0, 5, :, :4], W[0, 7, :, :4])
    table[1, 1], out[0, 1] = 99, -1
    rest = cache.Kp[0, [5, 8, 9, 10, 11]].clone()
    cache.evict(W, 20, kv_len, table.cuda(), out.cuda())
    assert cxa.cxa_device_status(1) == cxa.CXA_EPAGE
    assert torch.equal(rest, cache.Kp[0, [5, 8, 9, 10, 11]])


def test_evict_in_a_graph_and_on_streams():
    kv_len = torch.tensor([500, 300], dtype=torch.int32).cuda()
    table = torch.arange(64, dtype=torch.int32).view(2, 32).cuda()
    out = torch.arange(64, 78, dtype=torch.int32).view(2, 7).cuda()
    caches, want = [], []
    for i in range(3):
        c = cxa.PagedCache(78, 16, 2, 4, 64, "bf16")
        g = torch.Generator().manual_seed(i)
        c.Kp.copy_(torch.randn(c.Kp.shape, generator=g))
        W = c.new_weights()
        W.copy_(torch.rand(W.shape, generator=g))
        c.Kp[:, 64:] = 0
        W[:, 64:] = 0
        c.evict(W, 100, kv_len, table, out, first=2, recent=9)
        want.append((c.Kp.clone(), W.clone()))
        c.Kp[:, 64:] = 0
        W[:, 64:] = 0
        caches.append((c, W))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        caches[0][0].evict(caches[0][1], 100, kv_len, table, out, first=2, recent=9)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in caches]
    for i, ((c, W), s) in enumerate(zip(caches, streams)):
        with torch.cuda.stream(s):
            if i == 0:
                graph.replay()
            else:
                c.evict(W, 100, kv_len, table, out, first=2, recent=9)
    torch.cuda.synchronize()
    for (c, W), (K, V) in zip(caches, want):
        assert torch.equal(c.Kp, K) and torch.equal(W, V)


def test_python_refusals():
    b = Batch([1], [10]).fill()
    with pytest.raises(ValueError):
        b.cache.accumulate(0, b.q.cuda(), **b.d, max_new=1, weights=b.W[..., :8])
    with pytest.raises(cxa.CxaError):
        b.cache.accumulate(0, b.q.cuda().float(), **b.d, max_new=1, weights=b.W)
    with pytest.raises(cxa.CxaError):
        b.cache.accumulate(0, b.q.cuda(), **b.d, max_new=1, weights=b.W, decay=-1.0)
    out = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    ev = lambda **kw: b.cache.evict(**dict(dict(weights=b.W, keep=8, kv_len=b.d["kv_len"], page_table=b.d["page_table"],
                                                out_table=out), **kw))
    with pytest.raises(ValueError):
        ev(keep=0)
    with pytest.raises(ValueError):
        ev(weights=b.W.double())
    with pytest.raises(ValueError):
        ev(out_table=out.long())
    with pytest.raises(cxa.CxaError):
        ev(first=9)
    with pytest.raises(cxa.CxaError):
        ev(out_len=b.d["kv_len"])


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("pool", ["bf16", "f32"])
def test_a_decoder_that_evicts(pool):
    """A prompt and tokens are appended (keys rotated by their own positions, which go on counting over
    evictions), attend, and add to the weights; twice the cache is cut down into other pages, which become the
    sequences' own. The attention is compared with the plain one over the rows that were kept."""
    Hq, Hkv, dh, page, keep = 8, 4, 64, 16, 48
    cache = cxa.PagedCache(64, page, 1, Hkv, dh, pool)
    W = cache.new_weights()
    dt, rot = DT[pool], cxa.Rotary(dh)
    free = list(range(64))
    tables = [[], []]
    lens, pos = [0, 0], [0, 0]
    rows = [[torch.empty(0, Hkv, dh, dtype=torch.float64, device="cuda") for _ in range(2)] for _ in range(2)]
    heads = torch.arange(Hkv, device="cuda")

    def as_table(width=8):
        t = torch.full((2, width), -1, dtype=torch.int32)
        for b in range(2):
            t[b, :len(tables[b])] = torch.tensor(tables[b], dtype=torch.int32)
        return t.cuda()
    for step, n in enumerate(([90, 33], [1, 1], None, [1, 1], [4, 30], None, [1, 1])):
        if n is None:
            table = as_table()
            old = [list(t) for t in tables]
            for b in range(2):
                tables[b] = [free.pop() for _ in range(-(-min(lens[b], keep) // page))]
            out, kv_len = as_table(), torch.tensor(lens, dtype=torch.int32).cuda()
            cache.check_evict(keep, kv_len, table, out)
            kept, out_len = cache.evict(W, keep, kv_len, table, out, first=2, recent=10)
            for t in old:
                free.extend(t)
            lens = out_len.tolist()
            for b in range(2):
                at = kept[0, b, :, :lens[b]].long().T
                assert bool((at[:2] == torch.arange(2, device="cuda")[:, None]).all())
                rows[b] = [x[at, heads] for x in rows[b]]
            continue
        N = sum(n)
        for b in range(2):
            lens[b] += n[b]
            pos[b] += n[b]
            while len(tables[b]) * page < lens[b]:
                tables[b].append(free.pop())
        p = torch.cat([torch.arange(x - m, x) for x, m in zip(pos, n)]).int().cuda()
        q = randn(N, Hq, dh, seed=step, dtype=dt).cuda()
        k, v = (randn(N, Hkv, dh, seed=100 + 2 * step + i, dtype=dt).cuda() for i in range(2))
        q, k = cxa.qk_norm_rope(q, k, p, rotary=rot)
        batch = dict(q_start=torch.tensor([0, n[0], N], dtype=torch.int32).cuda(),
                     kv_len=torch.tensor(lens, dtype=torch.int32).cuda(), page_table=as_table())
        cache.append(0, k, v, **batch)
        got = cache.attend(0, q, **batch, max_new=max(n)).double()
        cache.accumulate(0, q, **batch, max_new=max(n), weights=W)
        for b in range(2):
            part = slice(0, n[0]) if b == 0 else slice(n[0], N)
            rows[b] = [torch.cat([x, y[part].double()]) for x, y in zip(rows[b], (k, v))]
            K, V = (x.repeat_interleave(Hq // Hkv, 1) for x in rows[b])
            s = torch.einsum("nhd,thd->hnt", q[part].double(), K) / math.sqrt(dh)
            see = torch.arange(lens[b], device="cuda")[None] <= torch.arange(lens[b] - n[b], lens[b], device="cuda")[:, None]
            w = torch.softmax(s.masked_fill(~see, -math.inf), -1)
            want = torch.einsum("hnt,thd->nhd", w, V)
            A = torch.einsum("hnt,thd->nhd", w, V.abs())
            e = 2.0 ** -7 if pool == "bf16" else 2.0 ** -16
            assert float(((got[part] - want).abs() - e * (A + want.abs())).max()) <= 0
            # the new tokens' own weights: their entries have started at zero
            own = w[:, :, lens[b] - n[b]:].sum(1).view(Hkv, -1, n[b]).sum(1)
            at = torch.arange(lens[b] - n[b], lens[b], device="cuda")
            gathered = W[0][as_table()[b][at // page].long(), :, at % page].T.double()
            assert float((gathered - own).abs().max()) <= 2.0 ** -10 * (Hq // Hkv)


@pytest.mark.parametrize("Hq, Hkv", [(8, 8), (8, 2), (5, 1), (12, 1), (20, 1)])
def test_single_tokens_beside_prompts_over_long_contexts(Hq, Hkv):
    """Enough keys that sequences of few query rows go a way of their own."""
    b = Batch([1, 70, 2, 0, 1, 3, 40], [70000, 300, 66000, 100, 1, 9000, 40], 256, Hq, Hkv, 64, "bf16", seed=Hq).fill()
    b.d["page_table"] = torch.cat([b.table, torch.full((7, 2000), -1, dtype=torch.int32)], 1).cuda()
    before = b.W.clone()
    first = b.accumulate().clone()
    b.close(before, first)
    b.W.copy_(before)
    assert torch.equal(b.accumulate(), first)


@pytest.mark.parametrize("pool", ["bf16", "f32"])
@pytest.mark.parametrize("n", [[1, 1, 0, 2], [3, 40, 1, 2]])
def test_scores_that_have_no_room(n, pool):
    """Rows of the table for more keys than scores are kept of: the keys are read twice instead."""
    b = Batch(n, [700, 90, 30, 2], 64, 4, 2, 128, pool, seed=6).fill()
    b.d["page_table"] = torch.cat([b.table, torch.full((4, 1 << 20), -1, dtype=torch.int32)], 1).cuda()
    before = b.W.clone()
    b.close(before, b.accumulate(decay=0.5), decay=0.5)


def test_evict_more_keys_than_shared_memory_holds():
    kv, keep, page = 400_003, 5000, 256
    need, out_need = -(-kv // page), -(-keep // page)
    cache = cxa.PagedCache(need + out_need, page, 1, 1, 64, "bf16")
    g = torch.Generator().manual_seed(3)
    cache.Kp.copy_(torch.randn(cache.Kp.shape, generator=g))
    cache.Vp.copy_(torch.randn(cache.Vp.shape, generator=g))
    W = cache.new_weights()
    W.copy_(torch.randint(0, 3000, W.shape, generator=g).float())      # (many are equal)
    perm = torch.randperm(need + out_need, generator=g).to(torch.int32)
    table, out = perm[None, :need].contiguous(), perm[None, need:].contiguous()
    t = torch.arange(kv)
    place = (table[0, t // page].long(), t % page)
    w = W.cpu()[0, :, 0][place]
    w[:7], w[-9:] = math.inf, math.inf
    want = torch.sort(torch.sort(w, descending=True, stable=True).indices[:keep]).values
    K = cache.Kp.cpu()[0, :, 0][place][want]
    kept, out_len = cache.evict(W, keep, torch.tensor([kv], dtype=torch.int32).cuda(), table.cuda(), out.cuda(),
                                first=7, recent=9)
    assert torch.equal(kept.cpu()[0, 0, 0].long(), want) and out_len.tolist() == [keep]
    t = torch.arange(keep)
    assert torch.equal(cache.Kp.cpu()[0, :, 0][out[0, t // page].long(), t % page], K)


def test_evict_with_too_few_pages_reports_them():
    """What has a page is copied; the positions without one are left out, and the status says so."""
    b = Batch([0, 0], [100, 20], 16, 2, 2, 64, "bf16", seed=8, spare=6).fill()
    free = [p for p in range(b.cache.num_pages) if p not in b.table.flatten().tolist()][:4]
    out = torch.tensor([[free[0], free[1]], [free[2], free[3]]], dtype=torch.int32).cuda()
    before = b.cache.Kp.clone()
    kept, out_len = b.cache.evict(b.W, 64, b.d["kv_len"], b.d["page_table"], out)
    torch.cuda.synchronize()
    assert cxa.cxa_device_status(1) == cxa.CXA_EPAGE and cxa.cxa_device_status(1) == cxa.CXA_OK
    assert out_len.tolist() == [64, 20]
    for h in range(2):
        t = kept[0, 0, h, :32].cpu().long()
        got = torch.cat([b.cache.Kp[0, free[0], h], b.cache.Kp[0, free[1], h]])
        page, at = b.table[0][t // 16].long(), t % 16
        assert torch.equal(got.cpu(), before.cpu()[0, page, h, at])


@pytest.mark.parametrize("pool", ["bf16", "f32"])
def test_threads_share_a_stream_and_its_workspace(pool):
    """Gathered weights and attention, enqueued by threads at once on one stream with one workspace: each call's
    kernels hand scratch to one another there, so each is enqueued whole."""
    bs = [Batch([1] * 5, [3000, 20, 900, 77, 2500], 64, 8, 2, 64, pool, seed=1).fill(),
          Batch([70, 1, 30], [6000, 900, 70], 64, 8, 2, 64, pool, seed=2).fill()]
    need = []
    for b in bs:
        b.cache.Vp.copy_(randn(*b.cache.Vp.shape, seed=9))
        need += [cxa.cxa_paged_weights_workspace_bytes(b.cache.handle, b.B, b.N, b.max_new, b.table.shape[1], 8),
                 cxa.cxa_paged_attention_workspace_bytes(8, 2, 64, b.max_new)]
    ws = torch.zeros(max(need), dtype=torch.uint8, device="cuda")
    calls = 40
    weights = [[b.W.clone() for _ in range(calls)] for b in bs]
    want = [(b.accumulate(), b.cache.attend(0, b.q.cuda(), **b.d, max_new=b.max_new)) for b in bs]
    got = [(w, [torch.zeros_like(a) for _ in range(calls)]) for w, (_, a) in zip(weights, want)]
    qs = [b.q.cuda() for b in bs]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()

    def accumulate(i):
        for w in got[i][0]:
            bs[i].cache.accumulate(0, qs[i], **bs[i].d, max_new=bs[i].max_new, weights=w, workspace=ws,
                                   stream=stream)

    def attend(i):
        for o in got[i][1]:
            bs[i].cache.attend(0, qs[i], **bs[i].d, max_new=bs[i].max_new, out=o, workspace=ws, stream=stream)

    threads = [threading.Thread(target=f, args=(i,)) for f in (accumulate, attend) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for (w, a), (ws_, as_) in zip(want, got):
        assert all(torch.equal(w, x) for x in ws_) and all(torch.equal(a, x) for x in as_)


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("pool", ["bf16", "f32"])
@pytest.mark.parametrize("n, Hq, at", [(3, 4, 1), (70, 4, 40), (300, 4, 10), (300, 10, 299), (90, 400, 30), (130, 2, 0)])
def test_a_query_that_is_not_finite_leaves_later_keys_alone(n, Hq, at, pool, value):
    """Keys behind the token's own have the weights of a batch whose queries are all finite, bit for bit."""
    b = Batch([n], [200 + n], 64, Hq, 2, 64, pool).fill()
    before = b.W.clone()
    clean = b.accumulate().clone()
    b.W.copy_(before)
    b.q[at, 0, 7] = value                 # of the first K/V head
    b.accumulate()
    p, slot = b.places(0)
    got, want = b.W.cpu()[0][p, :, slot], clean.cpu()[0][p, :, slot]
    assert torch.equal(got[:, 1], want[:, 1])
    assert torch.equal(got[200 + at + 1:, 0], want[200 + at + 1:, 0])
    assert bool(got[:200 + at + 1, 0].isnan().any())
    if value != value:
        assert bool(got[:200 + at + 1, 0].isnan().all())


@pytest.mark.parametrize("pool", ["bf16", "f32"])
def test_a_max_new_that_is_too_small_is_reported(pool):
    """A sequence that has no room is left out and reported; the others' weights are right. Where the call's kernels
    take it all the same, nothing is reported."""
    b = Batch([1, 5, 2], [300, 200, 90], 32, 8, 4, 64, pool).fill()
    before = b.W.clone()
    b.accumulate(max_new=2)
    assert cxa.cxa_device_status(1) == cxa.CXA_EINVAL
    p, at = b.places(1)
    assert torch.equal(b.W[0][p, :, at], before[0][p, :, at])
    b.n[1] = 0
    b.close(before, b.W)
    b.n[1] = 5
    b.W.copy_(before)
    b.accumulate(max_new=9)                       # 18 rows a K/V head: any sequence is taken
    assert cxa.cxa_device_status(1) == cxa.CXA_OK
    b.close(before, b.W)
    b.W.copy_(before)
    many = Batch([1, 60], [300, 200], 32, 8, 4, 64, pool).fill()
    before = many.W.clone()
    many.accumulate(max_new=9)
    assert cxa.cxa_device_status(1) == cxa.CXA_OK
    many.close(before, many.W)


@pytest.mark.parametrize("positions", [5120, 16384, 32768, 1 << 20])
def test_evict_in_wide_tables(positions):
    """Short and long sequences in one call, in tables as wide as the longest that a server allows."""
    kv, keep, L, Hkv, page = [448, 5000, 1, 4096, 0, 4097, 3000], 700, 2, 3, 64
    kv += [k for k in (16384, 16385, 30000) if k <= positions]
    b = Batch([0] * len(kv), kv, page, Hkv, Hkv, 64, "bf16", L=L, spare=len(kv) * 11 + 3)
    free = [p for p in range(b.cache.num_pages) if p not in set(b.table.flatten().tolist())]
    table = torch.full((len(kv), positions // page), -1, dtype=torch.int32)
    w = min(table.shape[1], b.table.shape[1])
    table[:, :w] = b.table[:, :w]
    out = torch.tensor(free[:len(kv) * 11], dtype=torch.int32).view(len(kv), 11)
    b.W.copy_((b.W * 50).floor())                                # (many ties)
    W, before = b.W.cpu(), randn(*b.cache.Kp.shape, seed=3, dtype=torch.bfloat16)
    b.cache.Kp.copy_(before)
    kept, out_len = b.cache.evict(b.W, keep, b.d["kv_len"], table.cuda(), out.cuda(), first=5, recent=100)
    assert out_len.tolist() == [min(k, keep) for k in kv]
    kept, K = kept.cpu().long(), b.cache.Kp.cpu()
    for s, n in enumerate(kv):
        m, t = min(n, keep), torch.arange(n)
        p, at = b.places(s)
        for l in range(L):
            for h in range(Hkv):
                x = W[l][p, h, at]
                x[(t < 5) | (t >= n - 100)] = math.inf
                want = torch.sort(torch.sort(x, descending=True, stable=True).indices[:m]).values
                assert torch.equal(kept[l, s, h, :m], want) and bool((kept[l, s, h, m:] == -1).all())
                j = torch.arange(m)
                assert torch.equal(K[l][out[s][j // page].long(), h, j % page], before[l][p[want], h, at[want]])


@pytest.mark.parametrize("pool", ["bf16", "f32"])
@pytest.mark.parametrize("n", [[1, 1, 0, 2], [3, 40, 1, 2]])
def test_a_wide_table_changes_nothing(n, pool):
    """Whether scores are kept is by the keys. (Whether single tokens beside prompts go a way of their own, which rounds
    differently, is by the table.)"""
    b = Batch(n, [700, 5000, 30, 2], 64, 4, 2, 128, pool, seed=6).fill()
    before = b.W.clone()
    want = b.accumulate(decay=0.5).clone()
    b.close(before, want, decay=0.5)
    b.d["page_table"] = torch.cat([b.table, torch.full((4, 1 << 20), -1, dtype=torch.int32)], 1).cuda()
    b.W.copy_(before)
    got = b.accumulate(decay=0.5)
    b.close(before, got, decay=0.5)
    assert torch.equal(got, want) or (pool == "bf16" and max(n) > 2)


@pytest.mark.parametrize("pool, n, more", [("bf16", [1, 1, 0, 2], 0), ("f32", [1, 1, 0, 2], 0), ("bf16", [1, 40, 2, 1], 21)])
def test_scores_that_a_workspace_has_room_for_or_not(pool, n, more):
    """In a wide table scores are kept in what the workspace has beyond its least size, if it holds all of them."""
    kv = [70000, 5000, 66000, 2] if more else [700, 5000, 30, 2]
    Hq, Hkv = (2 * more, more) if more else (4, 2)
    b = Batch(n, kv, 256, Hq, Hkv, 64, pool, seed=6).fill()
    b.d["page_table"] = torch.cat([b.table, torch.full((4, 1 << 20), -1, dtype=torch.int32)], 1).cuda()
    least = cxa.cxa_paged_weights_workspace_bytes(b.cache.handle, 4, b.N, b.max_new, b.d["page_table"].shape[1], Hq)
    before = b.W.clone()
    few = [k for m, k in zip(n, kv) if 1 <= m <= 2]
    chunks, rows = sum(-(-k // 128) for k in few) * Hkv, 2 * (Hq // Hkv)
    for room in (chunks, chunks - 1, 0, 1):
        ws = torch.zeros(least + room * rows * 512 + (1 << 12), dtype=torch.uint8, device="cuda")
        ws[cxa.CXA_PAGED_COUNTER_BYTES:] = 255
        size = least + room * rows * 512
        b.W.copy_(before)
        b.accumulate(workspace=ws[:size])
        b.close(before, b.W)
        assert bool((ws[size:] == 255).all())


@pytest.mark.parametrize("Hq, Hkv", [(8, 2), (5, 1), (12, 1), (16, 1), (20, 1)])
def test_single_tokens_beside_prompts_in_a_large_pool(Hq, Hkv):
    """A table and a pool that can hold so many keys that sequences of few query rows go a way of their own."""
    b = Batch([1, 70, 2, 0, 1, 3, 40], [70000, 300, 66000, 100, 1, 9000, 40], 256, Hq, Hkv, 64, "bf16", seed=Hq,
              spare=(1 << 20) // 256 // Hkv).fill()
    b.d["page_table"] = torch.cat([b.table, torch.full((7, 2000), -1, dtype=torch.int32)], 1).cuda()
    before = b.W.clone()
    first = b.accumulate().clone()
    b.close(before, first)
    b.W.copy_(before)
    assert torch.equal(b.accumulate(), first)
