"""Paged self-attention on the GPU (norms and rotation, append, attention) against plain
fp64 forms written out here.

Tolerances, per element, count roundings: u is half a step of the output type (bf16 2^-8,
fp32 2^-24).

* Norm and rotation: |got - ref| <= u |ref| + 2^-20 (|A| + |B|), A and B the two products
  of the pair: fp32 steps of the norm (64 or 128 squares, rsqrt, weight) and the sine and
  cosine (a phase rounded to 24 bits of half a turn: pi * 2^-24).
* Attention: |got - ref| <= u |ref| + (e_p + e_s) A, A = sum p |V| of the row. e_p is the
  probabilities' rounding: 2^-15 (two truncated bf16 parts) with bf16 tensors on the
  few-rows kernel, 2^-8 where they are one bf16 value, 2^-19 in fp32 (parts left out, ex2,
  sums of up to 2^11 terms); e_s that of the scores, 2 * 2^-21 * scale * max sum |q||k|
  (fp32 sums and the parts left out).
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


# ------------------------------------------------------------------ plain forms, fp64
def turn(x, pos, rotary=None, layout="half", eps=None, w=None):
    """Returns the result and the sum of the magnitudes added for it."""
    y = x.double().clone()
    if eps is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
        if w is not None:
            y = y * w.double()
    mag = y.abs()
    if rotary is None:
        return y, mag
    h, m = rotary.rot_dim // 2, rotary.attn_factor
    ang = pos.double()[:, None] * torch.tensor(rotary.freq, dtype=torch.float64)
    c, s = m * torch.cos(ang)[:, None], m * torch.sin(ang)[:, None]
    lo, hi = (slice(0, h), slice(h, 2 * h)) if layout == "half" else (slice(0, 2 * h, 2), slice(1, 2 * h, 2))
    a, b = y[..., lo].clone(), y[..., hi].clone()
    y[..., lo], y[..., hi] = a * c - b * s, a * s + b * c
    mag[..., lo] = mag[..., hi] = m * (a.abs() + b.abs())
    return y, mag


def close_turn(got, ref, mag):
    got = got.detach().cpu()
    over = (got.double() - ref).abs() - U[got.dtype] * ref.abs() - 2.0 ** -20 * mag
    assert got.numel() == 0 or float(over.max()) <= 0


class Batch:
    """Sequences with n new tokens of kv keys each, in shuffled pages."""

    def __init__(self, n, kv, page, Hq, Hkv, dh, act, pool, seed=0, L=1, layer=0, spare=3, pad=0, extra_cols=1):
        self.n, self.kv, self.page, self.Hq, self.Hkv, self.dh, self.layer = n, kv, page, Hq, Hkv, dh, layer
        self.B = len(n)
        need = [-(-k // page) for k in kv]
        P = sum(need) + spare
        self.cache = cxa.PagedCache(P, page, L, Hkv, dh, pool)
        g = torch.Generator().manual_seed(seed + 77)
        perm = torch.randperm(P, generator=g).tolist()
        width = max(need + [0]) + extra_cols
        self.table = torch.full((self.B, width), -1, dtype=torch.int32)
        for b in range(self.B):
            for i in range(need[b]):
                self.table[b, i] = perm.pop()
        starts = [0]
        for x in n:
            starts.append(starts[-1] + x)
        self.starts, self.N = starts, starts[-1] + pad
        self.q = randn(self.N, Hq, dh, seed=seed + 1, dtype=DT[act])
        self.K = [randn(k, Hkv, dh, seed=seed + 100 + b, dtype=DT[pool]) for b, k in enumerate(kv)]
        self.V = [randn(k, Hkv, dh, seed=seed + 500 + b, dtype=DT[pool]) for b, k in enumerate(kv)]
        self.d = dict(q_start=torch.tensor(starts, dtype=torch.int32).cuda(),
                      kv_len=torch.tensor(kv, dtype=torch.int32).cuda(), page_table=self.table.cuda())
        self.max_new = max(n + [1])

    def fill(self, rest=None):
        """Write every key's row into its page; all other rows of the pool hold `rest`."""
        Kp, Vp = self.cache.Kp[self.layer].cpu(), self.cache.Vp[self.layer].cpu()
        if rest is not None:
            Kp.fill_(rest)
            Vp.fill_(rest)
        for b in range(self.B):
            for t in range(0, self.kv[b], self.page):
                p, m = int(self.table[b, t // self.page]), min(self.page, self.kv[b] - t)
                Kp[p, :, :m] = self.K[b][t:t + m].transpose(0, 1)
                Vp[p, :, :m] = self.V[b][t:t + m].transpose(0, 1)
        self.cache.Kp[self.layer].copy_(Kp)
        self.cache.Vp[self.layer].copy_(Vp)
        return self

    def attend(self, q=None, **kw):
        kw.setdefault("max_new", self.max_new)
        return self.cache.attend(self.layer, (self.q if q is None else q).cuda(), **self.d, **kw)

    def reference(self, scale=None):
        """out, sum p |V|, and the largest scale * sum |q||k|, in fp64, on the GPU."""
        scale = scale or 1 / math.sqrt(self.dh)
        G = self.Hq // self.Hkv
        out = torch.zeros(self.N, self.Hq, self.dh, dtype=torch.float64, device="cuda")
        A = torch.zeros_like(out)
        big = 0.0
        for b in range(self.B):
            n, kv = self.n[b], self.kv[b]
            if n == 0 or kv == 0:
                continue
            q = self.q[self.starts[b]:self.starts[b + 1]].cuda().double()
            K, V = self.K[b].cuda().double(), self.V[b].cuda().double()
            tame = bool(V.isfinite().all())
            seen = torch.arange(kv, device="cuda")[None] <= (kv - n + torch.arange(n, device="cuda"))[:, None]
            for h in range(self.Hq):
                s = q[:, h] @ K[:, h // G].T * scale
                big = max(big, float((q[:, h].abs() @ K[:, h // G].abs().T * scale).nan_to_num(0, 0, 0).max()))
                s = s.masked_fill(~seen, -math.inf)
                top = s.amax(-1, keepdim=True)
                p = torch.where(seen, torch.exp(s - torch.where(top.isinf(), 0.0, top)), 0.0)
                l = p.sum(-1, keepdim=True)
                w = torch.where(l == 0, 0.0, p / l)
                rows = slice(self.starts[b], self.starts[b + 1])
                if tame:
                    out[rows, h], A[rows, h] = w @ V[:, h // G], w @ V[:, h // G].abs()
                    continue
                for i in range(n):
                    out[rows.start + i, h] = w[i, seen[i]] @ V[seen[i], h // G]
                    A[rows.start + i, h] = w[i, seen[i]] @ V[seen[i], h // G].abs()
        return out.cpu(), A.cpu(), big

    def close(self, got, scale=None, one_bf16=None):
        out, A, big = self.reference(scale)
        rows = slice(0, self.starts[-1])
        got = got.detach().cpu()
        if one_bf16 is None:    # a sequence of many rows may go to the kernel of one bf16 probability
            one_bf16 = self.max_new * (self.Hq // self.Hkv) > 16
        ep = 2.0 ** -19 if got.dtype == torch.float32 else 2.0 ** -8 if one_bf16 else 2.0 ** -15
        over = (got.double() - out).abs() - U[got.dtype] * out.abs() - (ep + 2 * 2.0 ** -21 * big) * A
        fin = out.isfinite()[rows]
        assert bool((got[rows].isfinite() == fin).all())
        assert not bool(fin.any()) or float(over[rows][fin].max()) <= 0


# ------------------------------------------------------------------ norms and rotation
ROT = [dict(rot_dim=64), dict(rot_dim=64, layout="interleaved"), dict(rot_dim=32, scaling="linear", factor=4.0),
       dict(rot_dim=48, layout="interleaved", scaling="ntk", factor=8.0), dict(rot_dim=2),
       dict(rot_dim=38, layout="half"), dict(rot_dim=10, layout="interleaved"),
       dict(rot_dim=64, scaling="wavelength", factor=16.0, orig_len=2048), None]


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("i", range(len(ROT)))
def test_norm_rope(dh, act, norm, i):
    kw = dict(ROT[i]) if ROT[i] else None
    if kw and dh == 128 and i in (0, 1, 7):
        kw["rot_dim"] = 128
    rot = cxa.Rotary(**kw) if kw else None
    layout = kw.get("layout", "half") if kw else "half"
    for N, Hq, Hk in [(1, 20, 20), (7, 6, 1), (3, 1, 9), (300, 8, 2)]:
        qkv = randn(N, Hq + 2 * Hk, dh, seed=N + Hq, dtype=DT[act]).cuda()      # strided slices of one projection
        q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
        before = qkv.clone()
        pos = torch.randint(-5, 1 << 20, (N,), generator=torch.Generator().manual_seed(N), dtype=torch.int32)
        pos[0] = 0
        pos[-1] = 2 ** 30 - 1 if N > 1 else 447
        wq, wk = 1 + randn(dh, seed=3, scale=0.2), 1 + randn(dh, seed=4, scale=0.2)
        args = dict(rotary=rot, norm_eps=1e-6 if norm else None)
        if norm and Hq != 8:
            args.update(q_weight=wq.cuda(), k_weight=wk.cuda())
        qo, ko = cxa.qk_norm_rope(q, k, pos.cuda(), **args)
        assert torch.equal(qkv, before)
        for got, x, w in [(qo, q, wq), (ko, k, wk)]:
            ref, mag = turn(x.cpu(), pos, rot, layout, args["norm_eps"], w if "q_weight" in args else None)
            close_turn(got, ref, mag)
        # in place, on the strided slices
        cxa.qk_norm_rope(q, k, pos.cuda(), q_out=q, k_out=k, **args)
        assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(qkv[:, Hq + Hk:], before[:, Hq + Hk:])


def test_norm_rope_queries_alone_and_empty():
    rot = cxa.Rotary(64)
    q = randn(5, 3, 64, seed=1).cuda()
    pos = torch.arange(5, dtype=torch.int32).cuda()
    qo, ko = cxa.qk_norm_rope(q, None, pos, rotary=rot)
    assert ko is None
    close_turn(qo, *turn(q.cpu(), pos.cpu(), rot))
    e = cxa.qk_norm_rope(q[:0], q[:0], pos[:0], rotary=rot)
    assert e[0].shape == (0, 3, 64) and e[1].shape == (0, 3, 64)


def test_norm_rope_far_positions_agree_with_near_ones():
    """With frequencies of whole eighths of a turn, position p and p + 8 * 10^7 coincide."""
    rot = cxa.Rotary(64, freq=[2 * math.pi * (i % 8) / 8 for i in range(32)])
    q = randn(9, 4, 64, seed=2).cuda()
    pos = torch.arange(9, dtype=torch.int32).cuda()
    a, _ = cxa.qk_norm_rope(q, None, pos, rotary=rot)
    b, _ = cxa.qk_norm_rope(q, None, pos + 80_000_000, rotary=rot)
    close_turn(b, *turn(q.cpu(), pos.cpu(), rot))
    assert float((a - b).abs().max()) <= 2.0 ** -20 * 8


def test_norm_rope_unrotated_channels_see_no_neighbours_infinity():
    q = torch.ones(2, 2, 64).cuda()
    q[:, 0, 5] = math.inf
    q[:, 1, 40] = math.nan
    out, _ = cxa.qk_norm_rope(q, None, torch.tensor([1, 2], dtype=torch.int32).cuda(), rotary=cxa.Rotary(16))
    assert bool(out[:, 0, 16:].eq(1).all()) and int(out[:, 0].isfinite().logical_not().sum()) == 2 * 2
    assert int(out[:, 1].isnan().sum()) == 2 and bool(out[:, 1, 40].isnan().all())


def test_rotated_rows_feed_the_contiguous_step():
    """Queries and keys rotated in front of cxa_self_attention_step: scores depend on distance alone."""
    B, L, H, T, S = 2, 2, 3, 64, 9
    rot = cxa.Rotary(64)
    c = cxa.CrossAttentionCache(B, T, L, H, 64, "f32")
    q0, k0 = randn(B, L * H, 64, seed=1), randn(B, L * H, 64, seed=2)
    outs, vs = [], []
    for s in range(S):
        pos = torch.full((B,), s, dtype=torch.int32)
        q, k = cxa.qk_norm_rope(q0.cuda(), k0.cuda(), pos.cuda(), rotary=rot, norm_eps=1e-6)
        v = randn(B, L, H, 64, seed=10 + s)
        vs.append(v)
        outs.append(c.self_attention_step(pos.cuda(), q.view(B, L, H, 64), k.view(B, L, H, 64), v.cuda()))
    qn, kn = turn(q0, torch.zeros(B), None, eps=1e-6)[0], turn(k0, torch.zeros(B), None, eps=1e-6)[0]
    for s in range(S):
        kr = torch.stack([turn(kn, torch.full((B,), float(t - s)), rot)[0] for t in range(s + 1)], 2)   # [B, LH, s+1, 64]
        p = torch.softmax((qn[:, :, None] * kr).sum(-1) / 8, -1)
        ref = (p[..., None] * torch.stack(vs[:s + 1], 3).double().view(B, L * H, s + 1, 64)).sum(2)
        assert float((outs[s].cpu().double().view(B, L * H, 64) - ref).abs().max()) <= 1e-4


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("act,pool", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("dh,page", [(64, 16), (128, 32), (64, 256)])
def test_append(act, pool, dh, page):
    for n, kv, Hq, Hkv, i, norm in [([1], [1], 4, 4, 0, True), ([1, 1, 1], [17, 1, 33], 8, 2, 3, False),
                                    ([0, 40, 0, 3, 1], [5, 50, 0, 3, 300], 6, 6, 5, True),
                                    ([70, 33], [70, 600], 5, 1, 1, True), ([2] * 70, [9] * 70, 2, 2, 8, False)]:
        bt = Batch(n, kv, page, Hq, Hkv, dh, act, pool, L=2, layer=1, pad=4)
        bt.cache.Kp.copy_(randn(*bt.cache.Kp.shape, seed=5))
        bt.cache.Vp.copy_(randn(*bt.cache.Vp.shape, seed=6))
        K0, V0 = bt.cache.Kp.cpu(), bt.cache.Vp.cpu()
        kw = ROT[i]
        rot = cxa.Rotary(**kw) if kw else None
        layout = kw.get("layout", "half") if kw else "half"
        qkv = randn(bt.N, Hq + 2 * Hkv, dh, seed=9, dtype=DT[act]).cuda()
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        wk = 1 + randn(dh, seed=8, scale=0.2)
        eps = 1e-5 if norm else None
        q_out = torch.full((bt.N, Hq, dh), 7.0, dtype=DT[act]).cuda()
        got = bt.cache.append(1, k, v, **bt.d, q=q, q_out=q_out, rotary=rot, norm_eps=eps, k_weight=wk.cuda())
        assert got is q_out
        T = bt.starts[-1]
        assert bool((q_out[T:] == 7).all())                       # rows behind the last sequence
        pos = torch.cat([torch.arange(c - a, c) for a, c in zip(n, kv)] + [torch.zeros(0)]).double()
        close_turn(q_out[:T], *turn(q[:T].cpu(), pos, rot, layout, eps))
        rk, mk = turn(k[:T].cpu(), pos, rot, layout, eps, wk)
        Kg, Vg = bt.cache.Kp.cpu(), bt.cache.Vp.cpu()
        touched = torch.zeros(Kg.shape[1], page, dtype=torch.bool)
        for b in range(bt.B):
            for j in range(n[b]):
                t = kv[b] - n[b] + j
                p, s, r = int(bt.table[b, t // page]), t % page, bt.starts[b] + j
                touched[p, s] = True
                close_turn(Kg[1, p, :, s], rk[r], mk[r])
                assert torch.equal(Vg[1, p, :, s], v[r].cpu().to(DT[pool]))
        assert torch.equal(Kg[0], K0[0]) and torch.equal(Vg[0], V0[0])
        keep = ~touched
        assert torch.equal(Kg[1].transpose(1, 2)[keep], K0[1].transpose(1, 2)[keep])
        assert torch.equal(Vg[1].transpose(1, 2)[keep], V0[1].transpose(1, 2)[keep])


def test_append_many_sequences_and_queries_in_place():
    n = [(b * 7) % 4 for b in range(1100)]
    bt = Batch(n, [x + b % 40 for b, x in enumerate(n)], 16, 2, 1, 64, "f32", "f32")
    rot = cxa.Rotary(64)
    k, v, q = (randn(bt.N, h, 64, seed=h + 3).cuda() for h in (1, 1, 2))
    want = q.clone()
    pos = torch.cat([torch.arange(c - a, c) for a, c in zip(bt.n, bt.kv)])
    bt.cache.append(0, k, v, **bt.d, q=q, q_out=q, rotary=rot)
    close_turn(q, *turn(want.cpu(), pos, rot))
    ref, mag = turn(k.cpu(), pos, rot)
    page = torch.cat([bt.table[b, torch.arange(c - a, c) // 16] for b, (a, c) in enumerate(zip(bt.n, bt.kv))]).long()
    close_turn(bt.cache.Kp.cpu()[0, page, 0, pos % 16], ref[:, 0], mag[:, 0])


# ------------------------------------------------------------------ attention
TYPES = [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")]
SHAPES = [  # n, kv, page, Hq, Hkv
    ([1], [1], 16, 1, 1),
    ([1], [448], 16, 8, 8),
    ([1, 1, 1, 1], [15, 16, 17, 333], 16, 8, 2),
    ([5, 5, 5], [5, 64, 1000], 32, 6, 6),
    ([3, 0, 1, 2], [3, 90, 129, 65], 64, 20, 4),
    ([1] * 40, [1 + 37 * b for b in range(40)], 256, 8, 1),
    ([130], [130], 128, 4, 4),
    ([63, 1, 257], [64, 2000, 700], 16, 5, 1),
    ([40, 200], [4097, 200], 128, 16, 2),
]


@pytest.mark.parametrize("act,pool", TYPES)
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_attention(act, pool, dh, i):
    n, kv, page, Hq, Hkv = SHAPES[i]
    bt = Batch(n, kv, page, Hq, Hkv, dh, act, pool, seed=i).fill()
    bt.close(bt.attend())
    bt.close(bt.attend(scale=0.3), scale=0.3)


@pytest.mark.parametrize("act,pool", TYPES)
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("n,kv,Hq,Hkv", [([1], [70001], 2, 1), ([24], [40003], 1, 1), ([200, 1], [30001, 9000], 2, 1),
                                         ([3, 1], [70, 50], 100, 1), ([9, 1, 70], [90, 20, 75], 130, 1),
                                         ([1] * 700, [1 + b % 40 for b in range(700)], 2, 1)])
def test_long_merges_many_heads_and_many_sequences(act, pool, dh, n, kv, Hq, Hkv):
    """One K/V head cut into more parts than are merged at once; more query heads on a K/V head
    than a tile has rows; more sequences than a block has threads."""
    bt = Batch(n, kv, 16 if len(n) > 10 else 256, Hq, Hkv, dh, act, pool).fill()
    got = bt.attend()
    bt.close(got)
    assert torch.equal(bt.attend(), got)


@pytest.mark.parametrize("act,pool", TYPES)
@pytest.mark.parametrize("n,kv", [([1, 1], [20, 470]), ([7, 5], [40, 470]), ([150, 90], [150, 470])])
def test_rows_behind_the_last_key_may_hold_anything(act, pool, n, kv):
    for rest in (math.nan, math.inf, -math.inf):
        bt = Batch(n, kv, 64, 4, 2, 64, act, pool).fill(rest=rest)
        bt.close(bt.attend())


@pytest.mark.parametrize("act,pool", TYPES)
@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("n,kv,bad", [([6], [40], 37), ([8, 3], [8, 100], 5), ([200], [460], 300), ([300], [300], 129),
                                      ([140], [140], 139)])
def test_a_later_token_s_infinities_do_not_reach_an_earlier_one(act, pool, dh, n, kv, bad):
    for what in (math.nan, math.inf):
        bt = Batch(n, kv, 16, 4, 2, dh, act, pool)
        bt.V[0][bad, 1, 3] = what
        bt.K[0][bad, 0, 5] = math.nan
        bt.fill()
        got = bt.attend().cpu()
        first = bad - (kv[0] - n[0])          # rows before it never see it
        want = Batch(n, kv, 16, 4, 2, dh, act, pool).fill().attend().cpu()
        assert bool(got[:max(first, 0)].isfinite().all())
        if len(n) > 1:
            assert torch.equal(got[n[0]:], want[n[0]:])
        assert bool(got[first:n[0], :2].isnan().all())        # heads of K/V head 0: a NaN score
        assert not bool(got[first:n[0], 2:, 3].isfinite().any())
        bt.close(got)


@pytest.mark.parametrize("act,pool", TYPES)
def test_large_scores_pick_one_key(act, pool):
    """A key along each query, 200 above the rest in the exponent: the result is its V."""
    n, kv = [1, 4, 150], [300, 260, 700]
    bt = Batch(n, kv, 32, 4, 4, 64, act, pool)
    for b in range(3):
        at = [0, 130, kv[b] - n[b]][b]
        for h in range(4):
            bt.K[b][:, h] = 0.01 * bt.K[b][:, h]
            q = bt.q[bt.starts[b], h].float()
            bt.q[bt.starts[b]:bt.starts[b + 1], h] = bt.q[bt.starts[b], h].clone()
            bt.K[b][at, h] = (q * 1600 / (q @ q)).to(DT[pool])
    bt.fill()
    got = bt.attend().cpu()
    for b, at in enumerate([0, 130, 550]):
        rows = slice(bt.starts[b], bt.starts[b + 1])
        assert torch.equal(got[rows], bt.V[b][at].to(got.dtype).expand(n[b], 4, 64))


def test_masked_scores_of_the_lowest_value():
    """K of the type's lowest value: scores of -inf weigh nothing, the rest is as without them."""
    bt = Batch([1, 30], [200, 200], 16, 2, 2, 64, "bf16", "bf16")
    bt.q = bt.q.abs() + 1
    for b in range(2):
        bt.K[b][50:90] = torch.finfo(torch.bfloat16).min
    bt.fill()
    got = bt.attend()
    assert bool(got.isfinite().all())
    one = Batch([1, 30], [160, 160], 16, 2, 2, 64, "bf16", "bf16")
    one.q = bt.q
    one.K, one.V = ([torch.cat([x[:50], x[90:]]) for x in y] for y in (bt.K, bt.V))
    one.close(got)


def test_empty_sequences_and_padding_are_left_alone():
    for n, kv in [([0, 0], [0, 10]), ([0, 3, 0], [7, 3, 0]), ([0], [0])]:
        bt = Batch(n, kv, 16, 4, 2, 64, "bf16", "bf16", pad=5).fill()
        out = torch.full((bt.N, 4, 64), 3.0, dtype=torch.bfloat16).cuda()
        bt.attend(out=out)
        assert bool((out[bt.starts[-1]:] == 3).all())
        bt.close(out)


@pytest.mark.parametrize("act,pool", TYPES)
def test_tokens_without_a_key_are_zero(act, pool):
    """kv_len below the new tokens: the first ones see nothing."""
    for n in (5, 200):
        bt = Batch([n], [n], 16, 4, 2, 64, act, pool).fill()
        bt.d["kv_len"] = torch.tensor([n - 3], dtype=torch.int32).cuda()
        got = bt.attend().cpu()
        assert bool((got[:3] == 0).all()) and bool(got[3:].isfinite().all())
        one = Batch([n - 3], [n - 3], 16, 4, 2, 64, act, pool)
        one.q, one.K, one.V = bt.q[3:], [bt.K[0][:n - 3]], [bt.V[0][:n - 3]]
        one.close(got[3:], one_bf16=n > 100)
        bt.d["kv_len"] = torch.tensor([0], dtype=torch.int32).cuda()
        assert bool((bt.attend() == 0).all())


def test_strided_queries_and_outputs():
    for n, kv in [([1, 3], [50, 40]), ([140], [200])]:
        bt = Batch(n, kv, 16, 6, 2, 64, "bf16", "bf16").fill()
        want = bt.attend()
        buf = torch.zeros(bt.N, 10, 64, dtype=torch.bfloat16).cuda()
        buf[:, 2:8] = bt.q.cuda()
        out = torch.full((bt.N, 9, 64), 5.0, dtype=torch.bfloat16).cuda()
        bt.cache.attend(0, buf[:, 2:8], **bt.d, max_new=bt.max_new, out=out[:, 1:7])
        assert torch.equal(out[:, 1:7], want)
        assert bool((out[:, 0] == 5).all()) and bool((out[:, 7:] == 5).all())


@pytest.mark.parametrize("max_new", [1, 4, 1000])
def test_a_wrong_bound_of_new_tokens_changes_nothing(max_new):
    bt = Batch([1, 60, 2, 300], [100, 90, 2, 1000], 32, 8, 4, 64, "bf16", "bf16").fill()
    bt.close(bt.attend(max_new=max_new), one_bf16=True)


def test_repeated_calls_agree_bit_for_bit():
    for n, kv in [([1] * 9, [3000 - 300 * b for b in range(9)]), ([300, 1, 40], [2000, 5000, 700])]:
        bt = Batch(n, kv, 64, 8, 2, 64, "bf16", "bf16").fill()
        want = bt.attend()
        for _ in range(5):
            assert torch.equal(bt.attend(), want)


def test_pages_outside_the_pool_are_left_out_and_reported():
    assert cxa.cxa_device_status(1) == cxa.CXA_OK
    for n in (1, 40):
        for bad in (-1, 10 ** 6, -2 ** 31):
            bt = Batch([n], [160], 16, 4, 2, 64, "bf16", "bf16").fill()
            bt.d["page_table"][0, 3] = bad
            got = bt.attend()
            assert cxa.cxa_device_status(1) == cxa.CXA_EPAGE
            keep = [t for t in range(160) if t // 16 != 3]
            one = Batch([n], [144], 16, 4, 2, 64, "bf16", "bf16")
            one.q, one.K, one.V = bt.q, [bt.K[0][keep]], [bt.V[0][keep]]
            one.close(got, one_bf16=n > 1)
            # an append into such a page, or behind the table's row, writes nothing
            bt.d["kv_len"] = torch.tensor([48 + n], dtype=torch.int32).cuda()
            if n == 1:
                K0, V0 = bt.cache.Kp.clone(), bt.cache.Vp.clone()
                k = randn(1, 2, 64, seed=1, dtype=torch.bfloat16).cuda()
                bt.cache.append(0, k, k, **bt.d)
                assert cxa.cxa_device_status(1) == cxa.CXA_EPAGE
                bt.d["kv_len"] = torch.tensor([16 * 11 + 1], dtype=torch.int32).cuda()
                bt.cache.append(0, k, k, **bt.d)
                assert cxa.cxa_device_status(1) == cxa.CXA_EPAGE
                assert torch.equal(bt.cache.Kp, K0) and torch.equal(bt.cache.Vp, V0)


@pytest.mark.parametrize("act,pool", TYPES)
@pytest.mark.parametrize("n", [1, 40])
def test_keys_behind_the_table_s_row_are_left_out_and_reported(act, pool, n):
    assert cxa.cxa_device_status(1) == cxa.CXA_OK
    bt = Batch([n], [160], 16, 4, 2, 64, act, pool, extra_cols=0).fill()
    bt.close(bt.attend(), one_bf16=n > 1)
    assert cxa.cxa_device_status(1) == cxa.CXA_OK
    bt.d["kv_len"] = torch.tensor([160 + n], dtype=torch.int32).cuda()      # no token sees less than 160
    got = bt.attend()
    assert cxa.cxa_device_status(1) == cxa.CXA_EPAGE
    one = Batch([1] * n, [160] * n, 16, 4, 2, 64, act, pool)
    one.q, one.K, one.V = bt.q, [bt.K[0]] * n, [bt.V[0]] * n
    one.close(got, one_bf16=n > 1)


def test_offsets_past_32_bits():
    """A pool of more than 2^32 elements, its sequences at both ends of it."""
    page, Hkv, dh = 256, 8, 64
    P = (1 << 32) // (page * Hkv * dh) + 40
    bt = Batch([1, 200], [300, 700], page, 8, Hkv, dh, "bf16", "bf16")
    bt.cache = cxa.PagedCache(P, page, 1, Hkv, dh, "bf16")
    remap = {}
    for b in range(2):
        for i in range(bt.table.shape[1]):
            t = int(bt.table[b, i])
            if t >= 0:
                bt.table[b, i] = remap.setdefault(t, P - 1 - len(remap) if len(remap) % 2 else len(remap))
    bt.d["page_table"] = bt.table.cuda()
    assert int(bt.table.max()) * page * Hkv * dh > 1 << 32
    for b in range(2):
        for t in range(0, bt.kv[b], page):
            p, m = int(bt.table[b, t // page]), min(page, bt.kv[b] - t)
            bt.cache.Kp[0, p, :, :m] = bt.K[b][t:t + m].transpose(0, 1).cuda()
            bt.cache.Vp[0, p, :, :m] = bt.V[b][t:t + m].transpose(0, 1).cuda()
    bt.close(bt.attend())
    k = randn(201, Hkv, dh, seed=4, dtype=torch.bfloat16).cuda()
    bt.cache.append(0, k, k, **bt.d)
    for b in range(2):
        t = bt.kv[b] - 1
        assert torch.equal(bt.cache.Vp[0, int(bt.table[b, t // page]), :, t % page], k[bt.starts[b + 1] - 1])


# ------------------------------------------------------------------ the run as it is used
@pytest.mark.parametrize("act,pool", TYPES)
@pytest.mark.parametrize("graph", [False, True])
def test_prompt_then_steps(act, pool, graph):
    """Prompts of two sequences in chunks, then single tokens and a proposal of three, two
    layers: append with norms and rotation, then attention, against one pass over the whole
    sequence in fp64 on the rows that the pool holds."""
    L, Hq, Hkv, dh, page = 2, 4, 2, 64, 16
    total = [150, 70]
    plan = [[100, 17], [40, 48], [1, 1], [1, 1], [3, 0], [5, 3]]
    rot = cxa.Rotary(48, scaling="wavelength", factor=4.0, orig_len=64)
    bt = Batch([0, 0], total, page, Hq, Hkv, dh, act, pool, L=L)
    w = (1 + randn(dh, seed=5, scale=0.2)).cuda()
    done = [0, 0]
    pad = 120
    bufs = {x: torch.zeros(pad, h, dh, dtype=DT[act]).cuda() for x, h in (("q", Hq), ("k", Hkv), ("v", Hkv))}
    q_start, kv_len = torch.zeros(3, dtype=torch.int32).cuda(), torch.zeros(2, dtype=torch.int32).cuda()
    table = bt.table.cuda()
    outs = [torch.zeros(pad, Hq, dh, dtype=DT[act]).cuda() for _ in range(L)]

    def step():
        for l in range(L):
            qr = bt.cache.append(l, bufs["k"] * (l + 1), bufs["v"] * (l + 1), q_start, kv_len, table, q=bufs["q"],
                                 rotary=rot, norm_eps=1e-6, q_weight=w, k_weight=w)
            bt.cache.attend(l, qr, q_start, kv_len, table, max_new=100, out=outs[l])

    g = None
    if graph:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()                       # a batch of nothing: loads the kernels
        torch.cuda.current_stream().wait_stream(s)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
    qs, got = [[], []], [[[], []] for _ in range(L)]
    for i, n in enumerate(plan):
        for x in bufs:
            bufs[x].copy_(randn(*bufs[x].shape, seed=1000 * i + ord(x), dtype=DT[act]))
        done = [d + a for d, a in zip(done, n)]
        q_start.copy_(torch.tensor([0, n[0], n[0] + n[1]], dtype=torch.int32))
        kv_len.copy_(torch.tensor(done, dtype=torch.int32))
        bt.cache.check(q_start.cpu(), kv_len.cpu(), table.cpu(), pad)
        if g:
            g.replay()
        else:
            step()
        lo = 0
        for b in range(2):
            qs[b].append(bufs["q"][lo:lo + n[b]].cpu())
            for l in range(L):
                got[l][b].append(outs[l][lo:lo + n[b]].cpu())
            lo += n[b]
    assert done == total
    for l in range(L):
        one = Batch(total, total, page, Hq, Hkv, dh, act, pool)
        for b in range(2):
            ids = [int(x) for x in bt.table[b, :-(-total[b] // page)]]
            one.K[b] = bt.cache.Kp[l, ids].cpu().transpose(1, 2).reshape(-1, Hkv, dh)[:total[b]]
            one.V[b] = bt.cache.Vp[l, ids].cpu().transpose(1, 2).reshape(-1, Hkv, dh)[:total[b]]
            qr, _ = cxa.qk_norm_rope(torch.cat(qs[b]).cuda(), None, torch.arange(total[b], dtype=torch.int32).cuda(),
                                     rotary=rot, norm_eps=1e-6, q_weight=w)
            one.q[one.starts[b]:one.starts[b + 1]] = qr.cpu()
        one.close(torch.cat([torch.cat(got[l][0]), torch.cat(got[l][1])]))


def test_two_streams_at_once():
    a = Batch([1] * 8, [4000 - 100 * b for b in range(8)], 64, 8, 2, 64, "bf16", "bf16", seed=1).fill()
    want = a.attend()
    streams = [torch.cuda.Stream() for _ in range(3)]
    q = a.q.cuda()
    torch.cuda.synchronize()
    outs = []
    for r in range(20):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(a.cache.attend(0, q, **a.d, max_new=1))
        out = torch.empty_like(want)
        torch.cuda.synchronize()
        outs.append(a.cache.attend(0, q, **a.d, max_new=1, stream=streams[r % 3].cuda_stream, out=out))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_results_on_another_stream_have_memory_of_that_stream():
    """Memory that the current stream still has work for is not handed to a call on another."""
    a = Batch([1] * 2, [300, 200], 16, 8, 2, 64, "bf16", "bf16").fill()
    want, q, s = a.attend(), a.q.cuda(), torch.cuda.Stream()
    pos = torch.arange(2, dtype=torch.int32).cuda()
    turned, _ = cxa.qk_norm_rope(q, None, pos, rotary=cxa.Rotary(64))
    torch.cuda.synchronize()
    for call, ref in ((lambda: a.cache.attend(0, q, **a.d, max_new=1, stream=s), want),
                      (lambda: cxa.qk_norm_rope(q, None, pos, rotary=cxa.Rotary(64), stream=s)[0], turned)):
        call()                                   # (kernels and workspace are there)
        torch.cuda.synchronize()
        old = [torch.empty_like(q) for _ in range(64)]
        torch.cuda._sleep(20_000_000)
        for x in old:
            x.fill_(7.0)
        del old, x
        got = call()
        torch.cuda.synchronize()
        assert torch.equal(got, ref)


def test_workspaces_are_kept_apart():
    a = Batch([1], [40], 16, 2, 2, 64, "bf16", "bf16").fill()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    kept = [a.cache.workspace(2, 1, stream=x).data_ptr() for x in (None, s, t)]
    assert len(set(kept)) == 3
    assert kept == [a.cache.workspace(2, 1, stream=x).data_ptr() for x in (None, s, t)]
    torch.cuda.synchronize()
    # the stream that is captured is the one the call names, whichever is current
    with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=s):
        with torch.cuda.stream(t):
            assert a.cache.workspace(2, 1, stream=s).data_ptr() not in kept
        assert a.cache.workspace(2, 1).data_ptr() not in kept
    assert kept[1] == a.cache.workspace(2, 1, stream=s).data_ptr()


def test_one_workspace_for_calls_of_all_shapes():
    cases = [Batch([200, 1], [3000, 9000], 64, 4, 1, dh, act, act, seed=dh).fill()
             for dh in (64, 128) for act in ("bf16", "f32")]
    cases.append(Batch([1], [60000], 64, 40, 1, 64, "bf16", "bf16").fill())
    want = [bt.attend() for bt in cases]
    n = max(cxa.cxa_paged_attention_workspace_bytes(bt.Hq, bt.Hkv, bt.dh, bt.max_new) for bt in cases)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")       # only the counters need be zero
    ws[:cxa.CXA_PAGED_COUNTER_BYTES] = 0
    for _ in range(2):
        for bt, ref in zip(cases, want):
            assert torch.equal(bt.attend(workspace=ws), ref)


def test_two_graphs_at_once():
    a = Batch([1] * 8, [4000 - 100 * b for b in range(8)], 64, 8, 2, 64, "bf16", "bf16", seed=1).fill()
    want, q = a.attend(), a.q.cuda()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append([a.cache.attend(0, q, **a.d, max_new=1) for _ in range(3)])
        graphs.append((g, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in graphs:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for os_ in outs for o in os_)


def test_python_refusals():
    bt = Batch([1, 2], [5, 9], 16, 4, 2, 64, "bf16", "bf16").fill()
    q = bt.q.cuda()
    with pytest.raises(ValueError):
        bt.cache.attend(0, q[:, :, :32], **bt.d, max_new=2)
    with pytest.raises(ValueError):
        bt.cache.attend(0, q.transpose(0, 1), **bt.d, max_new=2)
    with pytest.raises(ValueError):
        bt.cache.attend(0, bt.q, **bt.d, max_new=2)                       # on the host
    with pytest.raises(TypeError):
        bt.cache.attend(0, q.half(), **bt.d, max_new=2)
    with pytest.raises(TypeError):
        bt.cache.attend(0, q, **bt.d, max_new=2, out=torch.empty_like(q, dtype=torch.float32))
    with pytest.raises(ValueError):
        bt.cache.attend(0, q, bt.d["q_start"].long(), bt.d["kv_len"], bt.d["page_table"], max_new=2)
    with pytest.raises(ValueError):
        bt.cache.attend(0, q, bt.d["q_start"][:2], bt.d["kv_len"], bt.d["page_table"], max_new=2)
    with pytest.raises(cxa.CxaError):
        bt.cache.attend(1, q, **bt.d, max_new=2)
    with pytest.raises(cxa.CxaError):
        bt.cache.attend(0, q, **bt.d, max_new=2, out=q)
    with pytest.raises(ValueError):
        bt.cache.append(0, q, q, **bt.d)                                  # 4 heads, the pool has 2
    with pytest.raises(ValueError):
        cxa.qk_norm_rope(q[:1].expand(3, 4, 64), None, torch.zeros(3, dtype=torch.int32).cuda())
    f32 = cxa.PagedCache(4, 16, 1, 2, 64, "f32")
    with pytest.raises(cxa.CxaError):
        f32.attend(0, q, **bt.d, max_new=2)


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("G", [3, 4, 5, 7])
@pytest.mark.parametrize("n", [17, 60, 200])
def test_query_rows_of_no_token_change_no_bit(dh, G, n):
    """A 128-row tile also holds rows that are no token's of its sequence: padding behind the
    last sequence, the next sequence's tokens, and (G no divisor of 128) rows that no copy fills."""
    bt = Batch([n, 19], [n + 80000, 30000], 256, G, 1, dh, "bf16", "bf16", pad=50)
    for x in bt.K:          # scores that grow from chunk to chunk: rows with large q move their reference again and again
        x.mul_((1 + torch.arange(len(x)) // 64 % 16 / 2)[:, None, None])
    bt.q.mul_(0.25)
    bt.fill()
    filler = Batch([400], [400], 64, 4, 1, dh, "bf16", "bf16").fill()
    want = bt.attend()
    for i, scale in enumerate((0.0, 8.0, 60.0, math.inf, math.nan)):
        filler.attend(filler.q * (scale if scale < 1e3 else 1e4))      # what shared memory holds from before
        rest = randn(50, G, dh, seed=90 + i, dtype=torch.bfloat16)
        q = bt.q.clone()
        q[n + 19:] = rest * scale
        assert torch.equal(bt.attend(q)[:n + 19], want[:n + 19])
        q[n:n + 19] = rest[:19] * scale                                # the next sequence's
        assert torch.equal(bt.attend(q)[:n], want[:n])


def test_threads_share_a_stream_and_its_workspace():
    """Calls of two kernels, enqueued by threads at once on one stream: each is enqueued whole,
    so that the second kernels, which start early, never work on one another's scratch."""
    bts = [Batch([150, 1, 30], [20000, 900, 70], 64, 4, 1, dh, "bf16", "bf16", seed=s).fill() for s, dh in ((1, 64), (2, 128))]
    n = max(cxa.cxa_paged_attention_workspace_bytes(4, 1, bt.dh, bt.max_new) for bt in bts)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    want = [bt.attend() for bt in bts]
    outs = [[torch.zeros_like(w) for _ in range(40)] for w in want]
    qs = [bt.q.cuda() for bt in bts]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()

    def calls(i):
        for out in outs[i]:
            bts[i].cache.attend(0, qs[i], **bts[i].d, max_new=bts[i].max_new, out=out, workspace=ws, stream=stream)

    threads = [threading.Thread(target=calls, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in range(2) for o in outs[i])


@pytest.mark.parametrize("dh", [64, 128])
def test_attention_reads_what_the_grid_before_has_just_written(dh):
    """Append (which lets the next grid start early) and attention behind it, again and again over
    the same pages and queries: every call sees the rows of its own append, through copies too."""
    n, past, Hkv = 96, 700, 2
    bt = Batch([n], [past + n], 64, 4, Hkv, dh, "bf16", "bf16").fill()
    steps = []
    for i in range(12):
        k, v, q = (randn(n, h, dh, seed=10 * i + h + 40, dtype=torch.bfloat16).cuda() for h in (Hkv, Hkv, 4))
        steps.append((k, v, q, torch.zeros(n, 4, dh, dtype=torch.bfloat16, device="cuda")))
    qr = torch.empty_like(steps[0][2])
    torch.cuda.synchronize()
    for k, v, q, out in steps:
        bt.cache.append(0, k, v, **bt.d, q=q, q_out=qr)
        bt.cache.attend(0, qr, **bt.d, max_new=n, out=out)
    torch.cuda.synchronize()
    for k, v, q, out in steps:
        bt.K[0][past:], bt.V[0][past:], bt.q = k.cpu(), v.cpu(), q.cpu()
        bt.close(out)


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("n,kv", [(40, 2100), (300, 700), (300, 300)])
def test_bad_pages_among_chunks_of_many_rows(dh, page, n, kv):
    """Pages outside the pool at the start, in a row, at the causal limit and at the end: their keys
    are left out, whatever the places in shared memory held that no copy fills now; and a later
    token's infinity beside them stays with the tokens that see it."""
    poison = Batch([n], [kv], page, 4, 2, dh, "bf16", "bf16").fill(rest=math.nan)
    for t in (poison.cache.Kp, poison.cache.Vp):
        t.fill_(math.nan)
    bt = Batch([n], [kv], page, 4, 2, dh, "bf16", "bf16", seed=3)
    inf_at = kv - n + 5                                  # seen by the tokens from the sixth on
    bt.V[0][inf_at, 1, 3] = math.inf
    bt.fill()
    last = (kv - 1) // page
    bad = {i for i in (0, 2, 3, (kv - n) // page + 1, last) if i <= last and i != inf_at // page}
    for j, i in enumerate(sorted(bad)):
        bt.d["page_table"][0, i] = (-1, 10 ** 6, -2 ** 31)[j % 3]
    poison.attend()
    got = bt.attend().cpu()
    assert cxa.cxa_device_status(1) == cxa.CXA_EPAGE
    pos = torch.arange(kv)
    here = torch.tensor([i not in bad for i in range(last + 1)])[pos // page]
    K, V = bt.K[0].double(), bt.V[0].double()
    for h in range(4):
        q = bt.q[:, h].double()
        s = q @ K[:, h // 2].T / math.sqrt(dh)
        seen = (pos[None] <= (kv - n + torch.arange(n))[:, None]) & here[None]
        p = torch.softmax(s.masked_fill(~seen, -math.inf), -1).nan_to_num(0)       # (a row of bad pages alone: zero)
        big = float((q.abs() @ K[:, h // 2].abs().T / math.sqrt(dh)).max())
        Vh = V[:, h // 2].clone()
        hot = seen[:, inf_at] if h >= 2 else torch.zeros(n, dtype=torch.bool)
        Vh[inf_at, 3] = 0 if h >= 2 else Vh[inf_at, 3]
        ref, A = p @ Vh, p @ Vh.abs()
        g = got[:, h].double()
        assert bool(g[hot][:, 3].isinf().all())
        g[hot, 3] = ref[hot, 3]
        assert bool(((g - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * 2.0 ** -21 * big) * A).all())


def bad_page_call(stream=None):
    bt = Batch([1], [160], 16, 4, 2, 64, "bf16", "bf16").fill()
    bt.d["page_table"][0, 3] = -1
    q = bt.q.cuda()
    bt.cache.attend(0, q, **bt.d, max_new=1)         # (workspace and kernels are there)
    torch.cuda.synchronize()
    assert cxa.cxa_device_status(1) == cxa.CXA_EPAGE
    return lambda: bt.cache.attend(0, q, **bt.d, max_new=1, stream=stream)


def test_a_bad_page_is_not_lost_behind_a_timeout():
    """Two reports at once come one after the other; clearing takes back the one that was returned."""
    call = bad_page_call()
    call()
    assert cxa.cxa_selftest_wait_timeout(1000) == cxa.CXA_OK
    assert cxa.cxa_device_status(0) == cxa.CXA_ETIMEOUT
    assert cxa.cxa_device_status(1) == cxa.CXA_ETIMEOUT
    assert cxa.cxa_device_status(0) == cxa.CXA_EPAGE
    assert cxa.cxa_device_status(1) == cxa.CXA_EPAGE
    assert cxa.cxa_device_status(1) == cxa.CXA_OK


def test_device_status_waits_for_streams_of_any_kind():
    s = torch.cuda.Stream()                          # one that the default stream does not wait for
    call = bad_page_call(s)
    call()
    torch.cuda.synchronize()
    assert cxa.cxa_device_status(1) == cxa.CXA_EPAGE
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)
    call()
    assert cxa.cxa_device_status(1) == cxa.CXA_EPAGE
    torch.cuda.synchronize()
    assert cxa.cxa_device_status(1) == cxa.CXA_OK


def test_a_wide_table_gives_what_a_narrow_one_does():
    """A prompt of 65,536 tokens over a table of 2^20 positions (kept wide for a captured graph)."""
    n, past, page = 65536, 4000, 256
    need = -(-(n + past) // page)
    cache = cxa.PagedCache(need, page, 1, 8, 64, "bf16")
    cache.Kp.normal_()
    cache.Vp.normal_()
    q = torch.randn(n, 32, 64, device="cuda", dtype=torch.bfloat16)
    at = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, n], [n + past])]
    narrow = torch.randperm(need, device="cuda").to(torch.int32)[None].contiguous()
    wide = torch.full((1, 4096), -1, dtype=torch.int32, device="cuda")
    wide[:, :need] = narrow
    want = cache.attend(0, q, *at, narrow, max_new=n)
    assert bool(want.isfinite().all())
    assert torch.equal(cache.attend(0, q, *at, wide, max_new=n), want)
    # one bf16 probability, scores of up to 8 in magnitude
    # (the table's order of pages is the keys': the first token sees past + 1 of them)
    K = cache.Kp[0, narrow[0].long()].transpose(0, 1).reshape(8, -1, 64)
    V = cache.Vp[0, narrow[0].long()].transpose(0, 1).reshape(8, -1, 64)
    for i in (0, 12345, n - 1):
        kv = past + i + 1
        p = torch.softmax(torch.einsum("hgd,hkd->hgk", q[i].view(8, 4, 64).double(), K[:, :kv].double()) / 8, -1)
        ref = torch.einsum("hgk,hkd->hgd", p, V[:, :kv].double()).view(32, 64)
        A = torch.einsum("hgk,hkd->hgd", p, V[:, :kv].double().abs()).view(32, 64)
        assert bool(((want[i].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -16) * A).all())


def test_threads_own_default_streams_need_memory_of_the_caller():
    """One handle (2) stands for every thread's own default stream: no memory is kept or made for it."""
    a = Batch([1] * 2, [300, 200], 16, 8, 2, 64, "bf16", "bf16").fill()
    want, q, out = a.attend(), a.q.cuda(), torch.zeros(2, 8, 64, dtype=torch.bfloat16, device="cuda")
    ws = a.cache.workspace(8, 1)
    pos = torch.arange(2, dtype=torch.int32).cuda()
    turned, _ = cxa.qk_norm_rope(q, None, pos, rotary=cxa.Rotary(64))
    torch.cuda.synchronize()
    for kw in (dict(), dict(out=out), dict(workspace=ws)):
        with pytest.raises(ValueError, match="own default stream"):
            a.cache.attend(0, q, **a.d, max_new=1, stream=2, **kw)
    with pytest.raises(ValueError, match="own default stream"):
        a.cache.workspace(8, 1, stream=2)
    with pytest.raises(ValueError, match="own default stream"):
        cxa.qk_norm_rope(q, None, pos, rotary=cxa.Rotary(64), stream=2)
    got = []

    def calls():
        got.append(a.cache.attend(0, q, **a.d, max_new=1, stream=2, out=out, workspace=ws))
        got.append(cxa.qk_norm_rope(q, None, pos, rotary=cxa.Rotary(64), stream=2, q_out=torch.empty_like(q))[0])

    t = threading.Thread(target=calls)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want) and torch.equal(got[1], turned)


def test_workspaces_of_many_streams_are_bounded(monkeypatch):
    monkeypatch.setattr(cxa.PagedCache, "KEPT_WORKSPACES", 3)
    a = Batch([1] * 4, [2000, 900, 30, 4000], 16, 8, 2, 64, "bf16", "bf16").fill()
    want, q = a.attend(), a.q.cuda()
    streams = [torch.cuda.Stream() for _ in range(8)]
    torch.cuda.synchronize()
    outs = [a.cache.attend(0, q, **a.d, max_new=1, stream=s) for _ in range(6) for s in streams]
    assert len(a.cache._ws) == 3 and [s.cuda_stream for s in streams[-3:]] == list(a.cache._ws)
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    a.cache.close()
    assert not a.cache._ws
    with pytest.raises(cxa.CxaError, match="descriptor is NULL"):
        a.attend()


def test_counters_left_behind_go_with_the_kept_workspaces():
    """After a wait that ran out a kept workspace may hold counters: dropping it is enough."""
    a = Batch([1] * 4 + [60], [2000, 900, 30, 4000, 800], 16, 8, 2, 64, "bf16", "bf16").fill()
    want, s = a.attend(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (None, s):
        a.cache.workspace(8, 60, stream=stream)[:cxa.CXA_PAGED_COUNTER_BYTES] = 1
    torch.cuda.synchronize()
    a.cache.drop_workspaces()
    for stream in (None, s):
        got = a.attend(stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_starts_that_decrease_are_reported_and_touch_nothing_else(act):
    """Overlapping sequences, against the contract of q_start: reported, and never more work than
    can be numbered, however often they repeat."""
    bt = Batch([40, 3, 30], [300, 100, 90], 16, 4, 2, 64, act, act, pad=6).fill()
    bt.d["q_start"] = torch.tensor([0, 70, 20, 73], dtype=torch.int32).cuda()
    out = torch.full((bt.N, 4, 64), 3.0, dtype=DT[act]).cuda()
    K0, V0 = bt.cache.Kp.clone(), bt.cache.Vp.clone()
    bt.attend(out=out, max_new=70)
    assert cxa.cxa_device_status(1) == cxa.CXA_EINVAL
    assert cxa.cxa_device_status(1) == cxa.CXA_OK
    assert bool((out[73:] == 3).all()) and torch.equal(bt.cache.Kp, K0) and torch.equal(bt.cache.Vp, V0)
    bt.d["q_start"] = torch.tensor(bt.starts, dtype=torch.int32).cuda()
    bt.close(bt.attend())                                     # the workspace is as it was

    # 4096 sequences, every second one of all tokens: 3.2e9 chunks of 64 keys in tiles of 32 rows
    if act == "bf16":                                         # (items of 256 rows do not come to that many)
        return
    n, B = 32768, 4096
    c = cxa.PagedCache(256, 256, 1, 2, 64, act)
    q = torch.zeros(n, 2, 64, dtype=DT[act], device="cuda")
    out = torch.full_like(q, 3.0)
    starts = torch.tensor([0, n] * (B // 2) + [0], dtype=torch.int32).cuda()
    kv = torch.full((B,), 65536, dtype=torch.int32).cuda()
    table = torch.arange(256, dtype=torch.int32).cuda().expand(B, 256).contiguous()
    c.attend(0, q, starts, kv, table, max_new=n, out=out)
    assert cxa.cxa_device_status(1) == cxa.CXA_EINVAL
    assert bool((out == 3).all())


def test_chunks_on_streams_and_in_graphs_at_once():
    """The two kernels of a call on several streams, eager and replayed, each with its own scratch."""
    bts = [Batch([200, 1, 33], [9000, 3000, 500], 64, 5, 1, dh, "bf16", "bf16", seed=s).fill() for s, dh in ((1, 64), (2, 128))]
    want = [bt.attend() for bt in bts]
    qs = [bt.q.cuda() for bt in bts]
    call = lambda i, **kw: bts[i].cache.attend(0, qs[i], **bts[i].d, max_new=200, **kw)
    graphs, outs = [], []
    for i in (0, 1):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs += [(i, call(i)) for _ in range(3)]
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(8):
        for i in (0, 1):
            with torch.cuda.stream(streams[i]):
                graphs[i].replay()
            with torch.cuda.stream(streams[2 + i]):
                outs.append((i, call(i)))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i, o in outs)


@pytest.mark.parametrize("act,pool", TYPES)
@pytest.mark.parametrize("n", [1, 7, 90])
def test_sequences_share_the_pages_of_a_prefix(act, pool, n):
    """Three sequences whose tables begin with the same pages; their own pages follow."""
    page, prefix, own = 16, 160, [0, 33, 100]
    bt = Batch([n] * 3, [prefix + n + x for x in own], page, 4, 2, 64, act, pool)
    for b in (1, 2):
        bt.K[b][:prefix], bt.V[b][:prefix] = bt.K[0][:prefix], bt.V[0][:prefix]
        bt.table[b, :prefix // page] = bt.table[0, :prefix // page]
    bt.d["page_table"] = bt.table.cuda()
    bt.fill()
    bt.cache.check(bt.d["q_start"].cpu(), bt.d["kv_len"].cpu(), bt.table, bt.N)
    bt.close(bt.attend())
