"""Measured cases of the paged self-attention operators: head norms with the position
rotation, the append to a paged K/V cache, and the attention of new tokens over it.

Every case is one layer's call in a decoder that serves a batch of sequences. The pool of
pages is [layers][pages][kv heads][page size][head dim]; the new tokens of all sequences
are packed, sequence b owning rows q_start[b] .. q_start[b+1], the last of them at
position kv_len[b] - 1.

With ``own`` false, ``run`` computes an operator by elementary torch operations in 32 bits
(angles in 64); with ``own`` true it makes the package's calls.
"""
import math
import random

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


# ------------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one sequence on its way into the self-attention: latency
        dict(name="rope_token", op="rope", N=1, Hq=20, Hk=20, dh=64, act="bf16", rot=64, layout="half",
             scaling="none", norm=True, far=448),
        # every frame of 16 windows of up to 1500 frames through an encoder layer's rotation
        dict(name="rope_window", op="rope", N=24000, Hq=20, Hk=20, dh=64, act="bf16", rot=64, layout="half",
             scaling="none", norm=True, far=1500),
        # half of each head rotated, far positions, interleaved pairs, fp32, an odd token count
        dict(name="rope_partial", op="rope", N=5333, Hq=8, Hk=2, dh=64, act="f32", rot=32, layout="interleaved",
             scaling="wavelength", norm=False, far=1000000),
        # a decoding step of 16 sequences: one row each
        dict(name="append_step", op="append", B=16, new="one", total=16, kv=1500, Hq=8, Hkv=8, dh=64, page=16,
             act="bf16", pool="bf16", rot=64, layout="half", scaling="none", norm=True, with_q=True, lens_seed=11),
        # ragged prompts of 64 sequences admitted at once, queries and keys normalised and rotated
        dict(name="append_prompts", op="append", B=64, new="ragged", total=16391, kv=1024, Hq=32, Hkv=8, dh=128,
             page=64, act="bf16", pool="bf16", rot=128, layout="half", scaling="ntk", norm=True, with_q=True,
             lens_seed=12),
        # fp32 activations rounded into a bf16 pool, partial interleaved rotation, keys only
        dict(name="append_odd", op="append", B=5, new="ragged", total=1237, kv=4097, Hq=6, Hkv=6, dh=64, page=32,
             act="f32", pool="bf16", rot=48, layout="interleaved", scaling="linear", norm=False, with_q=False,
             lens_seed=13),
        # one token of one sequence over a decoder's full window: latency
        dict(name="attend_token", op="attend", B=1, new="one", total=1, kv=448, Hq=8, Hkv=8, dh=64, page=16,
             act="bf16", pool="bf16", lens_seed=21),
        # a serving batch of single tokens with shared key heads over ragged contexts
        dict(name="attend_batch", op="attend", B=64, new="one", total=64, kv=8192, Hq=32, Hkv=8, dh=128, page=64,
             act="bf16", pool="bf16", lens_seed=22),
        # five proposed tokens a sequence checked at once, fp32 throughout
        dict(name="attend_verify", op="attend", B=16, new="even", total=80, kv=1500, Hq=20, Hkv=20, dh=64, page=16,
             act="f32", pool="f32", lens_seed=23),
        # one token over one very long context
        dict(name="attend_long", op="attend", B=1, new="one", total=1, kv=262144, Hq=32, Hkv=4, dh=64, page=128,
             act="bf16", pool="bf16", lens_seed=24),
        # chunks of prompts beside sequences that decode, in one batch
        dict(name="attend_mixed", op="attend", B=24, new="mixed", total=2071, kv=8191, Hq=20, Hkv=20, dh=64, page=64,
             act="bf16", pool="bf16", lens_seed=25),
        # a chunk of a long prompt over what is cached of it
        dict(name="attend_chunk", op="attend", B=1, new="even", total=2048, kv=32768, Hq=20, Hkv=20, dh=64, page=128,
             act="bf16", pool="bf16", lens_seed=26),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "attend"])
    dh = rng.choice([64, 64, 128])
    rotary = dict(rot=rng.choice([dh, dh, dh // 2, 2 * rng.randint(1, dh // 2)]),
                  layout=rng.choice(["half", "interleaved"]),
                  scaling=rng.choice(["none", "linear", "ntk", "wavelength"]), norm=rng.random() < 0.5)
    if op == "rope":
        return dict(op=op, N=_log_int(rng, 1, 16000), Hq=rng.choice([1, 6, 8, 20, 32]), Hk=rng.choice([0, 1, 2, 8, 20]),
                    dh=dh, act=rng.choice(["bf16", "bf16", "f32"]), far=_log_int(rng, 16, 2000000), **rotary) \
            if dh == 64 else \
            dict(op=op, N=_log_int(rng, 1, 8000), Hq=rng.choice([1, 8, 20, 32]), Hk=rng.choice([0, 1, 2, 8]),
                 dh=dh, act=rng.choice(["bf16", "bf16", "f32"]), far=_log_int(rng, 16, 2000000), **rotary)
    act, pool = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
    Hkv = rng.choice([1, 2, 4, 6, 8, 20])
    G = rng.choice([1, 1, 2, 4, 5, 8]) if Hkv <= 8 else 1
    page = rng.choice([16, 32, 64, 128, 256])
    B = _log_int(rng, 1, 64)
    case = dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, dh=dh, page=page, act=act, pool=pool,
                lens_seed=rng.randrange(1 << 30))
    if op == "append":
        new = rng.choice(["one", "even", "ragged", "mixed"])
        case.update(new=new, total=B if new == "one" else max(B, _log_int(rng, 1, 12000)), kv=_log_int(rng, 1, 4096),
                    with_q=rng.random() < 0.6, **rotary)
        return case
    new = rng.choice(["one", "one", "even", "ragged", "mixed"])
    case.update(new=new, kv=_log_int(rng, 1, 65536), total=B if new == "one" else max(B, _log_int(rng, 1, 4096)))
    # no dearer than the largest listed cases of its kind
    while work(case)["flops"] > (3e11 if act == "bf16" else 1e10) or work(case)["bytes"] > 1e9:
        case["kv"] = max(1, case["kv"] * 2 // 3)
        if new != "one":
            case["total"] = max(B, case["total"] * 3 // 4)
        elif case["kv"] == 1:
            break
    return case


def _lengths(case):
    """New tokens and total keys of each sequence, from the case alone."""
    rng = random.Random(case["lens_seed"])
    B, total, new = case["B"], case["total"], case["new"]
    if new == "one":
        n = [1] * B
    elif new == "even":
        n = [total // B] * B
    elif new == "mixed":   # one sequence in six brings a chunk, the others one token
        big = [b for b in range(B) if b % 6 == 0]
        n = [1] * B
        rest = max(total - B, 0)
        for i, b in enumerate(big):
            n[b] += rest // len(big) + (1 if i < rest % len(big) else 0)
    else:                  # ragged, some sequences with nothing new
        w = [rng.random() ** 2 if rng.random() > 0.1 else 0.0 for _ in range(B)]
        s = sum(w) or 1.0
        n = [int(total * x / s) for x in w]
        n[B - 1] += max(0, total - sum(n))
    kv = []
    for b in range(B):
        past = max(0, case["kv"] - n[b])
        kv.append(n[b] + (past if B == 1 else rng.randint(past // 8, past)))
    return n, kv


def work(case):
    dh = case["dh"]
    ea = 2 if case["act"] == "bf16" else 4
    if case["op"] == "rope":
        el = case["N"] * (case["Hq"] + case["Hk"]) * dh
        return {"bytes": 2 * el * ea + 4 * case["N"], "flops": 6 * el}
    ep = 2 if case["pool"] == "bf16" else 4
    n, kv = _lengths(case)
    N = sum(n)
    meta = 4 * (2 * case["B"] + 1)
    if case["op"] == "append":
        rows = N * case["Hkv"] * dh
        q = N * case["Hq"] * dh if case["with_q"] else 0
        return {"bytes": 2 * rows * (ea + ep) + 2 * q * ea + meta, "flops": 6 * (rows + q)}
    pairs = sum(a * k - a * (a - 1) // 2 for a, k in zip(n, kv))
    pages = sum(-(-k // case["page"]) for a, k in zip(n, kv) if a)
    keys = sum(k for a, k in zip(n, kv) if a)
    return {"bytes": 2 * keys * case["Hkv"] * dh * ep + 2 * N * case["Hq"] * dh * ea + 4 * pages + meta,
            "flops": 4 * dh * case["Hq"] * pairs}


# ------------------------------------------------------------------------- inputs
_BASE, _FACTOR, _ORIG, _ALPHA, _BETA = 10000.0, 8.0, 4096, 1.0, 32.0


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 7)
    dh, act = case["dh"], _DT[case["act"]]

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    s = {"case": case}
    if case["op"] == "rope":
        N = case["N"]
        # q and k are slices of one projection's rows, as a fused projection leaves them
        qkv = randn(N, (case["Hq"] + 2 * case["Hk"]) * dh, dtype=act)
        s["q"] = qkv[:, :case["Hq"] * dh].unflatten(1, (case["Hq"], dh))
        s["k"] = qkv[:, case["Hq"] * dh:(case["Hq"] + case["Hk"]) * dh].unflatten(1, (case["Hk"], dh)) \
            if case["Hk"] else None
        s["pos"] = torch.randint(0, case["far"], (N,), generator=g, device="cuda", dtype=torch.int32)
    else:
        n, kv = _lengths(case)
        B, page, Hq, Hkv = case["B"], case["page"], case["Hq"], case["Hkv"]
        N = sum(n)
        need = [-(-k // page) for k in kv]
        pages = sum(need) + 3
        width = max(need) + 1
        perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b in range(B):
            table[b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
        starts = [0]
        for x in n:
            starts.append(starts[-1] + x)
        s.update(n=n, kv=kv, starts=starts, table=table,
                 q_start=torch.tensor(starts, dtype=torch.int32, device="cuda"),
                 kv_len=torch.tensor(kv, dtype=torch.int32, device="cuda"))
        layers = 2 if case["op"] == "append" else 1
        shape = (layers, pages, Hkv, page, dh)
        s["layer"] = layers - 1
        s["Kp"], s["Vp"] = randn(*shape, dtype=_DT[case["pool"]]), randn(*shape, dtype=_DT[case["pool"]])
        if case["op"] == "append":
            qkv = randn(N, (Hq + 2 * Hkv) * dh, dtype=act)
            s["q"] = qkv[:, :Hq * dh].unflatten(1, (Hq, dh)) if case["with_q"] else None
            s["k"] = qkv[:, Hq * dh:(Hq + Hkv) * dh].unflatten(1, (Hkv, dh))
            s["v"] = qkv[:, (Hq + Hkv) * dh:].unflatten(1, (Hkv, dh))
        else:
            s["q"] = randn(N, Hq, dh, dtype=act)
    if "rot" in case:
        s["wq"] = 1.0 + randn(dh, scale=0.1) if case["norm"] else None
        s["wk"] = 1.0 + randn(dh, scale=0.1) if case["norm"] else None
        s["eps"] = 1e-6 if case["norm"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if "rot" in case:
        freq, factor = _frequencies(case["rot"], case["scaling"])
        s["freq"], s["mscale"] = torch.tensor(freq, dtype=torch.float64, device="cuda"), factor
    if s["q"] is not None:
        s["q_out"] = torch.empty_like(s["q"], memory_format=torch.contiguous_format)
    if case["op"] == "rope" and s["k"] is not None:
        s["k_out"] = torch.empty_like(s["k"], memory_format=torch.contiguous_format)
    if own:
        from encoder_decoder_speech_gb300 import cxa
        if "rot" in case:
            s["rotary"] = cxa.Rotary(case["rot"], base=_BASE, layout=case["layout"], scaling=case["scaling"],
                                     factor=_FACTOR, orig_len=_ORIG, alpha=_ALPHA, beta=_BETA)
        if "page" in case:
            layers, pages, Hkv, page, dh = s["Kp"].shape
            cache = cxa.PagedCache(pages, page, layers, Hkv, dh, case["pool"])
            cache.Kp.copy_(s["Kp"])
            cache.Vp.copy_(s["Vp"])
            s["Kp"], s["Vp"], s["cache"] = cache.Kp, cache.Vp, cache
    return s


# ------------------------------------------------------------------------- plain forms
def _frequencies(rot, scaling):
    """Radians per position of each rotated pair, and the factor of the rotated values."""
    base = _BASE
    if scaling == "ntk":
        base = _BASE * _FACTOR ** (rot / (rot - 2)) if rot > 2 else _BASE
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        f = [x / _FACTOR for x in f]
    if scaling != "wavelength":
        return f, 1.0
    out = []
    for x in f:
        turns = _ORIG * x / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - _ALPHA) / (_BETA - _ALPHA)))
        out.append(x * keep + x / _FACTOR * (1.0 - keep))
    return out, 0.1 * math.log(_FACTOR) + 1.0


def _norm_rotate(x, pos, s, w):
    """x [N, H, dh] in its own type -> fp32, normalised and rotated."""
    case = s["case"]
    y = x.float()
    if s["eps"] is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * w
    rot = case["rot"]
    ang = pos.double()[:, None] * s["freq"][None, :]
    cos = (torch.cos(ang) * s["mscale"]).float()[:, None, :]
    sin = (torch.sin(ang) * s["mscale"]).float()[:, None, :]
    y = y.clone()
    if case["layout"] == "half":
        a, b = y[..., :rot // 2].clone(), y[..., rot // 2:rot].clone()
        y[..., :rot // 2] = a * cos - b * sin
        y[..., rot // 2:rot] = a * sin + b * cos
    else:
        a, b = y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = a * sin + b * cos
    return y


def _positions(s):
    return torch.cat([torch.arange(k - a, k, device="cuda") for a, k in zip(s["n"], s["kv"])])


def _plain_append(s):
    case, layer, page = s["case"], s["layer"], s["case"]["page"]
    pos = _positions(s)
    seq = torch.cat([torch.full((a,), b, dtype=torch.int64, device="cuda") for b, a in enumerate(s["n"])])
    where = s["table"][seq, pos // page].long()
    slot = pos % page
    s["Kp"][layer][where, :, slot] = _norm_rotate(s["k"], pos, s, s["wk"]).to(s["Kp"].dtype)
    s["Vp"][layer][where, :, slot] = s["v"].to(s["Vp"].dtype)
    if s["q"] is None:
        return s["Kp"], s["Vp"]
    s["q_out"].copy_(_norm_rotate(s["q"], pos, s, s["wq"]))
    return s["Kp"], s["Vp"], s["q_out"]


def _plain_attend(s):
    case, layer, page = s["case"], s["layer"], s["case"]["page"]
    Hq, Hkv, dh = case["Hq"], case["Hkv"], case["dh"]
    G = Hq // Hkv
    for b, (n, kv) in enumerate(zip(s["n"], s["kv"])):
        if n == 0:
            continue
        rows = slice(s["starts"][b], s["starts"][b + 1])
        ids = s["table"][b, :-(-kv // page)].long()
        K = s["Kp"][layer][ids].permute(1, 0, 2, 3).reshape(Hkv, -1, dh)[:, :kv].float()
        V = s["Vp"][layer][ids].permute(1, 0, 2, 3).reshape(Hkv, -1, dh)[:, :kv].float()
        q = s["q"][rows].float().reshape(n, Hkv, G, dh).permute(1, 2, 0, 3).reshape(Hkv, G * n, dh)
        hidden = torch.arange(kv, device="cuda")[None, :] > torch.arange(kv - n, kv, device="cuda").repeat(G)[:, None]
        o = torch.empty(Hkv, G * n, dh, device="cuda")
        step = max(1, int(5e8 // (G * n * kv)))
        for h in range(0, Hkv, step):   # a few heads at a time: the scores of all would not fit in earnest
            sc = (q[h:h + step] @ K[h:h + step].transpose(1, 2)) * (1.0 / math.sqrt(dh))
            sc = sc.masked_fill(hidden, float("-inf"))
            p = torch.exp(sc - sc.amax(-1, keepdim=True))
            o[h:h + step] = (p @ V[h:h + step]) / p.sum(-1, keepdim=True)
        s["q_out"][rows] = o.reshape(Hkv, G, n, dh).permute(2, 0, 1, 3).reshape(n, Hq, dh).to(s["q_out"].dtype)
    return s["q_out"]


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        if op == "append":
            return _plain_append(s)
        if op == "attend":
            return _plain_attend(s)
        s["q_out"].copy_(_norm_rotate(s["q"], s["pos"], s, s["wq"]))
        if s["k"] is None:
            return (s["q_out"],)
        s["k_out"].copy_(_norm_rotate(s["k"], s["pos"], s, s["wk"]))
        return s["q_out"], s["k_out"]
    if op == "attend":
        return s["cache"].attend(s["layer"], s["q"], s["q_start"], s["kv_len"], s["table"], max_new=max(s["n"]),
                                 out=s["q_out"])
    if op == "append":
        s["cache"].append(s["layer"], s["k"], s["v"], s["q_start"], s["kv_len"], s["table"], q=s["q"],
                          q_out=s.get("q_out"), rotary=s["rotary"], norm_eps=s["eps"], q_weight=s["wq"],
                          k_weight=s["wk"])
        return (s["Kp"], s["Vp"]) if s["q"] is None else (s["Kp"], s["Vp"], s["q_out"])
    from encoder_decoder_speech_gb300 import cxa
    q_out, k_out = cxa.qk_norm_rope(s["q"], s["k"], s["pos"], rotary=s["rotary"], norm_eps=s["eps"],
                                    q_weight=s["wq"], k_weight=s["wk"], q_out=s["q_out"], k_out=s.get("k_out"))
    return (q_out,) if s["k"] is None else (q_out, k_out)


# ------------------------------------------------------------------------- the definition in 64 bits
def _turned(x, positions, case, weight, eps):
    """One head vector after another by the definition: x / rms(x) * w, then each pair's
    complex number times m * exp(i * position * frequency)."""
    z = x.to(torch.float64)
    if eps is not None:
        z = weight.to(torch.float64) * z / torch.sqrt(z.pow(2).sum(-1, keepdim=True) / z.shape[-1] + eps)
    rot, pairs = case["rot"], case["rot"] // 2
    exponent = torch.arange(pairs, dtype=torch.float64, device=z.device) * 2.0 / rot
    if case["scaling"] == "ntk" and rot > 2:
        theta = torch.exp(-exponent * (math.log(_BASE) + math.log(_FACTOR) * rot / (rot - 2)))
    else:
        theta = torch.exp(-exponent * math.log(_BASE))
    m = 1.0
    if case["scaling"] == "linear":
        theta = theta / _FACTOR
    elif case["scaling"] == "wavelength":
        wavelength = 2 * math.pi / theta
        gamma = ((_ORIG / wavelength - _ALPHA) / (_BETA - _ALPHA)).clamp(0.0, 1.0)
        theta = (1 - gamma) * theta / _FACTOR + gamma * theta
        m = 1.0 + 0.1 * math.log(_FACTOR)
    spin = torch.polar(torch.full((len(positions), pairs), m, dtype=torch.float64, device=z.device),
                       positions.to(torch.float64)[:, None] * theta)[:, None, :]
    head, rest = z[..., :rot], z[..., rot:]
    if case["layout"] == "half":
        c = torch.complex(head[..., :pairs].contiguous(), head[..., pairs:].contiguous()) * spin
        head = torch.cat([c.real, c.imag], -1)
    else:
        c = torch.view_as_complex(head.reshape(*head.shape[:-1], pairs, 2).contiguous()) * spin
        head = torch.view_as_real(c).reshape(head.shape)
    return torch.cat([head, rest], -1)


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "rope":
        out = [_turned(s["q"], s["pos"], case, s["wq"], s["eps"])]
        if s["k"] is not None:
            out.append(_turned(s["k"], s["pos"], case, s["wk"], s["eps"]))
        return tuple(out)
    if case["op"] == "append":
        K, V = s["Kp"].double(), s["Vp"].double()
        at = torch.cat([torch.arange(s["kv"][b] - s["n"][b], s["kv"][b], device="cuda") for b in range(case["B"])])
        k = _turned(s["k"], at, case, s["wk"], s["eps"])
        for b in range(case["B"]):
            lo, hi = s["starts"][b], s["starts"][b + 1]
            first, done = s["kv"][b] - s["n"][b], 0
            while lo + done < hi:   # the run of rows that falls into one page
                t = first + done
                page, slot = int(s["table"][b, t // case["page"]]), t % case["page"]
                m = min(hi - lo - done, case["page"] - slot)
                K[s["layer"], page, :, slot:slot + m] = k[lo + done:lo + done + m].transpose(0, 1)
                V[s["layer"], page, :, slot:slot + m] = s["v"][lo + done:lo + done + m].double().transpose(0, 1)
                done += m
        if s["q"] is None:
            return K, V
        return K, V, _turned(s["q"], at, case, s["wq"], s["eps"])
    if work(case)["flops"] > 2e12:
        return None
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    G = case["Hq"] // case["Hkv"]
    for b in range(case["B"]):
        n, kv = s["n"][b], s["kv"][b]
        if n == 0:
            continue
        ids = [int(i) for i in s["table"][b].tolist()][:-(-kv // case["page"])]
        seen = torch.arange(kv, device="cuda")[None, :] <= torch.arange(kv - n, kv, device="cuda")[:, None]
        for h in range(case["Hkv"]):
            K = s["Kp"][0, ids, h].reshape(-1, case["dh"])[:kv].double()
            V = s["Vp"][0, ids, h].reshape(-1, case["dh"])[:kv].double()
            for r in range(h * G, (h + 1) * G):
                score = torch.einsum("id,jd->ij", s["q"][s["starts"][b]:s["starts"][b + 1], r].double(), K)
                score = torch.where(seen, score / math.sqrt(case["dh"]), -math.inf)
                out[s["starts"][b]:s["starts"][b + 1], r] = torch.softmax(score, -1) @ V
    return out
