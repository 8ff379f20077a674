"""Measured cases of what makes a long context's cache cheaper: the latent cache (one vector a
token that all heads share) with its append, its attention and its expansion into pages of
keys and values, and the eviction of tokens from paged keys and values by the attention weight
that they have gathered.

Every case is one call in a decoder that serves a batch of sequences, packed as elsewhere:
sequence b owns rows q_start[b] .. q_start[b+1] of the new tokens, the last of them at position
kv_len[b] - 1. Latent pages are [layers][pages][page size][latent + rope], pages of keys and of
values [layers][pages][kv heads][page size][head dim], gathered weights
[layers][pages][kv heads][page size].

With ``own`` false, ``run`` computes an operator by elementary torch operations in 32 bits
(angles in 64); with ``own`` true it makes the package's calls.
"""
import math
import random

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_BASE = 10000.0


# ------------------------------------------------------------------------- cases
def listed():
    return [
        # a decoding step of 16 sequences: one latent row each, normalised and rotated
        dict(name="latent_append_step", op="append", B=16, new="one", total=16, kv=1500, latent=256, rope=32,
             page=16, act="bf16", pool="bf16", layout="half", norm=True, lens_seed=31),
        # ragged prompts of 64 sequences admitted at once
        dict(name="latent_append_prompts", op="append", B=64, new="ragged", total=16391, kv=1024, latent=512, rope=64,
             page=64, act="bf16", pool="bf16", layout="interleaved", norm=True, lens_seed=32),
        # one token of one sequence over a decoder's full window, no rotated part: latency
        dict(name="latent_token", op="latent", B=1, new="one", total=1, kv=448, H=8, latent=256, rope=0, page=16,
             pool="bf16", lens_seed=41),
        # a serving batch of single tokens over ragged contexts
        dict(name="latent_batch", op="latent", B=64, new="one", total=64, kv=8192, H=20, latent=512, rope=64, page=64,
             pool="bf16", lens_seed=42),
        # one token with many heads over one very long context
        dict(name="latent_long", op="latent", B=1, new="one", total=1, kv=262144, H=64, latent=512, rope=64, page=128,
             pool="bf16", lens_seed=43),
        # five proposed tokens a sequence checked at once, fp32 throughout
        dict(name="latent_verify", op="latent", B=16, new="even", total=80, kv=1500, H=8, latent=128, rope=32, page=16,
             pool="f32", lens_seed=44),
        # short ragged contexts on their way into pages of keys and values, before their prompts' attention
        dict(name="expand_ragged", op="expand", B=24, kv=1500, H=8, dh=64, latent=256, rope=32, page=16, to_page=64,
             pool="bf16", lens_seed=51),
        # a long context expanded for the next chunk of its prompt
        dict(name="expand_long", op="expand", B=1, kv=32768, H=20, dh=128, latent=512, rope=64, page=128, to_page=128,
             pool="bf16", lens_seed=52),
        # the weights that a decoding step of 64 sequences adds, shared key heads, ragged contexts
        dict(name="weights_step", op="weights", B=64, new="one", total=64, kv=8192, Hq=32, Hkv=8, dh=128, page=64,
             pool="bf16", lens_seed=61),
        # the weights that a chunk of a prompt adds over what is cached of it
        dict(name="weights_prompt", op="weights", B=1, new="even", total=2048, kv=8192, Hq=20, Hkv=20, dh=64, page=128,
             pool="bf16", lens_seed=62),
        # every layer of a small decoder cut down to a quarter of its window
        dict(name="evict_window", op="evict", B=16, kv=448, L=6, Hkv=8, dh=64, page=16, pool="bf16", keep=112,
             first=4, recent=32, lens_seed=71),
        # long contexts cut down to an eighth
        dict(name="evict_long", op="evict", B=4, kv=65536, L=1, Hkv=8, dh=128, page=64, pool="bf16", keep=8192,
             first=4, recent=256, lens_seed=72),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "latent", "latent", "expand", "weights", "weights", "evict"])
    page = rng.choice([16, 32, 64, 128, 256])
    case = dict(op=op, B=_log_int(rng, 1, 64), page=page, lens_seed=rng.randrange(1 << 30))
    B = case["B"]
    if op in ("append", "latent", "expand"):
        case.update(latent=rng.choice([128, 256, 384, 512, 512]), rope=rng.choice([0, 16, 32, 64, 64]))
    if op == "append":
        act, pool = rng.choice([("bf16", "bf16"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
        new = rng.choice(["one", "even", "ragged", "mixed"])
        case.update(act=act, pool=pool, new=new, total=B if new == "one" else max(B, _log_int(rng, 1, 12000)),
                    kv=_log_int(rng, 1, 4096), layout=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.7)
        return case
    case["pool"] = rng.choice(["bf16", "bf16", "f32"])
    f32 = case["pool"] == "f32"
    if op == "expand":
        dh = rng.choice([64, 128])
        case.update(H=rng.choice([1, 6, 8, 20]), dh=dh, kv=_log_int(rng, 1, 32768), to_page=rng.choice([16, 64, 128, 256]))
        case["rope"] = min(case["rope"], dh - 16)
        while work(case)["flops"] > (1e11 if not f32 else 5e9) or work(case)["bytes"] > 4e8:
            case["kv"] = max(1, case["kv"] * 2 // 3)
            case["H"] = max(1, case["H"] * 3 // 4)
        return case
    if op == "evict":
        Hkv, L = rng.choice([1, 2, 6, 8, 20]), rng.choice([1, 1, 2, 6])
        kv = _log_int(rng, 1, 65536)
        keep = _log_int(rng, 1, 8192)
        first = rng.randint(0, keep // 8)
        case.update(kv=kv, L=L, Hkv=Hkv, dh=rng.choice([64, 128]), keep=keep, first=first,
                    recent=rng.randint(0, (keep - first) // 2))
        while case["B"] * case["kv"] * L * Hkv * case["dh"] > 2 ** 27 or work(case)["bytes"] > 3e8:
            case["B"] = max(1, case["B"] // 2)
            case["kv"] = max(1, case["kv"] * 2 // 3)
        return case
    new = rng.choice(["one", "one", "even", "ragged", "mixed"])
    case.update(new=new, kv=_log_int(rng, 1, 65536), total=B if new == "one" else max(B, _log_int(rng, 1, 2048)))
    if op == "latent":
        case["H"] = rng.choice([1, 4, 8, 16, 20, 32, 64, 128])
        most = 3e10 if not f32 else 3e9
    else:
        Hkv = rng.choice([1, 2, 4, 6, 8, 20])
        G = rng.choice([1, 1, 2, 4, 5, 8]) if Hkv <= 8 else 1
        case.update(Hq=G * Hkv, Hkv=Hkv, dh=rng.choice([64, 64, 128]))
        most = 3e10 if not f32 else 3e9
    while work(case)["flops"] > most or work(case)["bytes"] > 3e8:
        case["kv"] = max(1, case["kv"] * 2 // 3)
        if new != "one":
            case["total"] = max(B, case["total"] * 3 // 4)
        elif case["kv"] == 1:
            break
    return case


def _lengths(case):
    """New tokens and total keys of each sequence, from the case alone."""
    rng = random.Random(case["lens_seed"])
    B = case["B"]
    if "new" not in case:      # no new tokens in these calls
        return [0] * B, [case["kv"] if B == 1 else rng.randint(case["kv"] // 4 + 1, case["kv"]) if case["kv"] > 1 else 1
                         for _ in range(B)]
    total, new = case["total"], case["new"]
    if new == "one":
        n = [1] * B
    elif new == "even":
        n = [total // B] * B
    elif new == "mixed":       # one sequence in six brings a chunk, the others one token
        big = [b for b in range(B) if b % 6 == 0]
        n = [1] * B
        rest = max(total - B, 0)
        for i, b in enumerate(big):
            n[b] += rest // len(big) + (1 if i < rest % len(big) else 0)
    else:                      # ragged, some sequences with nothing new
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
    n, kv = _lengths(case)
    B, N, ep = case["B"], sum(n), 2 if case["pool"] == "bf16" else 4
    op, page = case["op"], case["page"]
    meta = 4 * (2 * B + 1)
    if op == "append":
        el, ea = N * (case["latent"] + case["rope"]), 2 if case["act"] == "bf16" else 4
        return {"bytes": el * (ea + ep) + meta, "flops": 5 * el}
    if op == "expand":
        dc, dr, H, dh, keys = case["latent"], case["rope"], case["H"], case["dh"], sum(kv)
        cols = H * (2 * dh - dr)
        return {"bytes": ep * (keys * (dc + dr) + dc * cols + keys * H * 2 * dh) + 4 * sum(-(-k // page) for k in kv),
                "flops": 2 * keys * dc * cols}
    if op == "evict":
        rows = case["L"] * case["Hkv"]
        kept = sum(min(k, case["keep"]) for k in kv)
        return {"bytes": rows * (4 * sum(kv) + kept * (4 * case["dh"] * ep + 4 + 4)) + meta, "flops": rows * sum(kv)}
    pairs = sum(a * k - a * (a - 1) // 2 for a, k in zip(n, kv))
    pages = sum(-(-k // page) for a, k in zip(n, kv) if a)
    keys = sum(k for a, k in zip(n, kv) if a)
    if op == "latent":
        dc, dr, H = case["latent"], case["rope"], case["H"]
        return {"bytes": ep * (keys * (dc + dr) + N * H * (2 * dc + dr)) + 4 * pages + meta,
                "flops": 2 * H * (2 * dc + dr) * pairs}
    dh, Hkv = case["dh"], case["Hkv"]
    return {"bytes": keys * Hkv * (dh * ep + 8) + N * case["Hq"] * dh * ep + 4 * pages + meta,
            "flops": 2 * dh * case["Hq"] * pairs}


# ------------------------------------------------------------------------- inputs
def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 11)
    op, B, page, dt = case["op"], case["B"], case["page"], _DT[case["pool"]]
    n, kv = _lengths(case)
    N = sum(n)

    def randn(*shape, dtype=torch.float32, scale=1.0):
        out = torch.empty(*shape, device="cuda", dtype=dtype)
        flat = out.view(-1)
        for at in range(0, flat.numel(), 1 << 28):      # a quarter of a GB of fp32 numbers at a time
            m = min(1 << 28, flat.numel() - at)
            flat[at:at + m] = torch.randn(m, generator=g, device="cuda") * scale
        return out

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def tables(lens, page, spare):
        """Pages in no order, some of the pool's unused."""
        need = [-(-k // page) for k in lens]
        perm = torch.randperm(sum(need) + spare, generator=g, device="cuda").to(torch.int32)
        table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, m in enumerate(need):
            table[b, :m] = perm[at:at + m]
            at += m
        return table

    starts = [0]
    for x in n:
        starts.append(starts[-1] + x)
    s = dict(case=case, n=n, kv=kv, starts=starts, q_start=ints(starts), kv_len=ints(kv))
    if op == "evict":
        # the destination's pages are other pages of the pool
        need = [-(-k // page) for k in kv]
        out = [min(k, case["keep"]) for k in kv]
        need_out = [-(-k // page) for k in out]
        pages = sum(need) + sum(need_out) + 3
        perm = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        s["table"] = torch.full((B, max(need) + 1), -1, dtype=torch.int32, device="cuda")
        s["to_table"] = torch.full((B, max(need_out)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b in range(B):
            s["table"][b, :need[b]] = perm[at:at + need[b]]
            at += need[b]
            s["to_table"][b, :need_out[b]] = perm[at:at + need_out[b]]
            at += need_out[b]
        shape = (case["L"], pages, case["Hkv"], page)
        s["Kp"], s["Vp"] = randn(*shape, case["dh"], dtype=dt), randn(*shape, case["dh"], dtype=dt)
        # sums of weights: a few tokens hold most of it, and some (unused) tie at nothing
        w = torch.exp(3.0 * torch.randn(*shape, generator=g, device="cuda") - 5.0)
        s["Wp"] = torch.where(torch.rand(*shape, generator=g, device="cuda") < 0.1, torch.zeros_like(w), w)
        return s
    s["table"] = tables(kv, page, 3)
    pages = sum(-(-k // page) for k in kv) + 3
    if op in ("append", "latent", "expand"):
        width = case["latent"] + case["rope"]
        layers = 2 if op == "append" else 1
        s["layer"] = layers - 1
        s["Cp"] = randn(layers, pages, page, width, dtype=dt)
        if op == "append":
            # c and kr are slices of one projection's rows
            row = randn(N, width, dtype=_DT[case["act"]])
            s["c"], s["kr"] = row[:, :case["latent"]], row[:, case["latent"]:] if case["rope"] else None
            s["w"] = 1.0 + randn(case["latent"], scale=0.1) if case["norm"] else None
            s["eps"] = 1e-6 if case["norm"] else None
        elif op == "latent":
            s["q"] = randn(N, case["H"], width, dtype=dt)
            # as for scores of unit variance in front of the softmax
            s["scale"] = 1.0 / math.sqrt(width)
        else:
            H, dh, dr, dc = case["H"], case["dh"], case["rope"], case["latent"]
            s["WK"] = randn(dc, H * (dh - dr), dtype=dt, scale=dc ** -0.5)
            s["WV"] = randn(dc, H * dh, dtype=dt, scale=dc ** -0.5)
            s["to_table"] = tables(kv, case["to_page"], 2)
            to_pages = sum(-(-k // case["to_page"]) for k in kv) + 2
            s["to_shape"] = (1, to_pages, H, case["to_page"], dh)
    else:
        shape = (1, pages, case["Hkv"], page)
        s["layer"] = 0
        s["Kp"] = randn(*shape, case["dh"], dtype=dt)
        s["Wp"] = torch.rand(*shape, generator=g, device="cuda")
        s["q"] = randn(N, case["Hq"], case["dh"], dtype=dt)
        s["decay"] = 1.0
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op, page, dt = case["op"], case["page"], _DT[case["pool"]]
    if op == "latent":
        s["out"] = torch.empty(sum(s["n"]), case["H"], case["latent"], dtype=dt, device="cuda")
    if op == "expand":
        s["Kp"], s["Vp"] = (torch.zeros(s["to_shape"], dtype=dt, device="cuda") for _ in range(2))
    if op == "evict":
        s["kept"] = torch.empty(case["L"], case["B"], case["Hkv"], case["keep"], dtype=torch.int32, device="cuda")
        s["out_len"] = torch.empty(case["B"], dtype=torch.int32, device="cuda")
    if not own:
        return s
    from encoder_decoder_speech_gb300 import cxa
    if op in ("append", "latent", "expand"):
        layers, pages = s["Cp"].shape[:2]
        cache = cxa.LatentCache(pages, page, layers, case["latent"], case["rope"], case["pool"])
        cache.Cp.copy_(s["Cp"])
        s["Cp"], s["cache"] = cache.Cp, cache
        if op == "append" and case["rope"]:
            s["rotary"] = cxa.Rotary(case["rope"], base=_BASE, layout=case["layout"])
        if op == "expand":
            to = cxa.PagedCache(s["to_shape"][1], case["to_page"], 1, case["H"], case["dh"], case["pool"])
            s["to"], s["Kp"], s["Vp"] = to, to.Kp, to.Vp
    else:
        layers, pages, Hkv, _, dh = s["Kp"].shape
        cache = cxa.PagedCache(pages, page, layers, Hkv, dh, case["pool"])
        cache.Kp.copy_(s["Kp"])
        if op == "evict":
            cache.Vp.copy_(s["Vp"])
        s["Kp"], s["Vp"], s["cache"] = cache.Kp, cache.Vp, cache
    return s


# ------------------------------------------------------------------------- plain forms
def _plain_append(s):
    case, layer, page, dc, dr = s["case"], s["layer"], s["case"]["page"], s["case"]["latent"], s["case"]["rope"]
    pos = torch.cat([torch.arange(k - a, k, device="cuda") for a, k in zip(s["n"], s["kv"])])
    seq = torch.cat([torch.full((a,), b, dtype=torch.int64, device="cuda") for b, a in enumerate(s["n"])])
    c = s["c"].float()
    if s["eps"] is not None:
        c = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + s["eps"]) * s["w"]
    row = c
    if dr:
        freq = _BASE ** (-2.0 * torch.arange(dr // 2, dtype=torch.float64, device="cuda") / dr)
        ang = pos.double()[:, None] * freq
        cos, sin = torch.cos(ang).float(), torch.sin(ang).float()
        kr = s["kr"].float()
        out = torch.empty_like(kr)
        if case["layout"] == "half":
            a, b = kr[:, :dr // 2], kr[:, dr // 2:]
            out[:, :dr // 2], out[:, dr // 2:] = a * cos - b * sin, a * sin + b * cos
        else:
            a, b = kr[:, 0::2], kr[:, 1::2]
            out[:, 0::2], out[:, 1::2] = a * cos - b * sin, a * sin + b * cos
        row = torch.cat([c, out], 1)
    s["Cp"][layer][s["table"][seq, pos // page].long(), pos % page] = row.to(s["Cp"].dtype)
    return s["Cp"]


def _hidden(n, kv):
    return torch.arange(kv, device="cuda")[None, :] > torch.arange(kv - n, kv, device="cuda")[:, None]


def _plain_latent(s):
    case, page, dc, H = s["case"], s["case"]["page"], s["case"]["latent"], s["case"]["H"]
    for b, (n, kv) in enumerate(zip(s["n"], s["kv"])):
        if n == 0:
            continue
        rows = slice(s["starts"][b], s["starts"][b + 1])
        C = s["Cp"][s["layer"]][s["table"][b, :-(-kv // page)].long()].flatten(0, 1)[:kv].float()
        q = s["q"][rows].float()
        hidden = _hidden(n, kv)[:, None, :]
        step = max(1, int(2e8 // (H * kv)))
        o = torch.empty(n, H, dc, device="cuda")
        for i in range(0, n, step):
            sc = (q[i:i + step] @ C.T) * s["scale"]
            sc = sc.masked_fill(hidden[i:i + step], float("-inf"))
            p = torch.exp(sc - sc.amax(-1, keepdim=True))
            o[i:i + step] = (p @ C[:, :dc]) / p.sum(-1, keepdim=True)
        s["out"][rows] = o.to(s["out"].dtype)
    return s["out"]


def _plain_expand(s):
    case, page, to_page = s["case"], s["case"]["page"], s["case"]["to_page"]
    dc, dr, H, dh = case["latent"], case["rope"], case["H"], case["dh"]
    WK, WV = s["WK"].float(), s["WV"].float()
    for b, kv in enumerate(s["kv"]):
        C = s["Cp"][s["layer"]][s["table"][b, :-(-kv // page)].long()].flatten(0, 1)[:kv].float()
        k = (C[:, :dc] @ WK).view(kv, H, dh - dr)
        k = torch.cat([C[:, None, dc:].expand(kv, H, dr), k], -1)
        v = (C[:, :dc] @ WV).view(kv, H, dh)
        at = torch.arange(kv, device="cuda")
        where, slot = s["to_table"][b][at // to_page].long(), at % to_page
        s["Kp"][0][where, :, slot] = k.to(s["Kp"].dtype)
        s["Vp"][0][where, :, slot] = v.to(s["Vp"].dtype)
    return s["Kp"], s["Vp"]


def _plain_weights(s):
    case, page, layer = s["case"], s["case"]["page"], s["layer"]
    Hq, Hkv, dh = case["Hq"], case["Hkv"], case["dh"]
    G = Hq // Hkv
    for b, (n, kv) in enumerate(zip(s["n"], s["kv"])):
        if n == 0:
            continue
        ids = s["table"][b, :-(-kv // page)].long()
        K = s["Kp"][layer][ids].permute(1, 0, 2, 3).reshape(Hkv, -1, dh)[:, :kv].float()
        q = s["q"][s["starts"][b]:s["starts"][b + 1]].float().reshape(n, Hkv, G, dh).permute(1, 2, 0, 3)
        q = q.reshape(Hkv, G * n, dh)
        hidden = _hidden(n, kv).repeat(G, 1)
        add = torch.empty(Hkv, kv, device="cuda")
        step = max(1, int(2e8 // (G * n * kv)))
        for h in range(0, Hkv, step):
            sc = (q[h:h + step] @ K[h:h + step].transpose(1, 2)) * (1.0 / math.sqrt(dh))
            sc = sc.masked_fill(hidden, float("-inf"))
            p = torch.exp(sc - sc.amax(-1, keepdim=True))
            add[h:h + step] = (p / p.sum(-1, keepdim=True)).sum(1)
        at = torch.arange(kv, device="cuda")
        where, slot = ids[at // page], at % page
        old = s["Wp"][layer][where, :, slot] * s["decay"]
        old[kv - n:] = 0.0
        s["Wp"][layer][where, :, slot] = old + add.T
    return s["Wp"]


def _plain_evict(s):
    case, page = s["case"], s["case"]["page"]
    first, recent = case["first"], case["recent"]
    s["kept"].fill_(-1)
    for b, kv in enumerate(s["kv"]):
        m = min(kv, case["keep"])
        at = torch.arange(kv, device="cuda")
        where, slot = s["table"][b][at // page].long(), at % page
        w = s["Wp"][:, where, :, slot].permute(1, 2, 0)                  # [layers, heads, keys]
        w = torch.where((at < first) | (at >= kv - recent), float("inf"), w)
        keep = torch.sort(torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :m], dim=-1).values
        s["kept"][:, b, :, :m] = keep.int()
        to = torch.arange(m, device="cuda")
        to_where, to_slot = s["to_table"][b][to // page].long(), to % page
        layer = torch.arange(case["L"], device="cuda")[:, None, None]
        head = torch.arange(case["Hkv"], device="cuda")[None, :, None]
        for pool in (s["Kp"], s["Vp"], s["Wp"]):
            pool[layer, to_where, head, to_slot] = pool[layer, where[keep], head, slot[keep]]
        s["out_len"][b] = m
    return s["Kp"], s["Vp"], s["Wp"], s["kept"], s["out_len"]


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return {"append": _plain_append, "latent": _plain_latent, "expand": _plain_expand, "weights": _plain_weights,
                "evict": _plain_evict}[op](s)
    cache = s["cache"]
    if op == "append":
        cache.append(s["layer"], s["c"], s["kr"], s["q_start"], s["kv_len"], s["table"], rotary=s.get("rotary"),
                     norm_eps=s["eps"], weight=s["w"])
        return s["Cp"]
    if op == "latent":
        return cache.attend(s["layer"], s["q"], s["q_start"], s["kv_len"], s["table"], max_new=max(s["n"]),
                            scale=s["scale"], out=s["out"])
    if op == "expand":
        cache.expand(s["layer"], s["WK"], s["WV"], s["kv_len"], s["table"], s["to"], 0, s["to_table"])
        return s["Kp"], s["Vp"]
    if op == "weights":
        return cache.accumulate(s["layer"], s["q"], s["q_start"], s["kv_len"], s["table"], max_new=max(s["n"]),
                                weights=s["Wp"], decay=s["decay"])
    cache.evict(s["Wp"], case["keep"], s["kv_len"], s["table"], s["to_table"], first=case["first"],
                recent=case["recent"], kept=s["kept"], out_len=s["out_len"])
    return s["Kp"], s["Vp"], s["Wp"], s["kept"], s["out_len"]


# ------------------------------------------------------------------------- the definition in 64 bits
def _sequence(pool, s, b):
    """Rows of sequence b in order: [keys, ...] of a pool of one layer, page by page."""
    page, kv = s["case"]["page"], s["kv"][b]
    ids = [int(i) for i in s["table"][b].tolist()][:-(-kv // page)]
    return pool[ids].double().reshape(-1, pool.shape[-1])[:kv]


def exact(case, seed):
    s = _inputs(case, seed)
    op, page = case["op"], case["page"]
    if op == "append":
        C = s["Cp"].double()
        z = s["c"].double()
        if s["eps"] is not None:
            z = s["w"].double() * z / torch.sqrt(z.pow(2).sum(-1, keepdim=True) / case["latent"] + s["eps"])
        at = torch.cat([torch.arange(s["kv"][b] - s["n"][b], s["kv"][b], device="cuda") for b in range(case["B"])])
        if case["rope"]:
            pairs = case["rope"] // 2
            theta = torch.exp(torch.arange(pairs, dtype=torch.float64, device="cuda") * (-math.log(_BASE) / pairs))
            spin = torch.polar(torch.ones(len(at), pairs, dtype=torch.float64, device="cuda"),
                               at.double()[:, None] * theta)
            kr = s["kr"].double()
            if case["layout"] == "half":
                turned = torch.complex(kr[:, :pairs].contiguous(), kr[:, pairs:].contiguous()) * spin
                turned = torch.cat([turned.real, turned.imag], -1)
            else:
                turned = torch.view_as_real(torch.view_as_complex(kr.reshape(-1, pairs, 2).contiguous()) * spin)
                turned = turned.reshape(-1, case["rope"])
            z = torch.cat([z, turned], -1)
        for b in range(case["B"]):
            lo, hi = s["starts"][b], s["starts"][b + 1]
            first, done = s["kv"][b] - s["n"][b], 0
            while lo + done < hi:   # the run of rows that falls into one page
                t = first + done
                m = min(hi - lo - done, page - t % page)
                C[s["layer"], int(s["table"][b, t // page]), t % page:t % page + m] = z[lo + done:lo + done + m]
                done += m
        return C
    if op == "evict":
        K, V, W = s["Kp"].double(), s["Vp"].double(), s["Wp"].double()
        kept = torch.full((case["L"], case["B"], case["Hkv"], case["keep"]), -1, dtype=torch.int32, device="cuda")
        lens = []
        for b in range(case["B"]):
            kv = s["kv"][b]
            m = min(kv, case["keep"])
            lens.append(m)
            src = [(int(s["table"][b, t // page]), t % page) for t in range(0, kv, page)]
            ids = torch.tensor([p for p, _ in src], device="cuda")
            dst = [int(p) for p in s["to_table"][b].tolist()]
            for layer in range(case["L"]):
                for h in range(case["Hkv"]):
                    w = s["Wp"][layer, ids, h].reshape(-1)[:kv].clone()
                    fixed = torch.zeros(kv, dtype=torch.bool, device="cuda")
                    fixed[:case["first"]] = True
                    if case["recent"]:
                        fixed[max(0, kv - case["recent"]):] = True
                    free = m - int(fixed.sum())
                    pick = fixed.clone()
                    if kv <= m:
                        pick[:] = True
                    elif free > 0:
                        rest = w[~fixed]
                        border = torch.kthvalue(rest, rest.numel() - free + 1).values
                        above = ~fixed & (w > border)
                        level = (~fixed & (w == border)).nonzero()[:, 0][:free - int(above.sum())]
                        pick |= above
                        pick[level] = True
                    index = pick.nonzero()[:, 0]
                    kept[layer, b, h, :m] = index.int()
                    for pool in (K, V, W):
                        flat = pool[layer, ids, h].reshape(len(src) * page, -1)[index]
                        for i in range(0, m, page):
                            run_ = flat[i:i + page]
                            pool[layer, dst[i // page], h, :len(run_)] = run_.reshape(len(run_), *pool.shape[4:])
        return K, V, W, kept, torch.tensor(lens, dtype=torch.int32, device="cuda")
    if work(case)["flops"] > 1e12:
        return None
    if op == "latent":
        out = torch.zeros(sum(s["n"]), case["H"], case["latent"], dtype=torch.float64, device="cuda")
        for b in range(case["B"]):
            n, kv = s["n"][b], s["kv"][b]
            if n == 0:
                continue
            C = _sequence(s["Cp"][s["layer"]], s, b)
            for i in range(n):
                see = kv - n + i + 1
                at = s["starts"][b] + i
                score = torch.einsum("hd,jd->hj", s["q"][at].double(), C[:see]) * s["scale"]
                out[at] = torch.einsum("hj,jd->hd", torch.softmax(score, -1), C[:see, :case["latent"]])
        return out
    if op == "expand":
        K, V = (torch.zeros(s["to_shape"], dtype=torch.float64, device="cuda") for _ in range(2))
        dc, dr, dh = case["latent"], case["rope"], case["dh"]
        for b in range(case["B"]):
            C = _sequence(s["Cp"][s["layer"]], s, b)
            for h in range(case["H"]):
                k = torch.empty(len(C), dh, dtype=torch.float64, device="cuda")
                k[:, :dr] = C[:, dc:]
                k[:, dr:] = torch.einsum("td,dc->tc", C[:, :dc], s["WK"][:, h * (dh - dr):(h + 1) * (dh - dr)].double())
                v = torch.einsum("td,dc->tc", C[:, :dc], s["WV"][:, h * dh:(h + 1) * dh].double())
                for i in range(0, len(C), case["to_page"]):
                    p, m = int(s["to_table"][b, i // case["to_page"]]), min(case["to_page"], len(C) - i)
                    K[0, p, h, :m], V[0, p, h, :m] = k[i:i + m], v[i:i + m]
        return K, V
    W = s["Wp"].double()
    G = case["Hq"] // case["Hkv"]
    for b in range(case["B"]):
        n, kv = s["n"][b], s["kv"][b]
        if n == 0:
            continue
        seen = torch.arange(kv, device="cuda")[None, :] <= torch.arange(kv - n, kv, device="cuda")[:, None]
        for h in range(case["Hkv"]):
            K = _sequence(s["Kp"][0, :, h], s, b)
            sums = torch.zeros(kv, dtype=torch.float64, device="cuda")
            for r in range(h * G, (h + 1) * G):
                score = torch.einsum("id,jd->ij", s["q"][s["starts"][b]:s["starts"][b + 1], r].double(), K)
                score = torch.where(seen, score / math.sqrt(case["dh"]), -math.inf)
                sums += torch.softmax(score, -1).sum(0)
            for i in range(0, kv, page):
                p, m = int(s["table"][b, i // page]), min(page, kv - i)
                fresh = torch.arange(i, i + m, device="cuda") >= kv - n
                W[0, p, h, :m] = torch.where(fresh, 0.0, s["decay"] * W[0, p, h, :m]) + sums[i:i + m]
    return W
