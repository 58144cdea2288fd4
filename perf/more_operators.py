"""Measured cases of the 4-bit cache: appending to it with the rotation on the way (and reading
the tokens back), choosing pages by a cheap score, and attention over all of it or over the pages
chosen.

One serving step over long contexts goes through them in a row: keys and values are appended to
pages in 4 bits and the pages' key bounds are brought up to date (``write_cache_group4``), every
query token chooses pages by those bounds (``select_pages``), and attends to them, or to all
(``attend_group4``).  ``own`` selects between the library's calls and the same operators in plain
torch.

A pool is uint8 [P, Hkv, ps / 16, 9 D]: for 16 tokens of a page and head 16 rows of D / 2 bytes of
E2M1 codes (channel 2c in the low half of byte c, 2c + 1 in the high), then 16 rows of D / 16 E4M3
scales, one for 16 channels.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step of 64 requests of 512..8192 tokens: k and q rotated, one token appended
        # to each, its page's bounds renewed: the smallest call of a serving loop, all latency
        {"name": "append, step of 64", "op": "append", "B": 64, "lo": 512, "hi": 8192, "new_lo": 1,
         "new_hi": 1, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128, "ps": 16, "dtype": "bf16",
         "mul": False, "bounds": True, "fused": True, "lens_seed": 1},
        # eight whole prompts of 256..4096 tokens, bandwidth
        {"name": "append, 8 prompts", "op": "append", "B": 8, "lo": 0, "hi": 0, "new_lo": 256,
         "new_hi": 4096, "Hq": 32, "Hkv": 8, "D": 128, "rot": 128, "ps": 64, "dtype": "bf16",
         "mul": True, "bounds": True, "fused": True, "lens_seed": 3},
        # pages for the same decode step: 64 of up to 512 each
        {"name": "select, step of 64", "op": "select", "B": 64, "lo": 512, "hi": 8192, "new_lo": 1,
         "new_hi": 1, "Hq": 32, "Hkv": 8, "D": 128, "ps": 16, "dtype": "bf16", "n": 64, "first": 1,
         "last": 2, "window": 0, "lens_seed": 1},
        # two long contexts: few rows, a long axis to score
        {"name": "select, 2 long", "op": "select", "B": 2, "lo": 100000, "hi": 131072, "new_lo": 1,
         "new_hi": 1, "Hq": 32, "Hkv": 8, "D": 128, "ps": 32, "dtype": "bf16", "n": 64, "first": 1,
         "last": 2, "window": 0, "lens_seed": 6},
        # pieces of long prompts, each of their tokens with a choice of its own
        {"name": "select, 4 pieces", "op": "select", "B": 4, "lo": 4096, "hi": 16384, "new_lo": 200,
         "new_hi": 300, "Hq": 28, "Hkv": 4, "D": 128, "ps": 32, "dtype": "f16", "n": 32, "first": 1,
         "last": 1, "window": 0, "lens_seed": 8},
        # the decode step of 64 requests over all keys: the cache is read once, HBM-bound
        {"name": "attend, step of 64", "op": "attend", "B": 64, "lo": 512, "hi": 8192, "new_lo": 1,
         "new_hi": 1, "Hq": 32, "Hkv": 8, "D": 128, "ps": 16, "dtype": "bf16", "cap": 0.0,
         "window": 0, "slopes": False, "prefix": 0, "mul": False, "n": 0, "lens_seed": 1},
        # one short request on a small model: the smallest attention call
        {"name": "attend, one short request", "op": "attend", "B": 1, "lo": 333, "hi": 333,
         "new_lo": 1, "new_hi": 1, "Hq": 4, "Hkv": 1, "D": 64, "ps": 16, "dtype": "f16", "cap": 0.0,
         "window": 0, "slopes": False, "prefix": 0, "mul": False, "n": 0, "lens_seed": 5},
        # two long contexts: a long axis to split; scores capped at 50
        {"name": "attend, 2 long, capped", "op": "attend", "B": 2, "lo": 100000, "hi": 131072,
         "new_lo": 1, "new_hi": 1, "Hq": 32, "Hkv": 8, "D": 128, "ps": 64, "dtype": "bf16",
         "cap": 50.0, "window": 0, "slopes": False, "prefix": 0, "mul": True, "n": 0,
         "lens_seed": 6},
        # prompt pieces behind cached images, whose tokens see one another in both directions
        {"name": "attend, 4 pieces, prefix", "op": "attend", "B": 4, "lo": 1024, "hi": 4096,
         "new_lo": 700, "new_hi": 1100, "Hq": 28, "Hkv": 4, "D": 128, "ps": 32, "dtype": "f16",
         "cap": 0.0, "window": 0, "slopes": False, "prefix": 1500, "mul": False, "n": 0,
         "lens_seed": 8},
        # one prompt of 8192 tokens, causal: matrix-unit-bound
        {"name": "attend, prompt of 8192", "op": "attend", "B": 1, "lo": 0, "hi": 0, "new_lo": 8192,
         "new_hi": 8192, "Hq": 32, "Hkv": 8, "D": 128, "ps": 16, "dtype": "bf16", "cap": 0.0,
         "window": 0, "slopes": False, "prefix": 0, "mul": False, "n": 0, "lens_seed": 9},
        # two long contexts, 64 pages of 32 tokens for each kv head
        {"name": "attend, 2 long, 64 pages", "op": "attend", "B": 2, "lo": 100000, "hi": 131072,
         "new_lo": 1, "new_hi": 1, "Hq": 32, "Hkv": 8, "D": 128, "ps": 32, "dtype": "bf16",
         "cap": 0.0, "window": 0, "slopes": False, "prefix": 0, "mul": False, "n": 64,
         "lens_seed": 6},
        # pieces of long prompts over the pages that each token chose
        {"name": "attend, pieces, 32 pages", "op": "attend", "B": 2, "lo": 4096, "hi": 16384,
         "new_lo": 200, "new_hi": 300, "Hq": 28, "Hkv": 4, "D": 128, "ps": 32, "dtype": "f16",
         "cap": 0.0, "window": 0, "slopes": False, "prefix": 0, "mul": True, "n": 32,
         "lens_seed": 8},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "append", "select", "select", "attend", "attend", "attend"])
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8, 12, 16])
    D = rng.choice([64, 128, 128])
    case = {"op": op, "B": 1, "lo": 0, "hi": 0, "new_lo": 1, "new_hi": 1, "Hq": Hkv * G, "Hkv": Hkv,
            "D": D, "ps": rng.choice([16, 32, 48, 64, 128]),
            "dtype": rng.choice(["bf16", "bf16", "f16"]), "lens_seed": rng.randrange(1 << 30)}
    if op == "append":
        case["B"] = _log_int(rng, 1, 100)
        case["hi"] = _log_int(rng, 1, 4000)
        case["new_hi"] = rng.choice([1, 5, _log_int(rng, 2, 16000 // case["B"])])
        case.update({"rot": rng.choice([D, D, D // 2, 0]), "mul": rng.random() < 0.4,
                     "bounds": rng.random() < 0.7, "fused": rng.random() < 0.5})
        return case
    kind = rng.choice(["decode", "draft", "piece"])
    if op == "select":
        case["B"] = _log_int(rng, 1, 4 if kind == "piece" else 64)
        pages = _log_int(rng, 12, (200000 // case["B"] if kind != "piece" else 8000) // case["ps"])
        case["hi"] = pages * case["ps"] + rng.randrange(case["ps"])
        # requests with fewer pages than are chosen stand beside others
        case["lo"] = rng.choice([0 if case["B"] >= 8 else case["hi"] // 2, case["hi"] // 2, case["hi"]])
        if kind == "draft":
            case["new_hi"] = case["new_lo"] = rng.randrange(2, 9)
        if kind == "piece":
            case["new_hi"] = _log_int(rng, 10, 800 // case["B"])
        n = _log_int(rng, 4, max(4, min(200, pages // 3)))
        first = rng.randrange(0, min(4, n - 2))
        case.update({"n": n, "first": first, "last": rng.randrange(1, min(3, n - 1 - first) + 1),
                     "window": rng.choice([0, 0, 0, _log_int(rng, 2 * n * case["ps"], pages * case["ps"])])})
        return case
    case.update({"cap": rng.choice([0.0, 0.0, 20.0, 50.0]),
                 "window": rng.choice([0, 0, 0, _log_int(rng, 1, 3000)]),
                 "slopes": rng.random() < 0.3, "prefix": rng.choice([0, 0, _log_int(rng, 1, 900)]),
                 "mul": rng.random() < 0.3, "n": 0})
    if kind == "piece":
        case["B"] = _log_int(rng, 1, 8)
        case["hi"] = _log_int(rng, 1, 2500)
        case["new_hi"] = _log_int(rng, 30, 4000 // case["B"])
        case["new_lo"] = max(1, case["new_hi"] // 2)
    else:
        case["B"] = _log_int(rng, 1, 64)
        case["hi"] = _log_int(rng, 2, 200000 // case["B"])
        case["lo"] = rng.choice([0, case["hi"] // 4, case["hi"]])
        if kind == "draft":
            case["new_hi"] = case["new_lo"] = rng.randrange(2, 9)
    if rng.random() < 0.4:
        case["n"] = _log_int(rng, 1, max(2, 4096 // case["ps"]))
        if kind == "piece":   # each token has keys of its own in the plain form
            case["B"], case["new_hi"] = 1, min(case["new_hi"], 150)
            case["new_lo"] = min(case["new_lo"], case["new_hi"])
    return case


def _lens(case):
    """(tokens cached before the step, new tokens) of each request, by the case alone."""
    r = random.Random(case["lens_seed"])
    old = [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(case["B"])]
    return old, new


def _pages(n, ps):
    return (n + ps - 1) // ps


def work(case):
    op = case["op"]
    old, new = _lens(case)
    T, ps, Hq, Hkv, D = sum(new), case["ps"], case["Hq"], case["Hkv"], case["D"]
    row = D * 9 // 16                                     # a token of a head in 4 bits
    if op == "append":
        # k, v (and q) in, the codes out (q too); the bounds of the pages touched, with the codes
        # their earlier tokens have; the new tokens' codes in again and their values out
        kept = sum(o % ps for o, n in zip(old, new) if n) if case["bounds"] else 0
        touched = sum(_pages(o + n, ps) - o // ps for o, n in zip(old, new) if n)
        n = 2 * T * Hkv * (2 * D + row) + 2 * T * Hkv * (row + 2 * D)
        n += 4 * T * Hq * D if case["rot"] else 0
        n += kept * Hkv * row + touched * Hkv * (2 * D + 4) if case["bounds"] else 0
        return {"bytes": n, "flops": 3 * T * (Hq + Hkv) * case["rot"] + 4 * T * Hkv * D}
    if op == "select":
        pairs = pages = 0
        for o, n in zip(old, new):
            last = o + n - 1
            lo = max(0, o + 1 - case["window"]) // ps if case["window"] else 0
            pages += last // ps - lo + 1
            for i in range(n):
                lo = max(0, o + i + 1 - case["window"]) // ps if case["window"] else 0
                pairs += (o + i) // ps - lo + 1
        # bounds of every page once, queries in, the choice out
        return {"bytes": pages * Hkv * (2 * D + 4) + 4 * pages + 2 * T * Hq * D
                + 4 * T * Hkv * case["n"], "flops": 4 * pairs * Hq * D}
    pairs = seen = 0
    for o, n in zip(old, new):
        L = o + n
        if case["n"]:
            some = sum(min(case["n"] * ps, o + i + 1) for i in range(n))
            pairs += some
            seen += min(some, L)
            continue
        pre = min(case["prefix"], L)
        first = L
        for i in range(n):
            hi = max(o + i + 1, pre)
            lo = max(0, o + i + 1 - case["window"]) if case["window"] else 0
            pairs += hi - lo
            first = min(first, lo)
        seen += L - first
    return {"bytes": 2 * seen * Hkv * row + 4 * _pages(seen, ps) + 4 * T * Hq * D + 4 * T * Hq
            + 4 * T * Hkv * case["n"], "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------ the inputs

def _rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tables(old, new, ps, g, spare):
    """A random page assignment for old + new tokens: (table [B, W], pool size)."""
    need = torch.tensor([_pages(o + n, ps) for o, n in zip(old, new)], device="cuda")
    W = max(1, int(need.max()))
    total = int(need.sum())
    perm = torch.randperm(total + spare, generator=g, device="cuda").to(torch.int32)
    begin = (torch.cumsum(need, 0) - need)[:, None]
    j = torch.arange(W, device="cuda")[None, :]
    table = torch.where(j < need[:, None], perm[(begin + j).clamp(max=total + spare - 1)], -1)
    return table.to(torch.int32).contiguous(), total + spare


def _pool(g, P, Hkv, ps, D):
    """A pool of values of unit variance, larger in some pages and channels than in others."""
    x = torch.randn((P, Hkv, ps, D), generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn((P, Hkv, 1, 1), generator=g, device="cuda"))
    x *= torch.exp(0.3 * torch.randn((1, Hkv, 1, D), generator=g, device="cuda"))
    codes, scales = _encode(x)
    return torch.cat([codes.view(P, Hkv, ps // 16, 8 * D), scales.view(P, Hkv, ps // 16, D)], -1)


def prepare(case, seed):
    g = _rng(seed)
    op = case["op"]
    s = {"case": case}
    old, new = _lens(case)
    B, ps, Hq, Hkv, D, dt = (case["B"], case["ps"], case["Hq"], case["Hkv"], case["D"],
                             DT[case["dtype"]])
    T = sum(new)
    s["table"], P = _tables(old, new, ps, g, 3)
    s["old"], s["total"] = _i32(old), _i32([o + n for o, n in zip(old, new)])
    s["cu"] = torch.cumsum(torch.tensor(new), 0).to(torch.int32).cuda()
    s["max_new"], s["T"], s["P"] = max(new), T, P
    s["W"] = s["table"].shape[1]
    s["k_mul"] = s["v_mul"] = None
    if case.get("mul"):
        for name in ("k_mul", "v_mul"):
            s[name] = torch.exp2(torch.randn(Hkv, generator=g, device="cuda") - 1.0)

    def normal(shape):
        return torch.randn(shape, generator=g, device="cuda").to(dt)

    if op == "append":
        s["k_pool"], s["v_pool"] = _pool(g, P, Hkv, ps, D), _pool(g, P, Hkv, ps, D)
        grow = torch.exp(0.5 * torch.randn((T, 1, 1), generator=g, device="cuda"))
        x = (torch.randn((T, Hq + 2 * Hkv, D), generator=g, device="cuda") * grow).to(dt)
        if not case["fused"]:   # else columns of one fused projection
            s["q"], s["k"], s["v"] = (y.contiguous() for y in x.split([Hq, Hkv, Hkv], 1))
        else:
            s["q"], s["k"], s["v"] = x.split([Hq, Hkv, Hkv], 1)
        s["cos"] = s["sin"] = None
        if case["rot"]:
            half = case["rot"] // 2
            inv = 1e6 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
            angle = torch.arange(max(o + n for o, n in zip(old, new)), dtype=torch.float64,
                                 device="cuda")[:, None] * inv
            s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["bounds"] = s["bscale"] = None
        if case["bounds"]:
            s["bounds"] = torch.zeros((P, Hkv, 2, D), dtype=torch.int8, device="cuda")
            s["bscale"] = torch.ones((P, Hkv), device="cuda")
        return s
    s["q"] = normal((T, Hq, D))
    if op == "select":
        # bounds around a mean of each channel, larger in some pages than in others
        size = torch.exp(0.5 * torch.randn((P, Hkv, 1), generator=g, device="cuda"))
        mean = size * torch.randn((P, Hkv, D), generator=g, device="cuda")
        half = size * torch.randn((P, Hkv, D), generator=g, device="cuda").abs()
        top = torch.maximum((mean + half).abs(), (mean - half).abs()).amax(-1)
        s["bscale"] = torch.exp2(torch.ceil(torch.log2(top / 127.0)))
        unit = s["bscale"][..., None]
        s["bounds"] = torch.stack([torch.floor((mean - half) / unit), torch.ceil((mean + half) / unit)],
                                  2).clamp_(-127, 127).to(torch.int8)
        return s
    s["k_pool"], s["v_pool"] = _pool(g, P, Hkv, ps, D), _pool(g, P, Hkv, ps, D)
    s["slopes"] = (2.0 ** (-8.0 * (torch.arange(Hq, device="cuda") + 1) / Hq)
                   if case["slopes"] else None)
    s["prefix"] = (_i32([min(case["prefix"], o + n) for o, n in zip(old, new)])
                   if case["prefix"] else None)
    s["selected"] = None
    if case["n"]:
        # the newest page of each token and others of its past, in their order
        at = torch.cat([o + torch.arange(n) for o, n in zip(old, new)]).cuda()
        key = torch.rand((T, Hkv, max(s["W"], case["n"])), generator=g, device="cuda")
        j = torch.arange(key.shape[2], device="cuda")
        newest = (at // ps)[:, None, None]
        key = torch.where(j == newest, 2.0, torch.where(j < newest, key, -1.0))
        pick = key.topk(case["n"], -1)
        ids = torch.where(pick.values < 0, 1 << 30, pick.indices).sort(-1).values
        s["selected"] = torch.where(ids == 1 << 30, -1, ids).to(torch.int32).contiguous()
    return s


# --------------------------------------------------------------- the operators

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s)
    return {"append": _plain_append, "select": _plain_select, "attend": _plain_attend}[op](s)


def _own(op, s):
    import quantized_paged_kv_varlen_gb300 as lib
    c = s["case"]
    if op == "append":
        q = s["q"] if c["rot"] else None
        q_out = lib.write_cache_group4(
            s["k"], s["v"], s["cu"], s["table"], s["k_pool"], s["v_pool"], start_pos=s["old"],
            rope_cos=s["cos"], rope_sin=s["sin"], q=q, k_bounds=s["bounds"],
            bound_scale=s["bscale"], k_mul=s["k_mul"], v_mul=s["v_mul"])
        k, v = lib.read_cache_group4(s["k_pool"], s["v_pool"], s["cu"], s["table"], s["T"],
                                     start_pos=s["old"], k_mul=s["k_mul"], v_mul=s["v_mul"],
                                     dtype=s["k"].dtype)
        return {"q": q_out, "k": k, "v": v, "bounds": s["bounds"], "bscale": s["bscale"]}
    if op == "select":
        return lib.select_pages(s["q"], s["bounds"], s["bscale"], s["table"], s["cu"], s["total"],
                                c["ps"], c["n"], first=c["first"], last=c["last"],
                                window=c["window"], max_seqlen_q=s["max_new"])
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    out = lib.attend_group4(s["q"], s["k_pool"], s["v_pool"], s["table"], s["cu"], s["total"],
                            max_seqlen_q=s["max_new"], logit_cap=c["cap"], window=c["window"],
                            alibi_slopes=s["slopes"], prefix_lens=s["prefix"],
                            selected=s["selected"], k_mul=s["k_mul"], v_mul=s["v_mul"], lse=lse)
    return out, lse


def _encode(x):
    """float32 [..., D] -> (codes uint8 [..., D / 2], scales uint8 [..., D / 16])."""
    g = x.unflatten(-1, (-1, 16))
    six = torch.tensor(6.0, device=x.device)              # by a tensor: torch multiplies by 1 / 6
    scale = (g.abs().amax(-1) / six).clamp(max=448.0).to(torch.float8_e4m3fn)
    unit = scale.float()[..., None]
    y = torch.where(unit > 0, g / unit, torch.zeros_like(g))
    a = y.abs()
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
            + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5.0).byte())   # ties to the even code
    code = (code + (y < 0).byte() * 8).flatten(-2)
    return code[..., 0::2] | code[..., 1::2] << 4, scale.view(torch.uint8)


def _decode(codes, scales):
    """float32 [..., D] of codes uint8 [..., D / 2] and scales uint8 [..., D / 16]."""
    value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, 0, -0.5, -1, -1.5, -2, -3, -4, -6],
                         device=codes.device)
    x = torch.stack([value[(codes & 15).int()], value[(codes >> 4).int()]], -1).flatten(-2)
    return (x.unflatten(-1, (-1, 16)) * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _page_values(pages):
    """float32 [..., ps, D] of pool pages [..., ps / 16, 9 D]."""
    D = pages.shape[-1] // 9
    codes = pages[..., :8 * D].unflatten(-1, (16, D // 2)).flatten(-3, -2)
    scales = pages[..., 8 * D:].unflatten(-1, (16, D // 16)).flatten(-3, -2)
    return _decode(codes.contiguous(), scales.contiguous())


def _plain_append(s):
    c = s["case"]
    ps, D, half = c["ps"], c["D"], c["rot"] // 2
    T = s["k"].shape[0]
    cu, old = s["cu"].long(), s["old"].long()
    begin = torch.cat([cu.new_zeros(1), cu[:-1]])
    b = torch.searchsorted(cu, torch.arange(T, device="cuda"), right=True)
    pos = old[b] + torch.arange(T, device="cuda") - begin[b]
    page, o = s["table"][b, pos // ps].long(), pos % ps

    def turn(x):
        if not half:
            return x.float()
        cos, sin = s["cos"][pos][:, None], s["sin"][pos][:, None]
        u, w = x[..., :half].float(), x[..., half:2 * half].float()
        return torch.cat([u * cos - w * sin, w * cos + u * sin, x[..., 2 * half:].float()], -1)

    out = {"q": turn(s["q"]).to(s["q"].dtype) if half else None, "bounds": s["bounds"],
           "bscale": s["bscale"]}
    for name in ("k", "v"):
        x = turn(s[name]) if name == "k" else s[name].float()
        mul = s[name + "_mul"]
        if mul is not None:
            x = x / mul[:, None]
        pool, (codes, scales) = s[name + "_pool"], _encode(x)
        pool[..., :8 * D].unflatten(-1, (16, D // 2))[page, :, o // 16, o % 16] = codes
        pool[..., 8 * D:].unflatten(-1, (16, D // 16))[page, :, o // 16, o % 16] = scales
        y = _decode(codes, scales)
        out[name] = (y if mul is None else y * mul[:, None]).to(s[name].dtype)
    if c["bounds"]:
        W = s["W"]
        place = torch.unique(b * W + pos // ps)
        b, no = place // W, place % W
        page = s["table"][b, no].long()
        filled = (old + cu - begin)[b] - no * ps
        x = _page_values(s["k_pool"][page]) * 1024.0      # whole numbers
        here = (torch.arange(ps, device="cuda") < filled[:, None])[:, None, :, None]
        lo = torch.where(here, x, math.inf).amin(2)
        hi = torch.where(here, x, -math.inf).amax(2)
        top = torch.maximum(lo.abs(), hi.abs()).amax(-1)
        e = (top[..., None] > 127.0 * 2.0 ** torch.arange(16, device="cuda")).sum(-1)
        unit = torch.exp2(e.float())
        s["bounds"][page] = torch.stack([torch.floor(lo / unit[..., None]),
                                         torch.ceil(hi / unit[..., None])], 2).to(torch.int8)
        s["bscale"][page] = unit / 1024.0
    return out


def _rows(s):
    """Sequence and position of each query row."""
    cu, total = s["cu"].long(), s["total"].long()
    begin = torch.cat([cu.new_zeros(1), cu[:-1]])
    t = torch.arange(s["T"], device="cuda")
    b = torch.searchsorted(cu, t, right=True)
    return b, (total - cu)[b] + t


def _plain_select(s):
    c = s["case"]
    Hkv, D, ps, n, W = c["Hkv"], c["D"], c["ps"], c["n"], s["W"]
    b, at = _rows(s)
    q = s["q"].float().view(s["T"], Hkv, -1, D)
    top = q.abs().amax((2, 3), keepdim=True)
    q = torch.where(top > 0, torch.round(q * 127.0 / top), torch.zeros_like(q))
    page = s["table"].long().clamp(min=0)
    # one product for all rows of a request: rows [B, n, ...] of requests with fewer stay empty
    cu = s["cu"].long()
    begin = torch.cat([cu.new_zeros(1), cu[:-1]])
    m = s["max_new"]
    x = torch.zeros((c["B"], m) + q.shape[1:], device="cuda")
    i = torch.arange(s["T"], device="cuda") - begin[b]
    x[b, i] = q
    x = x.permute(0, 2, 1, 3, 4).flatten(2, 3)            # [B, Hkv, m G, D]
    bounds = s["bounds"][page].float().permute(0, 2, 3, 4, 1)   # [B, Hkv, 2, D, W]
    score = x.clamp(min=0) @ bounds[:, :, 1] + x.clamp(max=0) @ bounds[:, :, 0]
    score = score.view(c["B"], Hkv, m, -1, W).amax(3) * s["bscale"][page].transpose(1, 2)[:, :, None]
    score = score.permute(0, 2, 1, 3)[b, i]               # [T, Hkv, W]
    j = torch.arange(W, device="cuda")
    lo = ((at + 1 - c["window"]).clamp(min=0) // ps if c["window"] else torch.zeros_like(at))
    lo, hi = lo[:, None, None], (at // ps)[:, None, None]
    sure = (j < lo + c["first"]) | (j > hi - c["last"])
    score = torch.where(sure, math.inf, score)
    score = torch.where((j >= lo) & (j <= hi), score, -math.inf)
    best = torch.sort(score, dim=-1, descending=True, stable=True)
    ids = torch.where(best.values > -math.inf, best.indices, 1 << 30)[..., :n].sort(-1).values
    ids = torch.nn.functional.pad(ids, (0, max(0, n - W)), value=1 << 30)
    return torch.where(ids == 1 << 30, -1, ids).to(torch.int32)


def _softmax_times(S, V):
    m = S.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    S = S.sub_(m).exp_()
    l = S.sum(-1, keepdim=True)
    O = torch.matmul(S, V)
    return torch.where(l > 0, O / l, torch.zeros_like(O)), (m + torch.log(l))[..., 0]


def _plain_attend(s):
    c = s["case"]
    B, Hq, Hkv, D, ps, T, W = c["B"], c["Hq"], c["Hkv"], c["D"], c["ps"], s["T"], s["W"]
    G, n = Hq // Hkv, s["max_new"]
    b, at = _rows(s)
    total = s["total"].long()
    scale = torch.full((Hkv,), 1.0 / math.sqrt(D), device="cuda")
    if s["k_mul"] is not None:
        scale = scale * s["k_mul"]
    table = s["table"].long().clamp(min=0)
    if s["selected"] is not None:
        # every (token, kv head) has keys of its own
        ids = s["selected"].long()                        # [T, Hkv, n]
        page = table[b[:, None, None], ids.clamp(min=0)]
        h = torch.arange(Hkv, device="cuda")[None, :, None]
        j = ids[..., None] * ps + torch.arange(ps, device="cuda")
        j = torch.where(ids[..., None] < 0, 1 << 40, j).flatten(2)[:, :, None]      # [T, Hkv, 1, keys]
        K, V = (_page_values(s[x][page, h]).flatten(2, 3) for x in ("k_pool", "v_pool"))
        q = s["q"].float().view(T, Hkv, G, D)
        pos = at[:, None, None, None]
        end = total[b][:, None, None, None]
    else:
        K, V = (_page_values(s[x][table]).permute(0, 2, 1, 3, 4).reshape(B, Hkv, W * ps, D)
                for x in ("k_pool", "v_pool"))
        cu = s["cu"].long()
        begin = torch.cat([cu.new_zeros(1), cu[:-1]])
        i = torch.arange(n, device="cuda")
        rows = (begin[:, None] + i).clamp(max=T - 1)
        q = s["q"][rows].float().reshape(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
        pos = ((total - cu + begin)[:, None] + i).repeat(1, G)[:, None, :, None]    # [B, 1, G n, 1]
        j = torch.arange(W * ps, device="cuda")
        end = total[:, None, None, None]
    S = torch.matmul(q, K.transpose(2, 3)).mul_(scale[:, None, None])
    if c["cap"]:
        S = torch.tanh(S.div_(c["cap"])).mul_(c["cap"])
    if s["slopes"] is not None:
        slope = s["slopes"].view(Hkv, G)
        slope = slope[:, :, None] if s["selected"] is not None else slope.repeat_interleave(n, 1)[:, :, None]
        S += slope * (j - pos).float()
    hi = pos + 1
    if s["prefix"] is not None:
        pre = s["prefix"].long()
        hi = torch.maximum(hi, (pre[b] if s["selected"] is not None else pre)[:, None, None, None])
    see = j < torch.minimum(hi, end)
    if c["window"]:
        see = see & (j >= pos + 1 - c["window"])
    S.masked_fill_(~see, -math.inf)
    O, lse = _softmax_times(S, V)
    if s["v_mul"] is not None:
        O = O * s["v_mul"][:, None, None]
    if s["selected"] is None:
        r = torch.arange(T, device="cuda") - begin[b]
        O = O.view(B, Hkv, G, n, D).permute(0, 3, 1, 2, 4)[b, r]
        lse = lse.view(B, Hkv, G, n).permute(0, 3, 1, 2)[b, r]
    return O.reshape(T, Hq, D).to(s["q"].dtype), lse.reshape(T, Hq).contiguous()


# ------------------------------------------------------- the definitions in 64 bits

def _e4m3_table():
    """What the E4M3 codes 0 ... 126 stand for: 4 exponent bits with bias 7, 3 mantissa bits."""
    v = [(c & 7) / 8.0 * 2.0 ** -6 if c < 8 else (1 + (c & 7) / 8.0) * 2.0 ** ((c >> 3) - 7)
         for c in range(127)]
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _nearest(x, table):
    """The entry of an ascending table that is nearest to each x >= 0; ties to the even one."""
    mid = (table[1:] + table[:-1]) / 2
    n = torch.searchsorted(mid, x.contiguous())           # mid[n - 1] < x <= mid[n]
    tie = (n < mid.numel()) & (mid[n.clamp(max=mid.numel() - 1)] == x)
    return table[torch.where(tie & (n % 2 == 1), n + 1, n)]


def _exact_values(pool, page, h):
    """float64 [pages, ps, D] of head h's pages."""
    D = pool.shape[-1] // 9
    raw = pool[page, h].long()                            # [pages, ps / 16, 9 D]
    byte = raw[..., :8 * D].reshape(raw.shape[0], -1, D // 2)
    scale = _e4m3_table()[raw[..., 8 * D:].reshape(raw.shape[0], -1, D // 16)]
    mag = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=torch.float64, device="cuda") / 2
    x = torch.empty(byte.shape[:2] + (D,), dtype=torch.float64, device="cuda")
    x[..., 0::2] = mag[byte % 8] * (1 - 2 * (byte // 8 % 2))
    x[..., 1::2] = mag[byte // 16 % 8] * (1 - 2 * (byte // 128))
    return x * scale.repeat_interleave(16, -1)


def exact(case, seed):
    op = case["op"]
    if op == "select":
        return None                                        # whole numbers only
    s = prepare(case, seed)
    f64 = torch.float64
    old, new = _lens(case)
    ps, Hq, Hkv, D = case["ps"], case["Hq"], case["Hkv"], case["D"]
    if op == "append":
        half = case["rot"] // 2
        pos = torch.cat([o + torch.arange(n) for o, n in zip(old, new)]).cuda()

        def turn(x):
            x = x.to(f64)
            if half:
                z = torch.complex(x[..., :half], x[..., half:2 * half])
                z = z * torch.complex(s["cos"].to(f64), s["sin"].to(f64))[pos][:, None]
                x = torch.cat([z.real, z.imag, x[..., 2 * half:]], -1)
            return x

        steps = torch.tensor([0, 1, 2, 3, 4, 6, 8, 12], dtype=f64, device="cuda") / 2
        out = {"q": turn(s["q"]) if half else None, "bounds": None, "bscale": None}
        for name in ("k", "v"):
            x = turn(s[name]) if name == "k" else s[name].to(f64)
            mul = s[name + "_mul"]
            mul = torch.ones(Hkv, dtype=f64, device="cuda") if mul is None else mul.to(f64)
            x = (x / mul[:, None]).reshape(x.shape[0], Hkv, D // 16, 16)
            unit = _nearest(x.abs().amax(-1) / 6, _e4m3_table())[..., None]
            y = torch.where(unit > 0, x / unit.clamp(min=1e-300), 0 * x)
            y = torch.copysign(_nearest(y.abs(), steps), y) * unit
            out[name] = y.reshape(x.shape[0], Hkv, D) * mul[:, None]
        return out
    G = Hq // Hkv
    table = s["table"].tolist()
    T = sum(new)
    o_all = torch.zeros((T, Hq, D), dtype=f64, device="cuda")
    lse_all = torch.empty((T, Hq), dtype=f64, device="cuda")
    k_mul = [1.0] * Hkv if s["k_mul"] is None else s["k_mul"].to(f64).tolist()
    v_mul = [1.0] * Hkv if s["v_mul"] is None else s["v_mul"].to(f64).tolist()
    slopes = s["slopes"].to(f64) if s["slopes"] is not None else None
    t0 = 0
    for b in range(case["B"]):
        L, n = old[b] + new[b], new[b]
        pg = torch.tensor(table[b][:_pages(L, ps)], device="cuda")
        i = torch.arange(n, device="cuda")[:, None] + old[b]
        j = torch.arange(L, device="cuda")[None, :]
        see = (j <= i) | (j < min(case["prefix"], L))
        if case["window"]:
            see &= j > i - case["window"]
        for h in range(Hkv):
            K = _exact_values(s["k_pool"], pg, h).reshape(-1, D)[:L] * k_mul[h]
            V = _exact_values(s["v_pool"], pg, h).reshape(-1, D)[:L] * v_mul[h]
            mine = see
            if s["selected"] is not None:
                ids = s["selected"][t0:t0 + n, h].long()
                chosen = torch.zeros((n, pg.numel() + 1), dtype=torch.bool, device="cuda")
                chosen.scatter_(1, torch.where(ids < 0, pg.numel(), ids), True)
                mine = see & chosen[:, :-1].repeat_interleave(ps, 1)[:, :L]
            for a in range(h * G, h * G + G):
                x = s["q"][t0:t0 + n, a].to(f64) @ K.T / math.sqrt(D)
                if case["cap"]:
                    x = case["cap"] * torch.tanh(x / case["cap"])
                if slopes is not None:
                    x = x + slopes[a] * (j - i)
                x = x.masked_fill(~mine, -math.inf)
                lse = torch.logsumexp(x, -1)
                lse_all[t0:t0 + n, a] = lse
                o_all[t0:t0 + n, a] = torch.exp(x - lse[:, None]).nan_to_num(0.0) @ V
        t0 += n
    return o_all, lse_all
