"""Measured cases of the page-scaled 8-bit cache: page assignment, rotary
positions with several axes, the cache write and the attention that reads it.

One serving step of a continuous batch goes through all four: requests get
pages and slots on the GPU (``assign_pages``), queries and keys are rotated
at positions with one or several axes (``rope_axes``), keys and values are
appended to a paged cache in 8 bits with one scale per page and kv head
(``write_cache_page8``), and the queries attend to that cache
(``attend_page8``).  ``own`` selects between the library's calls and the
same operators in plain torch.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step of the benchmark's batch (64 requests of 512..8192 tokens): the smallest
        # call of a serving loop, all latency
        {"name": "pages, step of 64", "op": "pages", "B": 64, "lo": 512, "hi": 8192, "new_lo": 1,
         "new_hi": 1, "ps": 16, "lens_seed": 1},
        # 256 prompts and prompt pieces admitted at once, among them requests that only decode
        {"name": "pages, 256 prompts", "op": "pages", "B": 256, "lo": 0, "hi": 2048, "new_lo": 1,
         "new_hi": 512, "ps": 16, "lens_seed": 2},
        # a video prompt: queries and keys of 16384 tokens, (time, height, width) over 64 pairs
        {"name": "rope, video of 16384", "op": "rope", "T": 16384, "Hq": 32, "Hkv": 8, "D": 128,
         "s0": 16, "s1": 24, "s2": 24, "inter": False, "dtype": "bf16", "fused": True},
        # the same rotation in a decode step of 64 requests
        {"name": "rope, step of 64", "op": "rope", "T": 64, "Hq": 28, "Hkv": 4, "D": 128,
         "s0": 24, "s1": 20, "s2": 20, "inter": True, "dtype": "bf16", "fused": False},
        # eight prompts of the benchmark's prefill (256..4096 tokens, 32 heads, page 64) written whole
        {"name": "write, 8 prompts", "op": "write", "B": 8, "lo": 0, "hi": 0, "new_lo": 256,
         "new_hi": 4096, "Hkv": 32, "D": 128, "ps": 64, "fmt": "e4m3", "dtype": "bf16",
         "hnd": False, "lens_seed": 3},
        # one token appended to each of 64 requests: partly filled pages are rescaled
        {"name": "write, step of 64", "op": "write", "B": 64, "lo": 512, "hi": 8192, "new_lo": 1,
         "new_hi": 1, "Hkv": 8, "D": 128, "ps": 16, "fmt": "int8", "dtype": "bf16", "hnd": False,
         "lens_seed": 4},
        # the decode step of the benchmark's batch: the cache is read once, HBM-bound
        {"name": "attend, step of 64", "op": "attend", "B": 64, "lo": 512, "hi": 8192, "new_lo": 1,
         "new_hi": 1, "Hq": 32, "Hkv": 8, "D": 128, "ps": 16, "fmt": "e4m3", "dtype": "bf16",
         "hnd": False, "cap": 0.0, "window": 0, "slopes": False, "prefix": 0, "lens_seed": 1},
        # one short request on a small model: the smallest attention call
        {"name": "attend, one short request", "op": "attend", "B": 1, "lo": 333, "hi": 333,
         "new_lo": 1, "new_hi": 1, "Hq": 4, "Hkv": 1, "D": 64, "ps": 16, "fmt": "int8",
         "dtype": "f16", "hnd": False, "cap": 0.0, "window": 0, "slopes": False, "prefix": 0,
         "lens_seed": 5},
        # two requests with long contexts: few rows, a long axis to split; scores capped at 50
        {"name": "attend, 2 long, capped", "op": "attend", "B": 2, "lo": 100000, "hi": 131072,
         "new_lo": 1, "new_hi": 1, "Hq": 32, "Hkv": 8, "D": 128, "ps": 64, "fmt": "int8",
         "dtype": "bf16", "hnd": True, "cap": 50.0, "window": 0, "slopes": False, "prefix": 0,
         "lens_seed": 6},
        # five drafted tokens per request checked in one call, with a bias that falls with distance
        {"name": "attend, drafts of 5, biased", "op": "attend", "B": 32, "lo": 1024, "hi": 4096,
         "new_lo": 5, "new_hi": 5, "Hq": 32, "Hkv": 8, "D": 128, "ps": 16, "fmt": "e4m3",
         "dtype": "bf16", "hnd": False, "cap": 0.0, "window": 0, "slopes": True, "prefix": 0,
         "lens_seed": 7},
        # prompt pieces behind cached images: the image's tokens see one another in both directions
        {"name": "attend, 4 pieces, prefix", "op": "attend", "B": 4, "lo": 1024, "hi": 4096,
         "new_lo": 700, "new_hi": 1100, "Hq": 28, "Hkv": 4, "D": 128, "ps": 32, "fmt": "int8",
         "dtype": "f16", "hnd": False, "cap": 0.0, "window": 0, "slopes": False, "prefix": 1500,
         "lens_seed": 8},
        # one prompt of 8192 tokens, causal: matrix-unit-bound
        {"name": "attend, prompt of 8192", "op": "attend", "B": 1, "lo": 0, "hi": 0, "new_lo": 8192,
         "new_hi": 8192, "Hq": 32, "Hkv": 8, "D": 128, "ps": 16, "fmt": "e4m3", "dtype": "bf16",
         "hnd": False, "cap": 0.0, "window": 0, "slopes": False, "prefix": 0, "lens_seed": 9},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "rope", "write", "write", "attend", "attend", "attend"])
    seed = rng.randrange(1 << 30)
    ps = rng.choice([16, 32, 48, 64, 128])
    if op == "pages":
        new_hi = rng.choice([1, 1, 7, _log_int(rng, 2, 700)])
        return {"op": op, "B": _log_int(rng, 1, 300), "lo": 0, "hi": _log_int(rng, 1, 6000),
                "new_lo": min(1, new_hi), "new_hi": new_hi, "ps": ps, "lens_seed": seed}
    D = rng.choice([64, 128, 128])
    if op == "rope":
        half = D // 2
        s0 = rng.randrange(4, half // 2)
        s1 = (half - s0) // 2
        return {"op": op, "T": _log_int(rng, 1, 9000), "Hq": rng.choice([1, 4, 12, 20, 28, 32]),
                "Hkv": rng.choice([1, 2, 4, 8]), "D": D, "s0": s0, "s1": s1, "s2": half - s0 - s1,
                "inter": rng.random() < 0.5, "dtype": rng.choice(["bf16", "f16", "f32"]),
                "fused": rng.random() < 0.5}
    case = {"op": op, "B": 1, "lo": 0, "hi": 0, "new_lo": 1, "new_hi": 1, "Hkv": 1, "D": D, "ps": ps,
            "fmt": rng.choice(["e4m3", "int8"]), "dtype": rng.choice(["bf16", "bf16", "f16"]),
            "hnd": rng.random() < 0.3, "lens_seed": seed}
    if op == "write":
        case["B"] = _log_int(rng, 1, 100)
        case["Hkv"] = rng.choice([1, 2, 3, 4, 8])
        case["hi"] = _log_int(rng, 1, 4000)
        case["new_hi"] = rng.choice([1, 5, _log_int(rng, 2, 60000 // case["B"])])
        return case
    Hkv, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 8, 12, 16])
    case.update({"Hkv": Hkv, "Hq": Hkv * G, "cap": rng.choice([0.0, 0.0, 20.0, 50.0]),
                 "window": rng.choice([0, 0, 0, _log_int(rng, 1, 3000)]),
                 "slopes": rng.random() < 0.3, "prefix": rng.choice([0, 0, _log_int(rng, 1, 900)])})
    kind = rng.choice(["decode", "draft", "piece"])
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
    if op == "rope":
        es = 4 if case["dtype"] == "f32" else 2
        n = case["T"] * (case["Hq"] + case["Hkv"]) * case["D"]
        # queries and keys in and out, three positions and the table rows they name
        return {"bytes": 2 * n * es + case["T"] * 12, "flops": 3 * n}
    old, new = _lens(case)
    T, B, ps = sum(new), case["B"], case["ps"]
    if op == "pages":
        held = sum(_pages(o, ps) for o in old)
        got = sum(_pages(o + n, ps) - _pages(o, ps) for o, n in zip(old, new))
        # lengths in; pages held and taken read and the table written; cu, lengths, slots, positions
        W = max(_pages(o + n, ps) for o, n in zip(old, new))
        return {"bytes": 4 * (2 * B + held + got + B * W + 2 * B + 2 * T), "flops": 4 * T}
    Hkv, D = case["Hkv"], case["D"]
    if op == "write":
        touched = sum(_pages(o + n, ps) - o // ps for o, n in zip(old, new) if n)
        # k and v in 16 bits in, 8 bits out; the partly filled pages' codes in; scales; indices
        kept = sum(o % ps for o, n in zip(old, new) if n)
        return {"bytes": 2 * T * Hkv * D * 3 + 2 * kept * Hkv * D + 8 * touched * Hkv
                + 4 * (touched + 2 * B), "flops": 4 * T * Hkv * D}
    Hq = case["Hq"]
    pairs = seen_tokens = 0
    for b, (o, n) in enumerate(zip(old, new)):
        L = o + n
        pre = min(case["prefix"], L)
        first = L
        for i in range(n):
            hi = max(o + i + 1, pre)
            lo = max(0, o + i + 1 - case["window"]) if case["window"] else 0
            pairs += hi - lo
            first = min(first, lo)
        seen_tokens += L - first
    return {"bytes": 2 * seen_tokens * Hkv * D + 8 * Hkv * _pages(seen_tokens, ps)
            + 4 * T * Hq * D + 4 * T * Hq + 4 * _pages(seen_tokens, ps),
            "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------ the inputs

def _rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tables(old, new, ps, g, spare):
    """A random page assignment for old + new tokens: (table [B, W], pool size, permutation)."""
    need = torch.tensor([_pages(o + n, ps) for o, n in zip(old, new)], device="cuda")
    W = max(1, int(need.max()))
    total = int(need.sum())
    perm = torch.randperm(total + spare, generator=g, device="cuda").to(torch.int32)
    begin = (torch.cumsum(need, 0) - need)[:, None]
    j = torch.arange(W, device="cuda")[None, :]
    table = torch.where(j < need[:, None], perm[(begin + j).clamp(max=total + spare - 1)], -1)
    return table.to(torch.int32).contiguous(), total + spare, perm


def prepare(case, seed):
    g = _rng(seed)
    op = case["op"]
    s = {"case": case}

    def normal(shape, dtype):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    if op == "rope":
        T, Hq, Hkv, D, dt = case["T"], case["Hq"], case["Hkv"], case["D"], DT[case["dtype"]]
        half = D // 2
        if case["fused"]:   # q and k are columns of one fused projection
            x = normal((T, Hq + 2 * Hkv, D), dt)
            s["q"], s["k"] = x[:, :Hq], x[:, Hq:Hq + Hkv]
        else:
            s["q"], s["k"] = normal((T, Hq, D), dt), normal((T, Hkv, D), dt)
        n = max(T, 64)
        # frames of 16 x 24 patches: time, height and width positions
        t = torch.arange(T, device="cuda") + torch.randint(0, 64, (1,), generator=g, device="cuda")
        s["pos"] = torch.stack([t // 384, t % 384 // 24, t % 24]).to(torch.int32)
        inv = 1e6 ** (-2.0 * torch.arange(half, dtype=torch.float64, device="cuda") / D)
        angle = torch.arange(n, dtype=torch.float64, device="cuda")[:, None] * inv
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        s["axis"] = _pair_axis(case)
        s["axis_t"] = torch.tensor(list(s["axis"]), device="cuda")
        return s
    old, new = _lens(case)
    B, ps = case["B"], case["ps"]
    total = [o + n for o, n in zip(old, new)]
    cu = torch.cumsum(torch.tensor(new), 0).to(torch.int32).cuda()
    if op == "pages":
        held = [_pages(o, ps) for o in old]
        full, P, perm = _tables(old, new, ps, g, 100)
        j = torch.arange(full.shape[1], device="cuda")[None, :]
        s["table"] = torch.where(j < _i32(held)[:, None], full, -1).to(torch.int32).contiguous()
        taken = torch.zeros(P, dtype=torch.bool, device="cuda")
        taken[s["table"][s["table"] >= 0].long()] = True
        free = perm[~taken[perm.long()]]
        s["free"] = torch.cat([free, torch.zeros(P - free.numel(), dtype=torch.int32, device="cuda")])
        s["count"] = _i32([free.numel()])
        s["old"], s["new"], s["P"], s["T"] = _i32(old), _i32(new), P, sum(new)
        return s
    Hkv, D, dt, T = case["Hkv"], case["D"], DT[case["dtype"]], sum(new)
    s["table"], P, _ = _tables(old, new, ps, g, 3)
    s["old"], s["total"], s["cu"] = _i32(old), _i32(total), cu
    # the pool: codes of values of unit variance, larger in some pages than in others
    pool_kind = torch.uint8 if case["fmt"] == "e4m3" else torch.int8
    qmax = 448.0 if case["fmt"] == "e4m3" else 127.0
    shape = (P, Hkv, ps, D) if case["hnd"] else (P, ps, Hkv, D)
    for name in ("k", "v"):
        size = torch.exp(0.5 * torch.randn((P, Hkv), generator=g, device="cuda"))
        amax = size * (3.5 + 0.3 * torch.rand((P, Hkv), generator=g, device="cuda"))
        x = torch.randn(shape, generator=g, device="cuda").clamp_(-3.4, 3.4)
        x.mul_((size / (amax / qmax))[:, :, None, None] if case["hnd"]
               else (size / (amax / qmax))[:, None, :, None])
        s[name + "_pool"] = (x.to(torch.float8_e4m3fn).view(torch.uint8) if case["fmt"] == "e4m3"
                             else x.round_().to(torch.int8))
        s[name + "_scale"] = amax / qmax
        del x
        assert s[name + "_pool"].dtype == pool_kind
    if op == "write":
        grow = torch.exp(0.5 * torch.randn((T, 1, 1), generator=g, device="cuda"))
        s["k"] = (torch.randn((T, Hkv, D), generator=g, device="cuda") * grow).to(dt)
        s["v"] = (torch.randn((T, Hkv, D), generator=g, device="cuda") * grow).to(dt)
        return s
    Hq = case["Hq"]
    s["q"] = normal((T, Hq, D), dt)
    s["max_new"] = max(new)
    s["slopes"] = (2.0 ** (-8.0 * (torch.arange(Hq, device="cuda") + 1) / Hq)
                   if case["slopes"] else None)
    s["prefix"] = _i32([min(case["prefix"], t) for t in total]) if case["prefix"] else None
    s["W"] = max(_pages(t, ps) for t in total)
    return s


def _pair_axis(case):
    """The axis of each pair: blocks of s0, s1, s2 pairs, or the three axes taking turns while
    the last two have pairs left."""
    half = case["D"] // 2
    if not case["inter"]:
        return bytes([0] * case["s0"] + [1] * case["s1"] + [2] * case["s2"])
    axis = [0] * half
    for a, n in ((1, case["s1"]), (2, case["s2"])):
        for i in range(a, min(half, 3 * n), 3):
            axis[i] = a
    return bytes(axis)


# --------------------------------------------------------------- the operators

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s)
    return {"pages": _plain_pages, "rope": _plain_rope, "write": _plain_write,
            "attend": _plain_attend}[op](s)


def _values(pool):
    """The pool's codes as numbers of their own type."""
    return pool.view(torch.float8_e4m3fn) if pool.dtype == torch.uint8 else pool


def _own(op, s):
    import quantized_paged_kv_varlen_gb300 as lib
    c = s["case"]
    if op == "pages":
        return lib.assign_pages(s["new"], s["old"], s["table"], s["free"], s["count"], c["ps"],
                                s["P"], s["T"])
    if op == "rope":
        return lib.rope_axes(s["q"], s["pos"], s["axis"], s["cos"], s["sin"], k=s["k"])
    layout = "HND" if c["hnd"] else "NHD"
    if op == "write":
        lib.write_cache_page8(s["k"], s["v"], s["cu"], s["table"], s["k_pool"], s["v_pool"],
                              s["k_scale"], s["v_scale"], start_pos=s["old"], kv_layout=layout)
        return _values(s["k_pool"]), _values(s["v_pool"]), s["k_scale"], s["v_scale"]
    lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    out = lib.attend_page8(s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["table"],
                           s["cu"], s["total"], max_seqlen_q=s["max_new"], logit_cap=c["cap"],
                           window=c["window"], alibi_slopes=s["slopes"], prefix_lens=s["prefix"],
                           kv_layout=layout, lse=lse)
    return out, lse


def _plain_pages(s):
    ps, T = s["case"]["ps"], s["T"]
    old, new, count = s["old"].long(), s["new"].long(), s["count"].long()
    W = s["table"].shape[1]
    held = (old + ps - 1) // ps
    need = (old + new + ps - 1) // ps - held
    last = torch.cumsum(need, 0)
    cu = torch.cumsum(new, 0)
    ok = (last <= count) & (old + new <= W * ps) & (cu <= T)
    j = torch.arange(W, device="cuda")[None, :]
    at = (count - 1 - (last - need)[:, None] - (j - held[:, None])).clamp(0, s["free"].numel() - 1)
    fresh = (j >= held[:, None]) & (j < (held + need)[:, None]) & ok[:, None]
    table = torch.where(j < held[:, None], s["table"], torch.where(fresh, s["free"][at], -1))
    total = torch.where(ok, old + new, old)
    left = count - torch.where(ok, need, 0).sum()
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu, t, right=True)
    pos = old[b] + t - (cu - new)[b]
    slot = table[b, (pos // ps).clamp(max=W - 1)].long() * ps + pos % ps
    slot, pos = torch.where(ok[b], slot, -1), torch.where(ok[b], pos, -1)
    i32 = torch.int32
    return table.to(i32), total.to(i32), left.to(i32), cu.to(i32), slot.to(i32), pos.to(i32)


def _plain_rope(s):
    half = s["cos"].shape[1]
    p = s["pos"].long()[s["axis_t"]].T                     # [T, pairs]
    pair = torch.arange(half, device="cuda")
    c, d = s["cos"][p, pair][:, None], s["sin"][p, pair][:, None]

    def turn(x):
        a, b = x[..., :half].float(), x[..., half:].float()
        return torch.cat([a * c - b * d, b * c + a * d], -1).to(x.dtype)

    return turn(s["q"]), turn(s["k"])


def _plain_write(s):
    c = s["case"]
    ps, e4m3 = c["ps"], c["fmt"] == "e4m3"
    T, B = s["k"].shape[0], c["B"]
    qmax = torch.tensor(448.0 if e4m3 else 127.0, device="cuda")
    cu, old = s["cu"].long(), s["old"].long()
    begin = torch.cat([cu.new_zeros(1), cu[:-1]])
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu, t, right=True)
    pos = old[b] + t - begin[b]
    page, o = s["table"][b, pos // ps].long(), pos % ps
    row = s["table"].long().gather(1, (old // ps).clamp(max=s["table"].shape[1] - 1)[:, None])[:, 0]
    part = (old % ps > 0) & (cu > begin)                   # a partly filled page is appended to
    row = torch.where(part, row, torch.zeros_like(row))

    def code(x):
        return x.to(torch.float8_e4m3fn).view(torch.uint8) if e4m3 else x.round().to(torch.int8)

    def value(x):
        return x.view(torch.float8_e4m3fn).float() if e4m3 else x.float()

    for name in ("k", "v"):
        x, pool, scale = s[name].float(), s[name + "_pool"], s[name + "_scale"]
        nhd = pool.transpose(1, 2) if c["hnd"] else pool
        P, H = scale.shape
        top = torch.full((P, H), -1.0, device="cuda")
        top.scatter_reduce_(0, page[:, None].expand(T, H), x.abs().amax(-1), "amax")
        keeps = torch.zeros(P, dtype=torch.bool, device="cuda")
        keeps[row[part]] = True
        fresh = top / qmax
        now = torch.where(keeps[:, None], torch.maximum(fresh, scale), fresh)
        now = torch.where(top >= 0, now, scale)
        # the codes that a grown page keeps, in units of its new scale
        was = nhd[row]
        v = value(was.contiguous()) * scale[row][:, None, :, None]
        n = now[row][:, None, :, None]
        again = code(torch.where(n > 0, v / n, torch.zeros_like(v)))
        change = part[:, None] & (torch.arange(ps, device="cuda")[None, :] < (old % ps)[:, None])
        change = change[:, :, None] & (now[row] > scale[row])[:, None, :]
        put = torch.where(change[..., None], again, was)
        nhd[row[part]] = put[part]
        n = now[page][:, :, None]
        nhd[page, o] = code(torch.where(n > 0, x / n, torch.zeros_like(x)))
        scale.copy_(now)
    return _values(s["k_pool"]), _values(s["v_pool"]), s["k_scale"], s["v_scale"]


def _plain_attend(s):
    c = s["case"]
    B, Hq, Hkv, D, ps = c["B"], c["Hq"], c["Hkv"], c["D"], c["ps"]
    G, W, n = Hq // Hkv, s["W"], s["max_new"]
    T = s["q"].shape[0]
    cu, total = s["cu"].long(), s["total"].long()
    begin = torch.cat([cu.new_zeros(1), cu[:-1]])
    bt = s["table"][:, :W].long().clamp(min=0)

    def gather(name):
        x = s[name + "_pool"][bt]                          # [B, W, ps, H, D] (HND: [B, W, H, ps, D])
        x = x.view(torch.float8_e4m3fn).float() if c["fmt"] == "e4m3" else x.float()
        sc = s[name + "_scale"][bt]                        # [B, W, H]
        if c["hnd"]:
            return x.mul_(sc[..., None, None]).permute(0, 2, 1, 3, 4).reshape(B, Hkv, W * ps, D)
        return x.mul_(sc[:, :, None, :, None]).permute(0, 3, 1, 2, 4).reshape(B, Hkv, W * ps, D)

    i = torch.arange(n, device="cuda")
    rows = (begin[:, None] + i).clamp(max=T - 1)           # [B, n]
    q = s["q"][rows].float().reshape(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    S = torch.matmul(q, gather("k").transpose(2, 3)).mul_(1.0 / math.sqrt(D)).view(B, Hkv, G, n, W * ps)
    if c["cap"]:
        S = torch.tanh(S.div_(c["cap"])).mul_(c["cap"])
    j = torch.arange(W * ps, device="cuda")
    at = (total - (cu - begin))[:, None] + i               # position of each query
    if s["slopes"] is not None:
        S += (s["slopes"].view(Hkv, G)[None, :, :, None, None]
              * (j - at[..., None])[:, None, None].float())
    hi = at + 1
    if s["prefix"] is not None:
        hi = torch.maximum(hi, s["prefix"].long()[:, None])
    see = j < torch.minimum(hi, total[:, None])[..., None]
    if c["window"]:
        see &= j >= (at + 1 - c["window"])[..., None]
    S.masked_fill_(~see[:, None, None], -math.inf)
    m = S.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    S = S.sub_(m).exp_()
    l = S.sum(-1, keepdim=True)
    O = torch.matmul(S.view(B, Hkv, G * n, W * ps), gather("v")).view(B, Hkv, G, n, D)
    O = torch.where(l > 0, O / l, torch.zeros_like(O))
    lse = (m + torch.log(l))[..., 0]
    b = torch.searchsorted(cu, torch.arange(T, device="cuda"), right=True)
    r = torch.arange(T, device="cuda") - begin[b]
    O = O.permute(0, 3, 1, 2, 4)[b, r].reshape(T, Hq, D).to(s["q"].dtype)
    return O, lse.permute(0, 3, 1, 2)[b, r].reshape(T, Hq).contiguous()


# ------------------------------------------------------- the definitions in 64 bits

def _e4m3_values():
    """What each E4M3 code stands for: 4 exponent bits with bias 7, 3 mantissa bits."""
    v = []
    for c in range(256):
        e, f, sign = (c >> 3) & 15, c & 7, -1.0 if c & 128 else 1.0
        v.append(math.nan if e == 15 and f == 7 else
                 sign * (f / 8.0 * 2.0 ** -6 if e == 0 else (1 + f / 8.0) * 2.0 ** (e - 7)))
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def exact(case, seed):
    op = case["op"]
    if op == "pages":
        return None                                        # whole numbers only
    s = prepare(case, seed)
    f64 = torch.float64
    if op == "rope":
        half = case["D"] // 2
        outs = []
        for x in (s["q"], s["k"]):
            z = torch.complex(x[..., :half].to(f64), x[..., half:].to(f64))
            w = torch.empty((case["T"], half), dtype=torch.complex128, device="cuda")
            for i, a in enumerate(_pair_axis(case)):
                at = s["pos"][a].long()
                w[:, i] = torch.complex(s["cos"][at, i].to(f64), s["sin"][at, i].to(f64))
            z = z * w[:, None]
            outs.append(torch.cat([z.real, z.imag], -1))
        return tuple(outs)
    old, new = _lens(case)
    ps, Hkv, D = case["ps"], case["Hkv"], case["D"]
    code = _e4m3_values() if case["fmt"] == "e4m3" else None

    def number(x):
        return code[x.long()] if code is not None else x.to(f64)

    table = s["table"].tolist()
    if op == "write":
        qmax = 448.0 if code is not None else 127.0
        outs = []
        pos_codes = torch.sort(code[:127])[0] if code is not None else None
        mids = (pos_codes[1:] + pos_codes[:-1]) / 2 if code is not None else None

        def nearest(x):
            if code is None:
                return torch.round(x).clamp(-127, 127)
            a = x.abs()
            n = torch.searchsorted(mids, a.contiguous())
            tie = (n < 126) & (mids[n.clamp(max=125)] == a)
            n = torch.where(tie & (n % 2 == 1), n + 1, n)   # ties to the even code
            return torch.copysign(pos_codes[n], x)

        scales = []
        for name in ("k", "v"):
            pool, scale = s[name + "_pool"], s[name + "_scale"].clone()
            vals = number(pool.transpose(1, 2) if case["hnd"] else pool)
            t0 = 0
            for b in range(case["B"]):
                x = s[name][t0:t0 + new[b]].to(f64)
                t0 += new[b]
                p = old[b]
                while p < old[b] + new[b]:
                    pg, o0 = table[b][p // ps], p % ps
                    n = min(ps - o0, old[b] + new[b] - p)
                    y = x[p - old[b]:p - old[b] + n]       # [n, H, D]
                    sc = (y.abs().amax((0, 2)) / qmax).float()
                    if o0:
                        sc = torch.maximum(sc, scale[pg])
                        up = (sc > scale[pg])[None, :, None]
                        kept = vals[pg, :o0] * scale[pg].to(f64)[None, :, None]
                        vals[pg, :o0] = torch.where(
                            up, nearest(kept / sc.to(f64).clamp(min=1e-300)[None, :, None]), vals[pg, :o0])
                    d = sc.to(f64)[None, :, None]
                    vals[pg, o0:o0 + n] = torch.where(d > 0, nearest(y / d.clamp(min=1e-300)), 0 * y)
                    scale[pg] = sc
                    p += n
            outs.append(vals.transpose(1, 2) if case["hnd"] else vals)
            scales.append(scale.to(f64))
        return outs[0], outs[1], scales[0], scales[1]
    G, Hq = case["Hq"] // Hkv, case["Hq"]
    outs, lses, t0 = [], [], 0
    slopes = s["slopes"].to(f64) if s["slopes"] is not None else None
    for b in range(case["B"]):
        L, n = old[b] + new[b], new[b]
        pg = torch.tensor(table[b][:_pages(L, ps)], device="cuda")
        kv = []
        for name in ("k", "v"):
            x = number(s[name + "_pool"][pg]) * (
                s[name + "_scale"][pg].to(f64)[:, :, None, None] if case["hnd"]
                else s[name + "_scale"][pg].to(f64)[:, None, :, None])
            x = x.transpose(1, 2) if case["hnd"] else x
            kv.append(x.reshape(-1, Hkv, D)[:L])
        q = s["q"][t0:t0 + n].to(f64)
        t0 += n
        i = torch.arange(n, device="cuda")[:, None] + old[b]
        j = torch.arange(L, device="cuda")[None, :]
        see = (j <= i) | (j < min(case["prefix"], L))
        if case["window"]:
            see &= j > i - case["window"]
        o = torch.zeros((n, Hq, D), dtype=f64, device="cuda")
        lse = torch.empty((n, Hq), dtype=f64, device="cuda")
        for h in range(Hq):
            x = q[:, h] @ kv[0][:, h // G].T / math.sqrt(D)
            if case["cap"]:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if slopes is not None:
                x = x + slopes[h] * (j - i)
            x = x.masked_fill(~see, -math.inf)
            lse[:, h] = torch.logsumexp(x, -1)
            p = torch.exp(x - lse[:, h:h + 1]).nan_to_num(0.0)
            o[:, h] = p @ kv[1][:, h // G]
        outs.append(o)
        lses.append(lse)
    return torch.cat(outs), torch.cat(lses)
