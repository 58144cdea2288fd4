"""One serving step over a page-scaled 8-bit cache: page assignment, rotary
positions with several axes, the cache write and the attention that reads it.

Test infrastructure only (see oracle/__init__.py).  Written as loops over
requests, pages and rows, from the definitions; attention in float64, the
quantiser in the float32 steps that fix its codes.
"""
import numpy as np

from . import e4m3

F32 = np.float32


# ------------------------------------------------------------ page assignment

def assign_pages(new_lens, seqlens, block_table, free_pages, free_count, page_size, num_tokens):
    """Returns (block_table, seqlens, free_count, cu, slots, positions, refused)."""
    B, W = block_table.shape
    table, lens = block_table.copy(), seqlens.copy()
    slots = np.full(num_tokens, -1, np.int32)
    pos = np.full(num_tokens, -1, np.int32)
    cu = np.zeros(B, np.int32)
    refused = []
    demand = taken = t = 0
    for b in range(B):
        n, L = int(new_lens[b]), int(seqlens[b])
        held = -(-L // page_size)
        table[b, max(0, held):] = -1
        if n < 0 or L < 0 or L + n > W * page_size:
            refused.append(b)
            if L < 0 or L > W * page_size:
                table[b] = block_table[b]
            t += max(n, 0) if L >= 0 else 0
            cu[b] = min(t, num_tokens)
            continue
        need = -(-(L + n) // page_size) - held
        first, demand = demand, demand + need
        if t + n > num_tokens or (need > 0 and demand > free_count):
            refused.append(b)
        else:
            for i in range(need):
                table[b, held + i] = free_pages[free_count - 1 - (first + i)]
            for k in range(n):
                p = L + k
                slots[t + k] = table[b, p // page_size] * page_size + p % page_size
                pos[t + k] = p
            lens[b] = L + n
            taken += need
        t += n
        cu[b] = min(t, num_tokens)
    return table, lens, free_count - taken, cu, slots, pos, refused


# ------------------------------------------------------------ rotary positions

def rope_axes(x, positions, pair_axis, cos, sin, inverse=False):
    """x float32 [T, H, D] -> the rotated float32 values (before the rounding
    to the output type), products and sums rounded one by one."""
    x = np.asarray(x, F32)
    y = x.copy()
    half = len(pair_axis)
    for i, a in enumerate(pair_axis):
        p = positions[a]
        c, s = cos[p, i].astype(F32)[:, None], sin[p, i].astype(F32)[:, None]
        if inverse:
            s = -s
        u, w = x[..., i], x[..., i + half]
        y[..., i] = (u * c).astype(F32) - (w * s).astype(F32)
        y[..., i + half] = (w * c).astype(F32) + (u * s).astype(F32)
    return y


# ------------------------------------------------------------------- the cache

def decode(codes):
    return e4m3.decode(codes).astype(np.float64) if codes.dtype == np.uint8 else codes.astype(np.float64)


def _encode(x, fmt):
    if fmt == "e4m3":
        return e4m3.encode_rne_satfinite(x)
    return np.clip(np.rint(x), -127, 127).astype(np.int8)


def write_page8(k, v, cu, start_pos, block_table, pools, scales, fmt):
    """k, v float32 [T, H, D]; pools (k, v) [P, ps, H, D] and scales (k, v)
    [P, H], updated in place.  A sequence that starts at -1 is not written."""
    ps = pools[0].shape[1]
    qmax = F32(448.0 if fmt == "e4m3" else 127.0)
    for x, pool, scale in zip((k, v), pools, scales):
        t = 0
        for b in range(len(cu)):
            if start_pos[b] < 0:       # a refused request
                t = int(cu[b])
                continue
            p, end = int(start_pos[b]), int(start_pos[b]) + int(cu[b]) - t
            while p < end:
                pg, o = int(block_table[b, p // ps]), p % ps
                n = min(ps - o, end - p)
                for h in range(pool.shape[2]):
                    y = x[t:t + n, h].astype(F32)
                    s = F32(np.abs(y).max()) / qmax
                    if o:
                        was = scale[pg, h]
                        s = max(was, s)
                        if s > was:
                            kept = (decode(pool[pg, :o, h]).astype(F32) * was).astype(F32)
                            pool[pg, :o, h] = _encode((kept / s).astype(F32), fmt)
                    pool[pg, o:o + n, h] = _encode((y / s).astype(F32) if s > 0 else 0 * y, fmt)
                    scale[pg, h] = s
                t += n
                p += n


def attend_page8(q, pools, scales, block_table, cu, lens, sm_scale, causal=True, cap=0.0, window=0,
                 slopes=None, prefix=None, skip_page=None, flush=None):
    """q float [T, Hq, D]; returns float64 (o [T, Hq, D], lse [T, Hq]).  flush
    (float64 [T, Hq, D]) receives max_j (p_j s_j) * sum_j |code_j|, s_j and
    code_j the value's scale and code."""
    T, Hq, D = q.shape
    ps, H = pools[0].shape[1], pools[0].shape[2]
    o = np.zeros((T, Hq, D))
    lse = np.full((T, Hq), -np.inf)
    t0 = 0
    for b in range(len(cu)):
        n, L = int(cu[b]) - t0, int(lens[b])
        pg = block_table[b, :-(-L // ps)]
        ok = np.ones(L, bool)
        if skip_page is not None:
            ok = np.repeat(pg != skip_page, ps)[:L]
            pg = np.where(pg != skip_page, pg, 0)
        S = np.repeat(scales[1][pg].astype(np.float64), ps, axis=0)[:L]
        C = np.abs(decode(pools[1][pg])).reshape(-1, H, D)[:L]
        K, V = (np.asarray(decode(p[pg]) * s[pg].astype(np.float64)[:, None, :, None]).reshape(-1, H, D)[:L]
                for p, s in zip(pools, scales))
        j = np.arange(L)
        for i in range(n):
            at = L - n + i
            see = ok.copy()
            if causal:
                see &= (j <= at) | (j < (int(prefix[b]) if prefix is not None else 0))
            if window:
                see &= j > at - window
            if not see.any():
                continue
            for h in range(Hq):
                x = sm_scale * (K[see, h * H // Hq] @ q[t0 + i, h].astype(np.float64))
                if cap:
                    x = cap * np.tanh(x / cap)
                if slopes is not None:
                    x = x + float(slopes[h]) * (j[see] - at)
                m = x.max()
                e = np.exp(x - m)
                o[t0 + i, h] = e @ V[see, h * H // Hq] / e.sum()
                if flush is not None:
                    flush[t0 + i, h] = ((e * S[see, h * H // Hq]).max() / e.sum()
                                        * C[see, h * H // Hq].sum(0))
                lse[t0 + i, h] = m + np.log(e.sum())
        t0 += n
    return o, lse
