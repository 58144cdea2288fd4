"""The paged cache in 4 bits: its codes, the write with the rotation on the
way, the pages' key bounds, the choice of pages and the attention.

Test infrastructure only (see oracle/__init__.py).  Written as loops over
requests, pages and rows, from the definitions; the quantiser in the float32
steps that fix its codes, bounds and scores in whole numbers, attention in
float64.

A pool is uint8 [P, H, ps / 16, 9 D]: 16 tokens' rows of D / 2 bytes of E2M1
codes (1 sign, 2 exponent, 1 mantissa bit; even channels in the low half of a
byte), then 16 rows of D / 16 E4M3 scales.
"""
import numpy as np

from . import e4m3

F32 = np.float32
#: magnitude of every E2M1 code: exponent 0 is subnormal (0, 1/2), else (1 + m/2) 2^(e-1)
E2M1 = np.array([(c & 1) / 2 if c < 2 else (1 + (c & 1) / 2) * 2.0 ** ((c >> 1) - 1) for c in range(8)])


def encode_e2m1(x):
    """Nearest code of each float (not NaN), ties to the even one, saturating."""
    a = np.abs(np.asarray(x, np.float64))
    mid = (E2M1[1:] + E2M1[:-1]) / 2
    n = np.searchsorted(mid, a)                       # mid[n - 1] < a <= mid[n]
    tie = (n < 7) & (mid[np.minimum(n, 6)] == a) & (n % 2 == 1)
    return (n + tie).astype(np.uint8) | (np.signbit(x).astype(np.uint8) << 3)


def encode(x):
    """float32 [..., D] -> codes [..., D] and scales [..., D / 16]."""
    g = np.asarray(x, F32).reshape(x.shape[:-1] + (-1, 16))
    bad = ~np.isfinite(g).all(-1)
    g = np.where(bad[..., None], F32(0), g)
    scale = e4m3.encode_rne_satfinite((np.abs(g).max(-1) / F32(6)).astype(F32))
    s = e4m3.decode(scale).astype(F32)[..., None]
    y = np.where(s > 0, g / np.where(s > 0, s, F32(1)), F32(0)).astype(F32)
    codes = encode_e2m1(y)
    codes[np.broadcast_to((s == 0) | bad[..., None], codes.shape)] = 0
    return codes.reshape(x.shape), np.where(bad, np.uint8(0x7F), scale)


def value(codes, scales):
    """float64 values of codes [..., D] and scales [..., D / 16]."""
    x = np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]
    return x * np.repeat(e4m3.decode(scales), 16, axis=-1)


def rows_of(pool):
    """(codes [P, H, ps, D], scales [P, H, ps, D / 16]) of a pool."""
    P, H, nb, W = pool.shape
    D = W // 9
    b = pool[..., :8 * D].reshape(P, H, nb * 16, D // 2)
    codes = np.stack([b & 15, b >> 4], -1).reshape(P, H, nb * 16, D)
    return codes, pool[..., 8 * D:].reshape(P, H, nb * 16, D // 16).copy()


def pool_of(codes, scales):
    P, H, ps, D = codes.shape
    b = (codes[..., 0::2] | codes[..., 1::2] << 4).reshape(P, H, ps // 16, 8 * D)
    return np.concatenate([b, scales.reshape(P, H, ps // 16, D)], -1).astype(np.uint8)


def rotate(x, pos, cos, sin):
    """x float32 [T, H, D]: pairs (i, i + R / 2), products and sums rounded one by one."""
    if cos is None:
        return np.asarray(x, F32)
    half = cos.shape[1]
    y = np.array(x, F32)
    c, s = cos[pos][:, None].astype(F32), sin[pos][:, None].astype(F32)
    u, w = y[..., :half].copy(), y[..., half:2 * half].copy()
    y[..., :half] = (u * c).astype(F32) - (w * s).astype(F32)
    y[..., half:2 * half] = (w * c).astype(F32) + (u * s).astype(F32)
    return y


def bounds_of(codes, scales):
    """(int8 [2, D], scale) of one page and head's tokens [n, D]."""
    if (scales & 0x7F == 0x7F).any():
        return np.zeros((2, codes.shape[1]), np.int8), F32(np.inf)
    x = np.rint(value(codes, scales) * 1024).astype(np.int64)
    lo, hi = x.min(0), x.max(0)
    e = 0
    while max(abs(lo).max(), abs(hi).max()) > 127 * 2 ** e:
        e += 1
    return np.stack([lo // 2 ** e, -(-hi // 2 ** e)]).astype(np.int8), F32(2.0 ** (e - 10))


def write(k, v, cu, start, table, pools, cos=None, sin=None, mul=(None, None), bounds=None, bscale=None):
    """k, v float32 [T, H, D]; pools (k, v), bounds, bscale updated in place."""
    ps = pools[0].shape[2] * 16
    rows = [rows_of(p) for p in pools]
    t = 0
    for b in range(len(cu)):
        s, n = int(start[b]), int(cu[b]) - t
        if s < 0:
            t = int(cu[b])
            continue
        for i in range(n):
            p = s + i
            pg, o = table[b, p // ps], p % ps
            for x, (codes, scales), m, turn in ((k, rows[0], mul[0], True), (v, rows[1], mul[1], False)):
                y = x[t + i][None].astype(F32)
                if turn:
                    y = rotate(y, np.array([p]), cos, sin)
                if m is not None:
                    y = (y / m[:, None]).astype(F32)
                c, sc = encode(y)
                codes[pg, :, o], scales[pg, :, o] = c[0], sc[0]
        if bounds is not None and n > 0:
            for page_no in range(s // ps, (s + n - 1) // ps + 1):
                pg, end = table[b, page_no], min(ps, s + n - page_no * ps)
                for h in range(bounds.shape[1]):
                    bounds[pg, h], bscale[pg, h] = bounds_of(rows[0][0][pg, h, :end], rows[0][1][pg, h, :end])
        t = int(cu[b])
    for p, r in zip(pools, rows):
        p[...] = pool_of(*r)


def tokens(pool, table_row, L, mul=None):
    """float64 [L, H, D]: a sequence's first L tokens."""
    ps = pool.shape[2] * 16
    codes, scales = rows_of(pool[table_row[:-(-L // ps)]])
    x = value(codes, scales).swapaxes(1, 2).reshape(-1, pool.shape[1], pool.shape[3] // 9)[:L]
    return x if mul is None else x * np.asarray(mul, np.float64)[:, None]


def select(q, bounds, bscale, table, cu, lens, ps, n, first=0, last=1, window=0, P=None):
    """q float [T, Hq, D] -> int32 [T, H, n] (rows behind the last sequence: -2)."""
    T, Hq, D = q.shape
    H = bounds.shape[1]
    G = Hq // H
    out = np.full((T, H, n), -2, np.int32)
    t0 = 0
    for b in range(len(cu)):
        rows, L = int(cu[b]) - t0, int(lens[b])
        for i in range(rows):
            at = L - rows + i
            out[t0 + i] = -1
            if at < 0 or L == 0:
                continue
            lo, hi = (max(0, at + 1 - window) // ps if window else 0), at // ps
            for h in range(H):
                x = q[t0 + i, h * G:h * G + G].astype(np.float64)
                a = np.abs(x).max()
                c = np.rint(x * 127 / a).astype(np.int64) if 0 < a < np.inf else np.zeros(x.shape, np.int64)
                scored = []
                for p in range(lo, hi + 1):
                    pg = table[b, p]
                    if pg < 0 or pg >= bounds.shape[0]:
                        continue
                    mn, mx = bounds[pg, h].astype(np.int64)
                    s = int(np.maximum(c * mn, c * mx).sum(1).max())
                    s = float(F32(F32(s) * bscale[pg, h])) if np.isfinite(bscale[pg, h]) else np.inf
                    sure = p - lo < first or hi - p < last
                    scored.append((not sure, -s, p))
                ids = sorted(p for _, _, p in sorted(scored)[:n])
                out[t0 + i, h, :len(ids)] = ids
        t0 += rows
    return out


def attend(q, pools, table, cu, lens, sm_scale, causal=True, cap=0.0, window=0, slopes=None, prefix=None,
           selected=None, mul=(None, None), bad_page=None, sizes=False):
    """float64 (o [T, Hq, D], lse [T, Hq]); with sizes also sum p |v| and max p *
    sum |v| of every output.  A listed page counts once for each time."""
    T, Hq, D = q.shape
    H, ps = pools[0].shape[1], pools[0].shape[2] * 16
    o, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    size, flush = np.zeros((T, Hq, D)), np.zeros((T, Hq, D))
    t0 = 0
    for b in range(len(cu)):
        n, L = int(cu[b]) - t0, int(lens[b])
        row = np.where(table[b] == bad_page, 0, table[b]) if bad_page is not None else table[b]
        K, V = (tokens(p, row, L, m) for p, m in zip(pools, mul))
        ok = np.ones(L, bool) if bad_page is None else np.repeat(table[b] != bad_page, ps)[:L]
        j = np.arange(L)
        for i in range(n):
            at = L - n + i
            see = ok.copy()
            if causal:
                see &= (j <= at) | (j < (int(prefix[b]) if prefix is not None else 0))
            if window:
                see &= j > at - window
            for h in range(Hq):
                times = see.astype(int)
                if selected is not None:
                    page = selected[t0 + i, h * H // Hq]
                    count = np.bincount(page[(page >= 0) & (page * ps < L)], minlength=L // ps + 1)
                    times = times * np.repeat(count, ps)[:L]
                at_j = np.repeat(j, times)
                if at_j.size == 0:
                    continue
                x = sm_scale * (K[at_j, h * H // Hq] @ q[t0 + i, h].astype(np.float64))
                if cap:
                    x = cap * np.tanh(x / cap)
                if slopes is not None:
                    x = x + float(slopes[h]) * (at_j - at)
                m = x.max()
                e = np.exp(x - m)
                v = V[at_j, h * H // Hq]
                o[t0 + i, h] = e @ v / e.sum()
                lse[t0 + i, h] = m + np.log(e.sum())
                if sizes:
                    size[t0 + i, h] = e @ np.abs(v) / e.sum()
                    flush[t0 + i, h] = np.abs(v).sum(0) / e.sum()
        t0 += n
    return (o, lse, size, flush) if sizes else (o, lse)
