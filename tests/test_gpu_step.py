"""GPU parity of the serving step on the device: page assignment, rotary
axes, the page-scaled 8-bit cache write, attention over it, and the four of
them together, against oracle/step.py.

Tolerances of the attention outputs.  o is rounded once to its type (half a
step, eps/2 relative), every P to f16 (2^-11 relative to its own p |v|), and
a score's float32 error d <= 2^-11 scales p by e^d, so
|got - want| <= eps/2 |want| + 2^-10 sum_j p_j |v_j| (1 + eps); the sum is
the oracle's output for |v|.  f16 has an end: P = 2^7 ... 2^15 for the key
with the largest weight w = p s (s its value's scale), and what rounds to a
multiple of 2^-24 is off by up to 2^-25 = 2^-32 of that P, for each key j on
its code c_j: another 2^-32 max_j (p_j s_j) sum_j |c_j|, which counts where the
heaviest keys have zeros in a dimension.  Scores: float32 sums of D exact products and a
handful of float32 operations, so the lse is within 2^-17 (1 + max |x|),
max |x| bounded by the largest |lse| of a test plus its spread."""
import numpy as np
import pytest
import torch

from oracle import rope as orope
from oracle import step

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


@pytest.fixture
def err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------ page assignment

def _assign_case(seed, B, W, ps, hi, new_hi, free):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, min(hi, W * ps) + 1, B).astype(np.int32)
    new = np.minimum(rng.integers(0, new_hi + 1, B), W * ps - lens).astype(np.int32)
    held = -(-lens // ps)
    perm = rng.permutation(int(held.sum()) + free + 3).astype(np.int32)
    table = np.full((B, W), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = perm[at:at + held[b]]
        at += held[b]
    pages = np.zeros(free + 5, np.int32)
    pages[:free] = perm[at:at + free]
    return new, lens, table, pages, free, len(perm)


@pytest.mark.parametrize("B,W,ps,hi,new_hi,free,pad", [
    (1, 1, 16, 0, 1, 1, 0), (1, 9, 1, 3, 5, 20, 3), (64, 513, 16, 8000, 1, 70, 0),
    (7, 40, 48, 900, 300, 60, 100), (256, 170, 16, 2048, 512, 9000, 5), (1025, 3, 16, 40, 1, 700, 9),
    (8192, 2, 7, 9, 3, 9000, 1), (33, 20, 16, 200, 60, 40, 0), (5, 6, 16, 80, 0, 4, 2)])
@pytest.mark.parametrize("in_place", [False, True])
def test_assign_pages(lib, err, B, W, ps, hi, new_hi, free, pad, in_place):
    new, lens, table, pages, count, P = _assign_case(B + W, B, W, ps, hi, new_hi, free)
    T = int(new.sum()) + pad
    want = step.assign_pages(new, lens, table, pages, count, ps, T)
    d = [i32(x) for x in (new, lens, table, pages, [count])]
    kw = dict(block_table_out=d[2], seqlens_out=d[1], free_count_out=d[4]) if in_place else {}
    got = lib.assign_pages(*d, ps, P, T, error_word=err, **kw)
    for g, w, name in zip(got, want, ("table", "lens", "count", "cu", "slots", "positions")):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1)), name
    assert int(err) == (lib.DEV_ERR_NO_PAGES if want[6] else 0)
    if not in_place:   # inputs are as they were
        for x, y in zip(d, (new, lens, table, pages, [count])):
            assert np.array_equal(x.cpu().numpy(), np.asarray(y))


def test_assign_pages_refuses_what_does_not_fit(lib, err):
    """Too long for its row, tokens past num_tokens, negative lengths, a
    count outside the list, a bad page id on the stack."""
    table = np.array([[4, -1], [5, -1], [6, 7], [-1, -1]], np.int32)
    args = lambda new, lens, count=2, pages=(1, 2): (i32(new), i32(lens), i32(table), i32(list(pages)), i32([count]))  # noqa: E731
    want = step.assign_pages(np.array([1, 40, 1, 2]), np.array([3, 16, 17, 0], np.int32), table,
                             np.array([1, 2]), 2, 16, 44)
    got = lib.assign_pages(*args([1, 40, 1, 2], [3, 16, 17, 0]), 16, 8, 44, error_word=err)
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))
    assert int(err) == lib.DEV_ERR_BAD_LENGTH
    err.zero_()
    got = lib.assign_pages(*args([2, 3, 2, 1], [3, 16, 17, 0]), 16, 8, 6, error_word=err)
    assert got[3].tolist() == [2, 5, 6, 6] and got[1].tolist() == [5, 19, 17, 0]
    assert got[4].tolist() == [67, 68, 32, 33, 34, -1] and int(err) == lib.DEV_ERR_BAD_LENGTH
    err.zero_()
    got = lib.assign_pages(*args([-1, 0, 1, 1], [3, -5, 17, 0]), 16, 8, 4, error_word=err)
    assert got[1].tolist() == [3, -5, 18, 1] and got[3].tolist() == [0, 0, 1, 2]
    assert got[0].tolist() == [[4, -1], [5, -1], [6, 7], [2, -1]] and int(err) == lib.DEV_ERR_BAD_LENGTH
    err.zero_()
    got = lib.assign_pages(*args([0, 0, 0, 1], [3, 16, 17, 0], count=3), 16, 8, 1, error_word=err)
    assert got[1].tolist() == [3, 16, 17, 0]
    assert int(err) == lib.DEV_ERR_BAD_LENGTH | lib.DEV_ERR_NO_PAGES
    err.zero_()
    got = lib.assign_pages(*args([0, 0, 0, 1], [3, 16, 17, 0], pages=(1, 8)), 16, 8, 1, error_word=err)
    assert got[4].tolist() == [-1] and got[0][3].tolist() == [-1, -1] and int(err) == lib.DEV_ERR_BAD_PAGE


def test_assign_pages_start_pos_may_take_the_lengths_place(lib, err):
    """start_pos over seqlens, the grown lengths elsewhere: every length is read
    before its place is written, a refused request's too."""
    new, lens, table, pages, count, P = _assign_case(40, 1500, 5, 16, 70, 30, 600)
    T = int(new.sum())
    want = step.assign_pages(new, lens, table, pages, count, 16, T)
    d = [i32(x) for x in (new, lens, table, pages, [count])]
    got = lib.assign_pages(*d, 16, P, T, error_word=err, start_pos=d[1])
    assert len(want[6]) > 100 and int(err) == lib.DEV_ERR_NO_PAGES
    for g, w in zip(got, want):
        assert np.array_equal(g.cpu().numpy().reshape(-1), np.asarray(w).reshape(-1))
    assert np.array_equal(d[1].cpu().numpy(), np.where(np.isin(np.arange(1500), want[6]), -1, lens))


# ------------------------------------------------------------ rotary positions

@pytest.mark.parametrize("T,Hq,Hkv,D,sections,inter,dtype,fused", [
    (1, 1, 1, 64, (32,), False, "bf16", False), (5, 28, 4, 128, (16, 24, 24), False, "bf16", True),
    (33, 3, 2, 80, (16, 12, 12), True, "f16", True), (130, 7, 1, 72, (9, 9), False, "f32", False),
    (3, 2, 3, 96, (10, 11), True, "bf16", True), (17, 5, 2, 128, (8, 8, 8, 8), False, "f32", True),
    (9, 1, 1, 10, (3,), False, "f16", False), (40, 2, 2, 256, (64, 32, 32), False, "bf16", False),
    (2000, 32, 8, 128, (24, 20, 20), True, "bf16", True)])
def test_rope_axes_bit_exact(lib, err, T, Hq, Hkv, D, sections, inter, dtype, fused):
    rng = np.random.default_rng(T)
    half, A = sum(sections), len(sections)
    dt = DT[dtype]
    x = torch.tensor(rng.standard_normal((T, Hq + 2 * Hkv, D)).astype(np.float32)).to(dt)
    dev = x.cuda()
    q, k = dev[:, :Hq], dev[:, Hq:Hq + Hkv]
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    cos, sin = lib.rope_table(1e4, 70, 2 * half)
    pos = rng.integers(0, 70, (A, T)).astype(np.int32)
    axis = lib.axis_sections(sections, interleaved=inter)
    assert sorted(axis) == sorted(sum(([a] * n for a, n in enumerate(sections)), []))
    for inverse in (False, True):
        gq, gk = lib.rope_axes(q, i32(pos), axis, cos, sin, k=k, inverse=inverse, error_word=err)
        for g, src in ((gq, x[:, :Hq]), (gk, x[:, Hq:Hq + Hkv])):
            w = step.rope_axes(src.float().numpy(), pos, axis, cos.cpu().numpy(), sin.cpu().numpy(), inverse)
            assert torch.equal(g.cpu(), torch.tensor(w).to(dt))
    only_q = lib.rope_axes(q, i32(pos), axis, cos, sin)
    ref = lib.rope_axes(q, i32(pos), axis, cos, sin, k=k)
    v = dev[:, Hq + Hkv:].clone()
    lib.rope_axes(q, i32(pos), axis, cos, sin, k=k, q_out=q, k_out=k)      # in place
    assert torch.equal(only_q, ref[0]) and torch.equal(q, ref[0]) and torch.equal(k, ref[1])
    assert torch.equal(dev[:, Hq + Hkv:], v) and int(err) == 0


def test_rope_axes_leaves_padding_and_reports_bad_positions(lib, err):
    cos, sin = lib.rope_table(1e4, 20, 64)
    q = torch.randn(4, 2, 64, device="cuda")
    out = torch.full_like(q, 7.0)
    pos = i32([[3, -1, 20, 19], [3, 5, 1, 2]])
    lib.rope_axes(q, pos, bytes([0, 1] * 16), cos, sin, q_out=out, error_word=err)
    assert (out[1:3] == 7.0).all() and (out[[0, 3]] != 7.0).any(dim=2).all()
    assert int(err) == lib.DEV_ERR_BAD_LENGTH
    err.zero_()
    lib.rope_axes(q, i32([[-1] * 4, [99] * 4]), bytes([0, 1] * 16), cos, sin, q_out=out, error_word=err)
    assert int(err) == 0
    one = i32([[1, 2, 3, 4]])
    a = lib.rope_axes(q, one.expand(3, 4), bytes([0] * 8 + [1] * 12 + [2] * 12), cos, sin)
    assert torch.equal(a, lib.rope_axes(q, one, bytes(32), cos, sin))


def test_rope_axes_inverse_is_the_gradient(lib):
    """For y = R(x) and a loss <w, y>, the gradient is R's transpose of w: the
    inverse rotation; also against differences (R is linear, so one step of any
    size gives the derivative up to float32 rounding)."""
    g = torch.Generator(device="cuda").manual_seed(1)
    cos, sin = lib.rope_table(1e4, 64, 64)
    pos = torch.randint(0, 64, (3, 11), generator=g, device="cuda").to(torch.int32)
    axis = lib.axis_sections((12, 10, 10))
    x, w, d = (torch.randn(11, 3, 64, generator=g, device="cuda") for _ in range(3))
    grad = lib.rope_axes(w, pos, axis, cos, sin, inverse=True).double()
    f = lambda z: (lib.rope_axes(z, pos, axis, cos, sin).double() * w.double()).sum()  # noqa: E731
    got, want = (grad * d.double()).sum(), (f(x + d) - f(x - d)) / 2
    # 2112 products of values below 6, each off by a few 2^-24
    assert abs(float(got - want)) < 2112 * 36 * 2.0 ** -22 / 8


# ------------------------------------------------------------------- the write

def _pool(P, ps, H, D, fmt, hnd, fill):
    shape = (P, H, ps, D) if hnd else (P, ps, H, D)
    return torch.full(shape, fill, dtype=torch.uint8 if fmt == "e4m3" else torch.int8, device="cuda")


def _nhd(pool, hnd):
    return (pool.transpose(1, 2) if hnd else pool).cpu().numpy().copy()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("lens,H,D,ps,dtype,hnd", [
    ([(0, 1)], 1, 64, 16, "bf16", False), ([(5, 30), (0, 0), (16, 16), (31, 2), (15, 1), (16, 1)], 3, 128, 16, "bf16", False),
    ([(40, 100), (0, 7), (47, 1)], 2, 64, 48, "f16", True), ([(100, 300), (0, 129)], 5, 128, 64, "bf16", True),
    ([(3, 1), (0, 700)], 1, 128, 1024, "f16", False), ([(200, 90)], 2, 64, 256, "bf16", False),
    ([(n, 1) for n in range(64)], 8, 128, 16, "bf16", False)])
def test_write_page8_bit_exact(lib, err, lens, H, D, ps, dtype, hnd, fmt):
    """A first write, then a second one that raises the scales of partly filled
    pages, lowers or keeps others: codes and scales equal the oracle's."""
    rng = np.random.default_rng(len(lens) + ps)
    W = max(-(-(a + n) // ps) for a, n in lens) + 1
    P = W * len(lens) + 2
    table = rng.permutation(P - 2)[:W * len(lens)].reshape(len(lens), W).astype(np.int32)
    fill = 0x7F if fmt == "e4m3" else 99
    kp, vp = _pool(P, ps, H, D, fmt, hnd, fill), _pool(P, ps, H, D, fmt, hnd, fill)
    ks, vs = torch.full((P, H), 5.0, device="cuda"), torch.full((P, H), 6.0, device="cuda")
    pools, scales = [_nhd(kp, hnd), _nhd(vp, hnd)], [ks.cpu().numpy(), vs.cpu().numpy()]
    for begin, n in (([0] * len(lens), [a for a, _ in lens]), ([a for a, _ in lens], [n for _, n in lens])):
        T = int(sum(n))
        if T == 0:
            continue
        x = rng.standard_normal((T + 3, 2 * H + 1, D)).astype(np.float32) * np.exp(rng.standard_normal((T + 3, 1, 1)))
        x[rng.integers(0, T, 3)] = 0.0
        x = torch.tensor(x.astype(np.float32)).to(DT[dtype])   # three rows behind the last sequence
        dev = x.cuda()
        cu = np.cumsum(n).astype(np.int32)
        lib.write_cache_page8(dev[:, :H], dev[:, H:2 * H], i32(cu), i32(table), kp, vp, ks, vs,
                              start_pos=i32(begin) if any(begin) else None,
                              kv_layout="HND" if hnd else "NHD", error_word=err)
        step.write_page8(x[:, :H].float().numpy(), x[:, H:2 * H].float().numpy(), cu, begin, table, pools, scales, fmt)
        assert np.array_equal(ks.cpu().numpy(), scales[0]) and np.array_equal(vs.cpu().numpy(), scales[1])
        # codes; E4M3's two zeros are one value
        for got, want in ((_nhd(kp, hnd), pools[0]), (_nhd(vp, hnd), pools[1])):
            same = got == want
            if fmt == "e4m3":
                same |= ((got | want) & 0x7F) == 0
            assert same.all()
    assert int(err) == 0


def test_write_page8_skips_bad_pages_and_lengths(lib, err):
    kp, vp = _pool(4, 16, 1, 64, "int8", False, 9), _pool(4, 16, 1, 64, "int8", False, 9)
    ks, vs = torch.full((4, 1), 5.0, device="cuda"), torch.full((4, 1), 5.0, device="cuda")
    x = torch.ones(40, 1, 64, device="cuda", dtype=torch.bfloat16)
    lib.write_cache_page8(x, x, i32([20, 40]), i32([[1, 4], [-1, 2]]), kp, vp, ks, vs, error_word=err)
    assert int(err) == lib.DEV_ERR_BAD_PAGE
    assert (kp[0] == 9).all() and (kp[3] == 9).all() and (kp[1] == 127).all()
    assert (kp[2, :4] == 127).all() and (kp[2, 4:] == 9).all() and ks[:, 0].tolist()[0::3] == [5.0, 5.0]
    err.zero_()   # positions past the row; rows past T
    lib.write_cache_page8(x, x, i32([20]), i32([[3, 0]]), kp, vp, ks, vs, start_pos=i32([30]), error_word=err)
    # slots 14, 15 join a page whose scale is 5: RNE(1 / 5) = 0
    assert int(err) == lib.DEV_ERR_BAD_LENGTH and (kp[3] == 9).all()
    assert (kp[0, :14] == 9).all() and (kp[0, 14:] == 0).all() and float(ks[0]) == 5.0
    err.zero_()
    before = kp.clone()
    lib.write_cache_page8(x, x, i32([50]), i32([[3, 0]]), kp, vp, ks, vs, error_word=err)
    assert int(err) == lib.DEV_ERR_BAD_LENGTH and torch.equal(kp, before)


# --------------------------------------------------------------- the attention

def _attend_case(seed, reqs, Hq, H, D, ps, fmt, dtype, hnd, slopes=False, prefix=None, size=1.0, pad=0):
    """reqs: (queries, cached tokens) per sequence.  Unused slots and pages hold
    NaN codes (E4M3); unused table entries -1."""
    rng = np.random.default_rng(seed)
    n_pages = [-(-L // ps) for _, L in reqs]
    P, W = sum(n_pages) + 2, max(n_pages + [1]) + 1
    perm = rng.permutation(P)
    table = np.full((len(reqs), W), -1, np.int32)
    at = 0
    for b, n in enumerate(n_pages):
        table[b, :n] = perm[at:at + n]
        at += n
    pools, scales = [], []
    for _ in range(2):
        if fmt == "e4m3":
            c = rng.integers(0, 256, (P, ps, H, D)).astype(np.uint8)
            c[(c & 0x7F) >= 0x7C] &= 0x87
        else:
            c = rng.integers(-127, 128, (P, ps, H, D)).astype(np.int8)
        used = np.zeros((P, ps), bool)
        for b, (_, L) in enumerate(reqs):
            for i in range(n_pages[b]):
                used[table[b, i], :min(ps, L - i * ps)] = True
        c[~used] = 0x7F if fmt == "e4m3" else -128
        unit = (20.0 if fmt == "e4m3" else 50.0)
        pools.append(c)
        scales.append((np.exp(rng.standard_normal((P, H))) / unit).astype(np.float32))
    T = sum(n for n, _ in reqs)
    q = torch.tensor((size * rng.standard_normal((T + pad, Hq, D))).astype(np.float32)).to(DT[dtype])
    c = dict(q=q, pools=pools, scales=scales, table=table, cu=np.cumsum([n for n, _ in reqs]).astype(np.int32),
             lens=np.array([L for _, L in reqs], np.int32), hnd=hnd, T=T,
             slopes=(2.0 ** (-8.0 * (np.arange(Hq) + 1) / Hq)).astype(np.float32) if slopes else None,
             prefix=np.array(prefix, np.int32) if prefix is not None else None)
    put = lambda p: torch.tensor(np.ascontiguousarray(p.swapaxes(1, 2)) if hnd else p).cuda()  # noqa: E731
    c["dev"] = dict(q=q.cuda(), kp=put(pools[0]), vp=put(pools[1]), ks=torch.tensor(scales[0]).cuda(),
                    vs=torch.tensor(scales[1]).cuda(), table=i32(table), cu=i32(c["cu"]), lens=i32(c["lens"]),
                    slopes=torch.tensor(c["slopes"]).cuda() if slopes else None,
                    prefix=i32(prefix) if prefix is not None else None)
    return c


def _run_attend(lib, c, err, max_q=0, out=None, lse=None, ws=None, **kw):
    d = c["dev"]
    return lib.attend_page8(d["q"], d["kp"], d["vp"], d["ks"], d["vs"], d["table"], d["cu"], d["lens"],
                            max_seqlen_q=max_q, alibi_slopes=d["slopes"], prefix_lens=d["prefix"],
                            kv_layout="HND" if c["hnd"] else "NHD", out=out, lse=lse, workspace=ws,
                            error_word=err, **kw)


def _check_attend(c, got, lse, causal=True, logit_cap=0.0, window=0, sm_scale=None, skip_page=None, rows=None):
    q = c["q"][:c["T"]].double().numpy()
    kw = dict(causal=causal, cap=logit_cap, window=window, slopes=c["slopes"], prefix=c["prefix"], skip_page=skip_page)
    scale = sm_scale or 1 / np.sqrt(q.shape[2])
    flush = np.zeros(q.shape)
    want, want_lse = step.attend_page8(q, c["pools"], c["scales"], c["table"], c["cu"], c["lens"], scale,
                                       flush=flush, **kw)
    mag = [c["pools"][0], c["pools"][1] & 0x7F if c["pools"][1].dtype == np.uint8 else np.abs(c["pools"][1])]
    size, _ = step.attend_page8(q, mag, c["scales"], c["table"], c["cu"], c["lens"], scale, **kw)
    eps = torch.finfo(c["q"].dtype).eps / 2
    g, l = f64(got)[:c["T"]], f64(lse)[:c["T"]]
    finite = bool(np.isfinite(g).all())
    assert finite
    tol = eps * np.abs(want) + 2.0 ** -10 * size * (1 + eps) + 2.0 ** -32 * flush + (2.0 ** -25 if c["q"].dtype == torch.float16 else 0)
    worst = float((np.abs(g - want) / (tol + 1e-300)).max()) if g.size else 0.0
    assert worst <= 1, worst
    same_empty = np.array_equal(np.isneginf(l), np.isneginf(want_lse))
    assert same_empty
    fin = np.isfinite(want_lse)
    spread = np.abs(want_lse[fin]).max() if fin.any() else 0.0
    off = float(np.abs(l[fin] - want_lse[fin]).max()) if fin.any() else 0.0
    assert off <= 2.0 ** -17 * (4 + 2 * spread), off


DECODE = [(1, 1), (1, 15), (1, 16), (1, 17), (1, 100), (1, 0), (1, 333), (1, 64)]
MIXED = [(1, 40), (5, 5), (0, 30), (3, 130), (20, 70), (2, 1), (7, 0), (1, 200)]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("Hq,H,D,ps,dtype,hnd", [
    (4, 1, 64, 16, "bf16", False), (32, 8, 128, 16, "bf16", False), (6, 2, 128, 48, "f16", True),
    (5, 5, 64, 64, "f16", False), (32, 2, 128, 32, "bf16", True), (40, 2, 64, 16, "bf16", False)])
@pytest.mark.parametrize("reqs", [DECODE, MIXED], ids=["decode", "mixed"])
def test_attend_page8(lib, err, reqs, Hq, H, D, ps, dtype, hnd, fmt):
    c = _attend_case(Hq + ps, reqs, Hq, H, D, ps, fmt, dtype, hnd, pad=2)
    out = torch.full_like(c["dev"]["q"], 7.0)
    lse = torch.full(out.shape[:2], 7.0, device="cuda")
    _run_attend(lib, c, err, max_q=max(n for n, _ in reqs), out=out, lse=lse)
    assert int(err) == 0 and (out[c["T"]:] == 7.0).all() and (lse[c["T"]:] == 7.0).all()
    _check_attend(c, out, lse)


@pytest.mark.parametrize("kw", [
    dict(logit_cap=20.0), dict(window=1), dict(window=33), dict(causal=False), dict(causal=False, window=20),
    dict(logit_cap=50.0, window=64, sm_scale=0.2), dict(sm_scale=3.0)], ids=str)
@pytest.mark.parametrize("slopes,prefix", [(False, None), (True, None), (False, [0, 50, 1, 90, 3, 9, 2, 10**9])])
def test_attend_page8_masks_caps_and_biases(lib, err, kw, slopes, prefix):
    for i, (fmt, dtype) in enumerate((("int8", "f16"), ("e4m3", "bf16"))):
        c = _attend_case(i, MIXED, 6, 2, (64, 128)[i], 16, fmt, dtype, bool(i), slopes=slopes, prefix=prefix)
        lse = torch.empty(c["q"].shape[:2], device="cuda")
        got = _run_attend(lib, c, err, lse=lse, **kw)
        _check_attend(c, got, lse, **kw)
    assert int(err) == 0


@pytest.mark.parametrize("reqs,Hq,H", [
    ([(1, 9000)], 4, 1), ([(1, 5000), (1, 3), (1, 7001)], 8, 2), ([(3, 4100)], 8, 8), ([(1, 300)] * 40, 16, 8),
    ([(1, 0)] * 3, 4, 1), ([(1, 31 * i % 97) for i in range(300)], 2, 1)])
def test_attend_page8_long_and_many(lib, err, reqs, Hq, H):
    """Runs that split one request, cover several, and cross empty ones."""
    c = _attend_case(len(reqs), reqs, Hq, H, 128, 16, "e4m3", "bf16", False)
    lse = torch.empty(c["q"].shape[:2], device="cuda")
    got = _run_attend(lib, c, err, max_q=max(n for n, _ in reqs), lse=lse)
    _check_attend(c, got, lse)
    assert int(err) == 0
    again = _run_attend(lib, c, err, max_q=max(n for n, _ in reqs))
    assert torch.equal(got, again)


TILES = [[(300, 300)], [(130, 700), (1, 50), (64, 64), (0, 9), (40, 300)], [(90, 1500)], [(200, 60), (33, 0), (30, 129)]]


@pytest.mark.parametrize("reqs", TILES, ids=["prompt", "mixed", "piece", "short_cache"])
@pytest.mark.parametrize("Hq,H,D,ps,fmt,dtype,hnd", [
    (2, 2, 128, 16, "e4m3", "bf16", False), (8, 2, 128, 64, "int8", "f16", True), (7, 1, 64, 48, "e4m3", "f16", False),
    (6, 2, 64, 128, "int8", "bf16", False)])
@pytest.mark.parametrize("kw,slopes,prefix", [
    (dict(), False, None), (dict(window=70), False, None), (dict(logit_cap=30.0), False, 100), (dict(causal=False), True, None),
    (dict(), True, None)], ids=["plain", "window", "cap_prefix", "full_bias", "bias"])
def test_attend_page8_many_rows(lib, err, reqs, Hq, H, D, ps, fmt, dtype, hnd, kw, slopes, prefix):
    """Sequences beside one another whose rows go in tiles of 128 and whose
    rows do not, runs that cut an item, rows before the first key."""
    c = _attend_case(Hq + len(reqs), reqs, Hq, H, D, ps, fmt, dtype, hnd, slopes=slopes,
                     prefix=[prefix] * len(reqs) if prefix else None, pad=3)
    out = torch.full_like(c["dev"]["q"], 7.0)
    lse = torch.full(out.shape[:2], 7.0, device="cuda")
    _run_attend(lib, c, err, max_q=max(n for n, _ in reqs), out=out, lse=lse, **kw)
    assert int(err) == 0 and (out[c["T"]:] == 7.0).all() and (lse[c["T"]:] == 7.0).all()
    _check_attend(c, out, lse, **kw)


def _attend_64bit(c, causal=True):
    """The attention of a case's sequences in float64 on the GPU, for sizes the
    oracle's loops are too slow for: (o, lse, sum_j p_j |v_j|)."""
    d, outs, t0 = c["dev"], [[], [], []], 0
    for b, (end, L) in enumerate(zip(c["cu"].tolist(), c["lens"].tolist())):
        n, pg = end - t0, torch.tensor(c["table"][b][:-(-L // c["pools"][0].shape[1])].astype(np.int64))
        kv = [torch.tensor(step.decode(p[pg]) * s[pg].astype(np.float64)[:, None, :, None]).cuda().flatten(0, 1)[:L]
              for p, s in zip(c["pools"], c["scales"])]
        q = d["q"][t0:end].double()
        at = torch.arange(n, device="cuda")[:, None] + L - n
        see = torch.arange(L, device="cuda")[None] <= at if causal else torch.ones(n, L, dtype=bool, device="cuda")
        for h in range(q.shape[1]):
            g = h * kv[0].shape[1] // q.shape[1]
            x = (q[:, h] @ kv[0][:, g].T / q.shape[2] ** 0.5).masked_fill(~see, -np.inf)
            lse = torch.logsumexp(x, -1)
            p = torch.exp(x - lse[:, None])
            for o, y in zip(outs, (p @ kv[1][:, g], lse, p @ kv[1][:, g].abs())):
                o.append(y)
        t0 = end
    H = d["q"].shape[1]
    return [torch.cat([torch.stack(o[i:i + H], 1) for i in range(0, len(o), H)]) for o in outs]


@pytest.mark.parametrize("reqs,Hq,H,D,fmt,dtype", [
    ([(1500, 5000)], 8, 8, 128, "e4m3", "bf16"), ([(700, 4100), (900, 2300), (1, 9000), (130, 130)], 28, 4, 128, "int8", "f16"),
    ([(2600, 2600)], 16, 4, 64, "int8", "bf16")])
@pytest.mark.parametrize("causal", [True, False])
def test_attend_page8_long_runs(lib, err, reqs, Hq, H, D, fmt, dtype, causal):
    """Every CTA gets dozens of key tiles: the rings wrap, running maxima move,
    and results do not depend on which warp is ahead (five times the same)."""
    c = _attend_case(11, reqs, Hq, H, D, 16, fmt, dtype, False)
    want, want_lse, size = _attend_64bit(c, causal)
    first = None
    for _ in range(5):
        lse = torch.empty(c["q"].shape[:2], device="cuda")
        got = _run_attend(lib, c, err, max_q=max(n for n, _ in reqs), lse=lse, causal=causal)
        eps = torch.finfo(c["q"].dtype).eps / 2
        # the tolerance of this file; all keys' codes and the largest weight bound its last term
        flush = 2.0 ** -32 * float(c["scales"][1].max()) * 448 * max(L for _, L in reqs)
        tol = eps * want.abs() + 2.0 ** -10 * size * (1 + eps) + flush + (2.0 ** -25 if dtype == "f16" else 0)
        worst = float(((got.double() - want).abs() / tol).max())
        assert worst <= 1, worst
        off = float((lse - want_lse).abs().max())
        assert off <= 2.0 ** -17 * (4 + 2 * float(want_lse.abs().max())), off
        first = got if first is None else first
        assert torch.equal(got, first)
    assert int(err) == 0


@pytest.mark.parametrize("reqs,Hq,H,D,fmt,dtype", [
    ([(40, 40)] * 60, 16, 8, 64, "int8", "f16"), ([(30, 45), (70, 64), (25, 1)] * 30, 8, 4, 128, "e4m3", "bf16")])
def test_attend_page8_segments_of_one_step(lib, err, reqs, Hq, H, D, fmt, dtype):
    """A CTA's steps are a new (item, kv head) each: the softmax warps are told
    of another one with every S, and take it for no other (ten times the same)."""
    c = _attend_case(12, reqs, Hq, H, D, 16, fmt, dtype, False)
    first = None
    for _ in range(10):
        lse = torch.empty(c["q"].shape[:2], device="cuda")
        got = _run_attend(lib, c, err, max_q=max(n for n, _ in reqs), lse=lse)
        if first is None:
            first = got
            _check_attend(c, got, lse)
        assert torch.equal(got, first) and int(err) == 0


@pytest.mark.parametrize("reqs", [[(130, 700)], [(300, 900), (40, 333), (1, 500)], [(1, 400), (3, 777)]], ids=["piece", "mixed", "split"])
@pytest.mark.parametrize("fmt,dtype,ps", [("e4m3", "bf16", 16), ("int8", "f16", 32)])
@pytest.mark.parametrize("entry", ["none", "junk"])
def test_attend_page8_pages_before_the_window(lib, err, reqs, fmt, dtype, ps, entry):
    """Pages that lie before every row's window may be given back: their entries
    are -1, or those of a page that holds NaN codes and scales, and are not read."""
    window = 70
    c = _attend_case(15, reqs, 4, 2, 128, ps, fmt, dtype, False)
    junk = sorted(set(range(c["pools"][0].shape[0])) - set(c["table"].reshape(-1).tolist()))[0]
    c["dev"]["ks"][junk] = float("nan")
    c["dev"]["vs"][junk] = float("inf")
    for b, (n, L) in enumerate(reqs):
        first = max(0, L - n + 1 - window) // ps
        assert first > 0
        c["dev"]["table"][b, :first] = -1 if entry == "none" else junk
    lse = torch.empty(c["q"].shape[:2], device="cuda")
    got = _run_attend(lib, c, err, max_q=max(n for n, _ in reqs), lse=lse, window=window)
    assert int(err) == 0
    _check_attend(c, got, lse, window=window)


def test_attend_page8_forms_agree(lib, err):
    """The bound on a sequence's queries picks the kernels, never the result's
    meaning: without one, and with one that is too small to be a bound."""
    c = _attend_case(3, [(50, 400), (3, 90)], 8, 2, 128, 16, "e4m3", "bf16", False)
    for max_q in (0, 50, 1000, 3):
        lse = torch.empty(c["q"].shape[:2], device="cuda")
        got = _run_attend(lib, c, err, max_q=max_q, lse=lse)
        _check_attend(c, got, lse)
        assert torch.equal(got, _run_attend(lib, c, err, max_q=max_q))
    assert int(err) == 0


@pytest.mark.parametrize("size", [1e-30, 1e-3, 300.0, 1e30])
def test_attend_page8_query_and_value_sizes(lib, err, size):
    """Query rows of any bf16 size (the softmax scale makes up for it), value
    scales that differ by 2^40 between pages, and zero scales."""
    c = _attend_case(2, [(1, 100), (2, 60)], 4, 2, 64, 16, "int8", "bf16", False, size=size)
    rng = np.random.default_rng(0)
    for x, name in ((c["scales"][1], "vs"),):
        x *= (2.0 ** rng.integers(-20, 21, x.shape)).astype(np.float32)
        c["dev"][name].copy_(torch.tensor(x))
    page = int(c["table"][0, 1])
    for p, s, pn, sn in ((c["pools"][0], c["scales"][0], "kp", "ks"), (c["pools"][1], c["scales"][1], "vp", "vs")):
        p[page] = 0
        s[page] = 0.0
        c["dev"][pn][page] = 0
        c["dev"][sn][page] = 0.0
    lse = torch.empty(c["q"].shape[:2], device="cuda")
    scale = 0.125 / size
    if not np.isfinite(np.float32(scale)) or scale < 1e-30:
        scale = 1e-30
    got = _run_attend(lib, c, err, lse=lse, sm_scale=scale)
    _check_attend(c, got, lse, sm_scale=float(np.float32(scale)))


@pytest.mark.parametrize("reqs,max_q", [([(1, 100), (2, 60), (1, 20)], 2), ([(90, 200), (1, 70)], 90)], ids=["split", "tiles"])
@pytest.mark.parametrize("fmt,dtype", [("int8", "f16"), ("e4m3", "bf16")])
def test_attend_page8_value_scales_of_zero(lib, err, reqs, max_q, fmt, dtype):
    """Pages whose value scale is 0 add nothing, whatever their codes, and lower
    nobody's weights: the others' scales are 2^-25 to 2^-30 of a usual one."""
    c = _attend_case(14, reqs, 4, 2, 64, 16, fmt, dtype, False)
    vs = c["scales"][1]
    vs *= (2.0 ** -np.random.default_rng(1).integers(25, 31, vs.shape)).astype(np.float32)
    if dtype == "f16":      # values that f16 holds
        vs *= np.float32(2.0 ** 20)
    vs[c["table"][0, 1]] = 0.0
    vs[c["table"][1, 0], 1] = 0.0
    c["dev"]["vs"].copy_(torch.tensor(vs))
    lse = torch.empty(c["q"].shape[:2], device="cuda")
    got = _run_attend(lib, c, err, max_q=max_q, lse=lse)
    _check_attend(c, got, lse)
    # a row that sees such pages only: its weights are as ever, its values count as 2^-80 of their codes
    c["dev"]["vs"].zero_()
    zero_lse = torch.empty_like(lse)
    got = _run_attend(lib, c, err, max_q=max_q, lse=zero_lse)
    top = 448.0 if fmt == "e4m3" else 127.0
    assert float(got.float().abs().max()) <= 2.0 ** -80 * top * 1.01
    # either lse is within the tolerance of this file
    assert float((zero_lse - lse).abs().max()) <= 2.0 ** -16 * (4 + 2 * float(lse.abs().max())) and int(err) == 0


@pytest.mark.parametrize("n", [1, 30], ids=["split", "tiles"])
def test_attend_page8_denominators_stay_finite(lib, err, n):
    """Four million keys of one weight under the smallest scale: the sum of
    P / scale is 2^22 2^7 2^80 at least, and lse = ln(keys)."""
    ps, L = 1024, 1 << 22
    kp = torch.zeros(1, ps, 1, 64, dtype=torch.int8, device="cuda")
    vp = torch.full_like(kp, 100)
    ks, vs = torch.ones(1, 1, device="cuda"), torch.full((1, 1), 2.0 ** -110, device="cuda")
    q = torch.randn(n, 1, 64, device="cuda", dtype=torch.bfloat16)
    lse = torch.empty(n, 1, device="cuda")
    got = lib.attend_page8(q, kp, vp, ks, vs, torch.zeros(1, L // ps, dtype=torch.int32, device="cuda"), i32([n]), i32([L]),
                           causal=False, lse=lse, error_word=err)
    # every P and every scale is a power of two; sums of 2^22 terms in runs of thousands, 2^-24 a step
    assert float((lse.double() - np.log(L)).abs().max()) <= 2.0 ** -9
    assert float((got.double() / (100 * 2.0 ** -80) - 1).abs().max()) <= 2.0 ** -8 + 2.0 ** -9 and int(err) == 0


@pytest.mark.parametrize("cap", [2.0, 1e3, 1e6, 1e9])
@pytest.mark.parametrize("reqs,max_q", [(DECODE, 1), ([(1, 300), (5, 130), (3, 77)], 5), ([(130, 400), (1, 50)], 130)],
                         ids=["decode", "drafts", "tiles"])
@pytest.mark.parametrize("slopes", [False, True])
def test_attend_page8_caps_of_any_size(lib, err, cap, reqs, max_q, slopes):
    """A cap far above the scores is no cap: the capped score's error stays
    relative to the score (2^-19 of it), not to the cap.  Scores of |x| < 2^8 so
    stay within the 2^-11 and the 2^-17 (1 + |x|) of this file."""
    for i, (fmt, dtype) in enumerate((("int8", "f16"), ("e4m3", "bf16"))):
        c = _attend_case(16 + i, reqs, 6, 2, (64, 128)[i], 16, fmt, dtype, False, slopes=slopes)
        lse = torch.empty(c["q"].shape[:2], device="cuda")
        got = _run_attend(lib, c, err, max_q=max_q, lse=lse, logit_cap=cap)
        _check_attend(c, got, lse, logit_cap=cap)
    assert int(err) == 0


@pytest.mark.parametrize("n", [3, 40], ids=["split", "tiles"])
def test_attend_page8_bias_at_far_positions(lib, err, n):
    """Behind 2^24 tokens float32 holds every second position only; the bias
    takes the distance of a key, which is small, and gives what it gives for
    the same pages near the start."""
    c = _attend_case(17, [(n, 217)], 2, 1, 64, 16, "int8", "f16", False)
    c["slopes"] = np.array([0.5, 1.0], np.float32)
    c["dev"]["slopes"] = torch.tensor(c["slopes"]).cuda()
    far = 1 << 24
    d = c["dev"]
    d["table"] = torch.cat([torch.zeros(1, far // 16, dtype=torch.int32, device="cuda"), d["table"]], 1).contiguous()
    d["lens"] = d["lens"] + far
    lse = torch.empty(c["q"].shape[:2], device="cuda")
    got = _run_attend(lib, c, err, max_q=n, lse=lse, window=100)
    assert int(err) == 0
    _check_attend(c, got, lse, window=100)


@pytest.mark.parametrize("reqs,max_q", [([(1, 9), (1, 30), (2, 40)], 2), ([(1, 9000), (3, 30)], 3), ([(60, 300), (1, 40)], 60),
                                        ([(60, 60)] * 200, 60)], ids=["whole", "pieces", "tiles", "whole_tiles"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_attend_page8_nan_queries_give_nan(lib, err, reqs, max_q, dtype):
    """A query with a NaN: NaN in its own rows of o and lse and in no others.
    (Those may round otherwise than beside a number: a warp's rows look at their
    running maxima together, m = maximum - 7 moves when one of them needs it, and
    P = 2^(y - m) rounds to f16 at other places.  So the others are held to this
    file's tolerance, which any m within the range of P keeps.)"""
    c = _attend_case(18, reqs, 4, 2, 64, 16, "int8", dtype, False)
    T = c["T"]

    class Rows(np.ndarray):     # a request of one page: an index of one element is still an array
        def __getitem__(self, i):
            return np.asarray(self)[np.asarray(i) if isinstance(i, torch.Tensor) else i]

    want, want_lse, size = _attend_64bit({**c, **{k: [x.view(Rows) for x in c[k]] for k in ("pools", "scales")}})
    lse = torch.empty(T, 4, device="cuda")
    rows = torch.zeros(T, 4, dtype=torch.bool, device="cuda")
    rows[0, 1] = rows[T // 2, 2] = rows[T - 1, 0] = True
    c["dev"]["q"][rows] = float("nan")
    got = _run_attend(lib, c, err, max_q=max_q, lse=lse)
    assert torch.isnan(got[rows]).all() and torch.isnan(lse[rows]).all() and int(err) == 0
    eps = torch.finfo(got.dtype).eps / 2
    flush = 2.0 ** -32 * float(c["scales"][1].max()) * 127 * max(L for _, L in reqs)
    tol = eps * want.abs() + 2.0 ** -10 * size * (1 + eps) + flush + (2.0 ** -25 if dtype == "f16" else 0)
    assert ((got.double() - want).abs() <= tol)[~rows].all()
    off = (lse - want_lse)[~rows].abs().max()
    assert float(off) <= 2.0 ** -17 * (4 + 2 * float(want_lse.abs().max()))


def test_attend_page8_skips_bad_pages_and_lengths(lib, err):
    c = _attend_case(4, [(1, 100), (2, 40), (1, 50)], 4, 2, 64, 16, "int8", "bf16", False)
    bad = int(c["table"][0, 2])
    c["dev"]["table"][0, 2] = c["pools"][0].shape[0]
    lse = torch.empty(c["q"].shape[:2], device="cuda")
    got = _run_attend(lib, c, err, lse=lse)
    assert int(err) == lib.DEV_ERR_BAD_PAGE
    _check_attend(c, got, lse, skip_page=bad)
    err.zero_()
    c["dev"]["lens"][1] = 10 ** 6
    c["dev"]["table"][0, 2] = bad
    got = _run_attend(lib, c, err, lse=lse)
    assert int(err) == lib.DEV_ERR_BAD_LENGTH and (got[1:3] == 0).all() and torch.isneginf(lse[1:3]).all()
    err.zero_()
    c["dev"]["cu"][2] = 10
    c["dev"]["lens"][1] = 40
    out = torch.full_like(c["dev"]["q"], 7.0)
    _run_attend(lib, c, err, out=out)
    assert int(err) == lib.DEV_ERR_BAD_LENGTH and (out[3:] == 7.0).all() and torch.equal(out[:1], got[:1])


def test_attend_page8_tiles_skip_bad_pages(lib, err):
    """A page outside the pool in the middle of a prompt in tiles: its keys are
    no keys, whatever the copies of other pages left in its place."""
    c = _attend_case(6, [(60, 500), (2, 300)], 8, 2, 128, 32, "e4m3", "bf16", False)
    bad = int(c["table"][0, 3])
    c["dev"]["table"][0, 3] = -5
    lse = torch.empty(c["q"].shape[:2], device="cuda")
    got = _run_attend(lib, c, err, max_q=60, lse=lse)
    assert int(err) == lib.DEV_ERR_BAD_PAGE
    _check_attend(c, got, lse, skip_page=bad)


@pytest.mark.parametrize("reqs,Hq,H", [([(1, 700), (1, 90), (2, 40)], 64, 1), ([(1, 300), (3, 50)], 150, 1), ([(140, 140)], 128, 1)])
def test_attend_page8_many_heads_per_kv_head(lib, err, reqs, Hq, H):
    """One kv head for up to 150 query heads: whole queries per tile, or (more
    than 128) the split form's tiles."""
    c = _attend_case(7, reqs, Hq, H, 64, 16, "int8", "f16", False)
    lse = torch.empty(c["q"].shape[:2], device="cuda")
    got = _run_attend(lib, c, err, max_q=max(n for n, _ in reqs), lse=lse)
    _check_attend(c, got, lse)
    assert int(err) == 0


def test_attend_page8_on_two_streams_at_once(lib, err):
    """Two calls that overlap, each with a workspace of its own, on streams that
    are not the tensors' own."""
    a = _attend_case(8, [(1, 3000)] * 16, 8, 2, 128, 16, "e4m3", "bf16", False)
    b = _attend_case(9, [(200, 900), (1, 5000)], 8, 2, 128, 16, "int8", "f16", False)
    want = [_run_attend(lib, x, err, max_q=200) for x in (a, b)]
    ws = [lib.attend_page8_workspace(len(x["lens"]), x["q"].shape[0], 8, 2, 128) for x in (a, b)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    for _ in range(10):
        for x, w, s, o in zip((a, b), ws, streams, outs):
            with torch.cuda.stream(s):
                _run_attend(lib, x, err, max_q=200, out=o, ws=w)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1]) and int(err) == 0


def test_step_with_nothing_to_do(lib, err):
    """No tokens, no sequences: no launch, nothing written."""
    c = _attend_case(1, [(2, 20)], 4, 2, 64, 16, "int8", "bf16", False)
    d = c["dev"]
    none = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert lib.attend_page8(none, d["kp"], d["vp"], d["ks"], d["vs"], d["table"], i32([0]), d["lens"]).shape == (0, 4, 64)
    lib.attend_page8(d["q"], d["kp"], d["vp"], d["ks"], d["vs"], d["table"][:0], i32([]), i32([]))
    before = d["kp"].clone()
    lib.write_cache_page8(none[:, :2], none[:, :2], i32([0]), d["table"], d["kp"], d["vp"], d["ks"], d["vs"], error_word=err)
    assert torch.equal(before, d["kp"])
    cos, sin = lib.rope_table(1e4, 8, 64)
    assert lib.rope_axes(none, i32(np.zeros((2, 0))), bytes(32), cos, sin).shape == (0, 4, 64)
    got = lib.assign_pages(i32([0]), d["lens"], d["table"], i32([]), i32([0]), 16, 8, 0, error_word=err)
    assert got[1].tolist() == [20] and got[3].tolist() == [0] and int(err) == 0


# ------------------------------------------------------------ the step as used

def test_step_grows_a_batch_in_a_replayed_graph(lib, err):
    """assign -> rotary -> write -> attend: two prompts admitted eagerly, then
    decode steps replayed from one captured graph whose lengths grow on the
    device, compared with the oracle step by step; a second graph over its own
    workspace replays on another stream."""
    B, H, Hq, D, ps, W, P, fmt = 3, 2, 8, 64, 16, 8, 20, "e4m3"
    rng = np.random.default_rng(0)
    cos, sin = lib.rope_table(1e4, W * ps, D)
    axis = lib.axis_sections((12, 10, 10))
    kp, vp = _pool(P, ps, H, D, fmt, False, 0), _pool(P, ps, H, D, fmt, False, 0)
    ks, vs = torch.zeros(P, H, device="cuda"), torch.zeros(P, H, device="cuda")
    o_pools, o_scales = [_nhd(kp, False), _nhd(vp, False)], [np.zeros((P, H), np.float32) for _ in range(2)]
    table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
    lens, count = i32([0] * B), i32([P])
    pages = i32(rng.permutation(P))
    o_state = (np.full((B, W), -1, np.int32), np.zeros(B, np.int32), P)

    def device_step(x, new, old, ws=None):
        T = x.shape[0]
        old.copy_(lens)
        _, _, _, cu, slots, pos = lib.assign_pages(new, lens, table, pages, count, ps, P, T, block_table_out=table,
                                                   seqlens_out=lens, free_count_out=count, error_word=err)
        q, k = lib.rope_axes(x[:, :Hq], pos.expand(3, T), axis, cos, sin, k=x[:, Hq:Hq + H], error_word=err)
        lib.write_cache_page8(k, x[:, Hq + H:], cu, table, kp, vp, ks, vs, start_pos=old, error_word=err)
        lse = torch.empty(T, Hq, device="cuda")
        return lib.attend_page8(q, kp, vp, ks, vs, table, cu, lens, lse=lse, workspace=ws, error_word=err), lse, q

    def oracle_step(x, new, o_state):
        T = int(sum(new))
        t, ln, cnt, cu, _, pos, refused = step.assign_pages(np.array(new), o_state[1], o_state[0],
                                                            pages.cpu().numpy(), o_state[2], ps, T)
        assert not refused
        c, s = cos.cpu().numpy(), sin.cpu().numpy()
        p3 = np.stack([pos] * 3)
        r = lambda y: torch.tensor(step.rope_axes(y.float().numpy(), p3, axis, c, s)).bfloat16()  # noqa: E731
        q, k = r(x[:, :Hq]), r(x[:, Hq:Hq + H])
        step.write_page8(k.float().numpy(), x[:, Hq + H:].float().numpy(), cu, o_state[1], t, o_pools, o_scales, fmt)
        return (t, ln, cnt), dict(q=q, pools=o_pools, scales=o_scales, table=t, cu=cu, lens=ln, T=T, slopes=None,
                                  prefix=None)

    def make(T):
        return torch.tensor(rng.standard_normal((T, Hq + 2 * H, D)).astype(np.float32)).bfloat16()

    new = [37, 5, 60]
    x = make(sum(new))
    old = i32([0] * B)
    got, lse, _ = device_step(x.cuda(), i32(new), old)
    o_state, c = oracle_step(x, new, o_state)
    _check_attend(c, got, lse)

    x_static, one = torch.zeros(B, Hq + 2 * H, D, dtype=torch.bfloat16, device="cuda"), i32([1] * B)
    ws = lib.attend_page8_workspace(B, B, Hq, H, D)
    side = torch.cuda.Stream()
    keep = [t.clone() for t in (table, lens, count, kp, vp, ks, vs)]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):   # warm-up on the side stream, then undone
        device_step(x_static, one, old, ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g_out = device_step(x_static, one, old, ws)
    for t, v in zip((table, lens, count, kp, vp, ks, vs), keep):
        t.copy_(v)
    for i in range(20):   # crosses page borders
        x = make(B)
        x_static.copy_(x.cuda())
        if i % 2:
            graph.replay()
        else:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                graph.replay()
            torch.cuda.current_stream().wait_stream(side)
        o_state, c = oracle_step(x, [1] * B, o_state)
        assert np.array_equal(lens.cpu().numpy(), o_state[1]) and np.array_equal(table.cpu().numpy(), o_state[0])
        _check_attend(c, g_out[0], g_out[1])
    assert int(count) == o_state[2] and int(err) == 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_step_leaves_the_pages_of_refused_requests_alone(lib, err, fmt):
    """A draft refused for want of pages, a request served, a prompt piece too
    long for its row and one past num_tokens, all but the served one with a
    partly filled page: the step changes no code and no scale of theirs,
    whatever their rows hold; served later, they give the oracle's results."""
    B, H, Hq, D, ps, W, P, T = 4, 2, 8, 64, 16, 4, 16, 36
    rng = np.random.default_rng(5)
    cos, sin = lib.rope_table(1e4, W * ps, D)
    axis = lib.axis_sections((12, 10, 10))
    kp, vp = _pool(P, ps, H, D, fmt, False, 0), _pool(P, ps, H, D, fmt, False, 0)
    ks, vs = torch.zeros(P, H, device="cuda"), torch.zeros(P, H, device="cuda")
    table = torch.full((B, W), -1, dtype=torch.int32, device="cuda")
    lens, pages, start = i32([0] * B), i32(rng.permutation(P)), i32([0] * B)
    o_pools, o_scales = [_nhd(kp, False), _nhd(vp, False)], [np.zeros((P, H), np.float32) for _ in range(2)]
    o_table, o_lens = np.full((B, W), -1, np.int32), np.zeros(B, np.int32)
    count = i32([0])

    def step_of(x, new, free, T):
        nonlocal o_table, o_lens
        count.fill_(free)
        want = step.assign_pages(np.array(new), o_lens, o_table, pages.cpu().numpy(), free, ps, T)
        o_start = np.where(np.isin(np.arange(B), want[6]), -1, o_lens)
        _, _, _, cu, _, pos = lib.assign_pages(i32(new), lens, table, pages, count, ps, P, T, block_table_out=table,
                                               seqlens_out=lens, free_count_out=count, start_pos=start, error_word=err)
        word = int(err)
        err.zero_()
        assert np.array_equal(start.cpu().numpy(), o_start) and np.array_equal(cu.cpu().numpy(), want[3])
        # what lies in rows that are not rotated: far larger than the cache's values
        k = torch.full((T, H, D), 1e20, dtype=torch.bfloat16, device="cuda")
        dev = x.cuda()
        q, k = lib.rope_axes(dev[:, :Hq], pos.expand(3, T), axis, cos, sin, k=dev[:, Hq:Hq + H], k_out=k, error_word=err)
        lib.write_cache_page8(k, dev[:, Hq + H:], cu, table, kp, vp, ks, vs, start_pos=start, error_word=err)
        lse = torch.empty(T, Hq, device="cuda")
        out = lib.attend_page8(q, kp, vp, ks, vs, table, cu, lens, lse=lse, error_word=err)
        assert int(err) == 0
        c, s = cos.cpu().numpy(), sin.cpu().numpy()
        o_k = torch.tensor(step.rope_axes(x[:, Hq:Hq + H].float().numpy(), np.stack([want[5]] * 3), axis, c, s)).bfloat16()
        step.write_page8(o_k.float().numpy(), x[:, Hq + H:].float().numpy(), want[3], o_start, want[0], o_pools, o_scales, fmt)
        for got, w in ((kp, o_pools[0]), (vp, o_pools[1])):
            same = _nhd(got, False) == w
            if fmt == "e4m3":
                same |= ((_nhd(got, False) | w) & 0x7F) == 0
            assert same.all()
        assert np.array_equal(ks.cpu().numpy(), o_scales[0]) and np.array_equal(vs.cpu().numpy(), o_scales[1])
        o_table, o_lens = want[0], want[1]
        assert np.array_equal(table.cpu().numpy(), o_table) and np.array_equal(lens.cpu().numpy(), o_lens)
        return want, word, q, out, lse

    def make(T, size=1.0):
        return torch.tensor((size * rng.standard_normal((T, Hq + 2 * H, D))).astype(np.float32)).bfloat16()

    held = [10, 21, 60, 5]
    _, word, *_ = step_of(make(sum(held)), held, P, sum(held))
    assert word == 0
    keep = [t.clone() for t in (kp, vp, ks, vs)]
    want, word, *_ = step_of(make(T, 50.0), [20, 5, 9, 4], 0, T)
    assert want[6] == [0, 2, 3] and word == lib.DEV_ERR_NO_PAGES | lib.DEV_ERR_BAD_LENGTH
    for b in (0, 2, 3):
        own = table[b][table[b] >= 0].long()
        for now, before in zip((kp, vp, ks, vs), keep):
            assert torch.equal(now[own], before[own])
    x = make(27)
    want, word, q, out, lse = step_of(x, [20, 0, 3, 4], int((pages >= 0).sum()) - 9, 27)
    assert want[6] == [] and word == 0
    _check_attend(dict(q=q.cpu(), pools=o_pools, scales=o_scales, table=o_table, cu=want[3], lens=o_lens, T=27, slopes=None,
                       prefix=None), out, lse)


def test_step_entry_points_refuse_other_tensors(lib):
    c = _attend_case(1, [(1, 20)], 4, 2, 64, 16, "int8", "bf16", False)
    d = c["dev"]
    with pytest.raises(TypeError):
        lib.attend_page8(d["q"].float(), d["kp"], d["vp"], d["ks"], d["vs"], d["table"], d["cu"], d["lens"])
    with pytest.raises(ValueError):
        lib.attend_page8(d["q"], d["kp"], d["vp"], d["ks"][:1], d["vs"], d["table"], d["cu"], d["lens"])
    with pytest.raises(ValueError):
        lib.attend_page8(d["q"], d["kp"], d["vp"], d["ks"], d["vs"], d["table"].cpu(), d["cu"], d["lens"])
    with pytest.raises(TypeError):
        lib.attend_page8(d["q"], d["kp"], d["vp"].view(torch.uint8), d["ks"], d["vs"], d["table"], d["cu"], d["lens"])
    with pytest.raises(lib.QpkvError):
        lib.attend_page8(d["q"], d["kp"], d["vp"], d["ks"], d["vs"], d["table"], d["cu"], d["lens"], logit_cap=-1.0)
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(lib.QpkvError) as e:
        lib.attend_page8(d["q"], d["kp"], d["vp"], d["ks"], d["vs"], d["table"], d["cu"], d["lens"], workspace=small)
    assert e.value.status == 3
    x = torch.zeros(3, 1, 64, device="cuda")
    cos, sin = lib.rope_table(1e4, 8, 64)
    with pytest.raises(ValueError):
        lib.rope_axes(x, i32([[0, 1]]), bytes(32), cos, sin)
    with pytest.raises(lib.QpkvError):
        lib.rope_axes(x, i32([[0, 1, 2]]), bytes([1] * 32), cos, sin)
    with pytest.raises(ValueError):
        lib.rope_axes(x, i32([[0, 1, 2]]), bytes(16), cos, sin)


def test_attend_page8_refuses_a_workspace_with_gaps(lib):
    """An expanded byte or every second one: as many elements as asked for, but
    not their bytes in a row."""
    c = _attend_case(1, [(1, 20)], 4, 2, 64, 16, "int8", "bf16", False)
    d = c["dev"]
    n = lib.attend_page8_workspace(1, 1, 4, 2, 64).numel()
    for ws in (torch.empty(1, dtype=torch.uint8, device="cuda").expand(n), torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2],
               torch.empty(n, dtype=torch.uint8)):
        with pytest.raises(ValueError):
            lib.attend_page8(d["q"], d["kp"], d["vp"], d["ks"], d["vs"], d["table"], d["cu"], d["lens"], workspace=ws)
