"""GPU parity of the 4-bit cache: the write with the rotation and the bounds,
the read, the choice of pages and the attention, and all of them in a step,
against oracle/group4.py.

Codes, scales, bounds, rotated queries and chosen pages are equal bit for bit.
Tolerances of the attention outputs.  o is rounded once to its type (half a
step, eps/2 relative), every P to f16 (2^-11 relative to its own p |v|), and
a score's float32 error d <= 2^-11 scales p by e^d, so |got - want| <= eps/2
|want| + 2^-10 sum_j p_j |v_j| (1 + eps); K, V and q are exact.  f16 has an
end: P = 2^7 ... 2^15 for the key with the largest weight, and what rounds to a
multiple of 2^-24 is off by up to 2^-25 = 2^-32 of that P for each key: another
2^-32 max_j p_j sum_j |v_j|.  Scores: float32 sums of D exact products and a
handful of float32 operations, so the lse is within 2^-17 (1 + max |x|), max |x|
bounded by the largest |lse| of a test plus its spread."""
import numpy as np
import pytest
import torch

from oracle import group4

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def i32(x):
    return torch.as_tensor(np.asarray(x, np.int32)).cuda()


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def dev(x):
    return torch.tensor(x).cuda()


@pytest.fixture
def err():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def same_pool(got, want):
    """Codes and scales, the two zeros of a code being one value."""
    (c, s), (d, r) = group4.rows_of(got.cpu().numpy()), group4.rows_of(want)
    return np.array_equal(s, r) and ((c == d) | ((c | d) & 7 == 0)).all()


# ------------------------------------------------------------------- the write

WRITES = [
    ([(0, 1)], 1, 64, 16, "bf16", 64, False, False), ([(5, 30), (0, 0), (16, 16), (31, 2), (15, 1), (16, 1)], 3, 128, 16, "bf16", 128, True, True),
    ([(40, 100), (0, 7), (47, 1)], 2, 64, 48, "f16", 32, True, True), ([(100, 300), (0, 129)], 5, 128, 64, "bf16", 64, False, True),
    ([(3, 1), (0, 700)], 1, 128, 1024, "f16", 96, True, True), ([(200, 90)], 2, 64, 256, "bf16", 0, True, True),
    ([(n, 1) for n in range(64)], 8, 128, 16, "bf16", 128, False, True), ([(n % 37, n % 5) for n in range(150)], 2, 128, 32, "f16", 0, False, False)]


@pytest.mark.parametrize("lens,H,D,ps,dtype,rot,mul,bounds", WRITES)
def test_write_bit_exact(lib, err, lens, H, D, ps, dtype, rot, mul, bounds):
    """A first write, then one that appends to partly filled pages: codes, scales,
    bounds and rotated queries equal the oracle's, slots and pages that were not
    written are as they were, and reading back gives the oracle's values."""
    rng = np.random.default_rng(len(lens) + ps)
    B, dt, Hq = len(lens), DT[dtype], 2 * H + 1
    W = max(-(-(a + n) // ps) for a, n in lens) + 1
    P = W * B + 2
    table = rng.permutation(P)[:W * B].reshape(B, W).astype(np.int32)
    pools = [np.full((P, H, ps // 16, 9 * D), f, np.uint8) for f in (0x5A, 0x37)]
    dp = [dev(p) for p in pools]
    bd, bs = np.full((P, H, 2, D), 77, np.int8), np.full((P, H), 3.0, np.float32)
    dbd, dbs = dev(bd), dev(bs)
    cos = sin = ck = sk = None
    if rot:
        cos, sin = lib.rope_table(1e4, max(a + n for a, n in lens), rot)
        ck, sk = cos.cpu().numpy(), sin.cpu().numpy()
    muls = [np.exp(rng.standard_normal(H)).astype(np.float32) for _ in range(2)] if mul else [None, None]
    dm = [None if m is None else dev(m) for m in muls]
    for begin, n in (([0] * B, [a for a, _ in lens]), ([a for a, _ in lens], [n for _, n in lens])):
        T = int(sum(n))
        if T == 0:
            continue
        x = rng.standard_normal((T + 3, Hq + 2 * H, D)) * np.exp(rng.standard_normal((T + 3, 1, 1)))
        x[rng.integers(0, T, 3), :, :32] = 0.0
        x[rng.integers(0, T, 2)] *= 2.0 ** -9          # scales of zero among them
        x = torch.tensor(x.astype(np.float32)).to(dt)  # three rows behind the last sequence
        xd = x.cuda()
        if H == 2:
            q, k, v = (y.contiguous() for y in xd.split([Hq, H, H], 1))
        else:
            q, k, v = xd.split([Hq, H, H], 1)
        cu = np.cumsum(n).astype(np.int32)
        out = torch.full((T + 3, Hq, D), 7.0, dtype=dt, device="cuda") if rot else None
        got = lib.write_cache_group4(k, v, i32(cu), i32(table), *dp, start_pos=i32(begin) if any(begin) else None, rope_cos=cos, rope_sin=sin,
                                     q=q if rot else None, q_out=out, k_bounds=dbd if bounds else None, bound_scale=dbs if bounds else None,
                                     k_mul=dm[0], v_mul=dm[1], error_word=err)
        kf, vf = x[:, Hq:Hq + H].float().numpy(), x[:, Hq + H:].float().numpy()
        group4.write(kf, vf, cu, begin, table, pools, ck, sk, muls, bd if bounds else None, bs)
        assert same_pool(dp[0], pools[0]) and same_pool(dp[1], pools[1])
        assert np.array_equal(dbd.cpu().numpy(), bd) and np.array_equal(dbs.cpu().numpy(), bs)
        if rot:
            pos = np.concatenate([np.arange(a, a + m) for a, m in zip(begin, n)])
            want = torch.tensor(group4.rotate(x[:T, :Hq].float().numpy(), pos, ck, sk)).to(dt)
            assert got is out and torch.equal(got[:T].cpu(), want) and (got[T:] == 7.0).all()
            again = q.clone(memory_format=torch.preserve_format) if H == 2 else xd.clone().split([Hq, H, H], 1)[0]
            ret = lib.write_cache_group4(k, v, i32(cu), i32(table), *dp, start_pos=i32(begin), rope_cos=cos, rope_sin=sin, q=again,
                                         q_out=again, k_mul=dm[0], v_mul=dm[1], error_word=err)
            assert ret is again and torch.equal(again[:T], got[:T]) and torch.equal(again[T:], q[T:])   # in place
        for t in (torch.bfloat16, torch.float16):
            back = [torch.full((T + 3, H, D), 5.0, dtype=t, device="cuda") for _ in range(2)]
            lib.read_cache_group4(*dp, i32(cu), i32(table), T + 3, start_pos=i32(begin), k_mul=dm[0], v_mul=dm[1], k_out=back[0],
                                  v_out=back[1], error_word=err)
            for g, p, m in zip(back, pools, muls):
                parts = []
                for b in range(B):
                    w = group4.tokens(p, table[b], begin[b] + n[b])[begin[b]:].astype(np.float32)
                    parts.append(w if m is None else (w * m[:, None]).astype(np.float32))
                assert torch.equal(g[:T].cpu(), torch.tensor(np.concatenate(parts)).to(t)) and (g[T:] == 5.0).all()
    assert int(err) == 0


def test_write_of_values_at_the_ends(lib, err):
    """Exact ties of codes and scales, saturated scales, the smallest scales, signed
    zeros, infinities and NaN; bf16 beyond f16's range."""
    rng = np.random.default_rng(0)
    T, H, D, ps = 96, 1, 64, 32
    x = rng.standard_normal((T, H, D)).astype(np.float32)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
    for i in range(32):                     # amax = 6 s, s with every mantissa: x / s meets every tie
        s = (1 + (i % 8) / 8) * 2.0 ** (i // 8 - 2)
        x[i, 0] = (np.tile(ties, 8) * s * rng.choice([-1, 1], 64)).astype(np.float32)
    x[32] *= 1e6
    x[33] *= 1e30
    x[34, 0, 3] = np.inf
    x[35, 0, 40] = np.nan
    x[36, 0, 17] = -np.inf
    x[37] = -0.0
    for i in range(38, 60):                 # amax / 6 between two scales, the smallest among them
        x[i] = np.clip(x[i], -1, 1) * 6 * 2.0 ** -9 * (i - 37) / 2
    x = torch.tensor(x).bfloat16()
    pools = [np.zeros((4, H, 2, 9 * D), np.uint8) for _ in range(2)]
    dp, bd, bs = [dev(p) for p in pools], np.zeros((4, H, 2, D), np.int8), np.zeros((4, H), np.float32)
    dbd, dbs, table = dev(bd), dev(bs), np.array([[2, 0, 3]], np.int32)
    lib.write_cache_group4(x.cuda(), x.cuda(), i32([T]), i32(table), *dp, k_bounds=dbd, bound_scale=dbs, error_word=err)
    group4.write(x.float().numpy(), x.float().numpy(), [T], [0], table, pools, bounds=bd, bscale=bs)
    assert same_pool(dp[0], pools[0]) and same_pool(dp[1], pools[1])
    assert np.array_equal(dbd.cpu().numpy(), bd) and np.array_equal(dbs.cpu().numpy(), bs) and np.isinf(bs[0, 0])
    k, v = lib.read_cache_group4(*dp, i32([T]), i32(table), T)
    nan = torch.isnan(k[:, 0]).cpu().numpy()
    want = np.zeros((T, D), bool)
    want[34, :16] = want[35, 32:48] = want[36, 16:32] = True
    assert np.array_equal(nan, want) and int(err) == 0
    # the bounds of a page whose NaN token is written over
    y = torch.ones(32, 1, 64, dtype=torch.bfloat16, device="cuda")
    lib.write_cache_group4(y, y, i32([32]), i32([[0]]), *dp, k_bounds=dbd, bound_scale=dbs, error_word=err)
    # E4M3(1 / 6) = 11 / 64, and 1 is stored as 6 of those: 66 / 64
    assert (dbd[0] == 66).all() and float(dbs[0, 0]) == 2.0 ** -6


def test_write_leaves_out_what_does_not_fit(lib, err):
    H, D, ps = 1, 64, 16
    mk = lambda: [torch.full((4, H, 1, 9 * D), 9, dtype=torch.uint8, device="cuda") for _ in range(2)]  # noqa: E731
    x = torch.ones(40, H, D, dtype=torch.bfloat16, device="cuda")
    cos, sin = lib.rope_table(1e4, 24, D)
    k, v = mk()
    lib.write_cache_group4(x, x, i32([20, 40]), i32([[1, 4], [-1, 2]]), k, v, error_word=err)
    assert int(err) == lib.DEV_ERR_BAD_PAGE and (k[0] == 9).all() and (k[3] == 9).all() and not (k[1] == 9).any()
    codes, scales = group4.rows_of(k[2].cpu().numpy()[None])
    assert (scales[0, 0, :4] != 9).all() and (scales[0, 0, 4:] == 9).all()
    err.zero_()      # past the row
    k, v = mk()
    lib.write_cache_group4(x, x, i32([20]), i32([[3, 0]]), k, v, start_pos=i32([30]), error_word=err)
    assert int(err) == lib.DEV_ERR_BAD_LENGTH and (k[3] == 9).all()
    scales = group4.rows_of(k[0].cpu().numpy()[None])[1]
    assert (scales[0, 0, :14] == 9).all() and (scales[0, 0, 14:] != 9).all()
    for cu, start, kw in (([50], [0], {}), ([20, 10], [0, 0], {}), ([20], [5], dict(rope_cos=cos, rope_sin=sin)),
                          ([20], [-2], {})):
        err.zero_()   # more rows than there are; a length below zero; past the rope tables; a start below -1
        k, v = mk()
        q_out = torch.full_like(x, 7.0)
        if kw:
            kw = dict(kw, q=x, q_out=q_out)
        lib.write_cache_group4(x, x, i32(cu), i32([[3, 0, 1, 2]] * len(cu)), k, v, start_pos=i32(start), error_word=err, **kw)
        assert int(err) == lib.DEV_ERR_BAD_LENGTH and (q_out == 7.0).all()
        if len(cu) == 1:
            assert (k == 9).all() and (v == 9).all()
    err.zero_()      # a refused request between two served ones
    k, v = mk()
    q_out = torch.full_like(x, 7.0)
    lib.write_cache_group4(x, x, i32([3, 20, 24]), i32([[0], [1], [2]]), k, v, start_pos=i32([4, -1, 0]), rope_cos=cos, rope_sin=sin, q=x,
                           q_out=q_out, error_word=err)
    assert int(err) == 0 and (k[1] == 9).all() and (k[3] == 9).all() and (q_out[3:20] == 7.0).all() and (q_out[24:] == 7.0).all()
    scales = group4.rows_of(v.cpu().numpy())[1]
    assert (scales[0, 0, :4] == 9).all() and (scales[0, 0, 4:7] != 9).all() and (scales[2, 0, :4] != 9).all() and (scales[2, 0, 4:] == 9).all()
    back = [torch.full_like(x, 7.0) for _ in range(2)]
    lib.read_cache_group4(k, v, i32([3, 20, 24]), i32([[0], [1], [2]]), 40, start_pos=i32([4, -1, 0]), k_out=back[0], v_out=back[1], error_word=err)
    assert int(err) == 0 and (back[1][3:20] == 7.0).all() and (back[1][24:] == 7.0).all() and (back[1][:3] == 66 / 64).all()
    lib.read_cache_group4(k, v, i32([3, 23]), i32([[-1], [1]]), 40, error_word=err)
    assert int(err) == lib.DEV_ERR_BAD_LENGTH | lib.DEV_ERR_BAD_PAGE


# --------------------------------------------------------------- the selection

def _select_case(seed, reqs, Hq, H, D, ps, dtype, pad=0, extreme=False):
    rng = np.random.default_rng(seed)
    n_pages = [-(-L // ps) for _, L in reqs]
    P, W = sum(n_pages) + 2, max(n_pages + [1]) + 1
    perm = rng.permutation(P)
    table = np.full((len(reqs), W), -1, np.int32)
    at = 0
    for b, n in enumerate(n_pages):
        table[b, :n] = perm[at:at + n]
        at += n
    T = sum(n for n, _ in reqs)
    x = rng.standard_normal((T + pad, Hq, D)).astype(np.float32)
    if extreme:      # sums at their largest, scores that tie in their dozens
        x = np.sign(x)
        bounds = np.where(rng.random((P, H, 2, D)) < 0.02, 126, 127).astype(np.int8) * np.array([-1, 1], np.int8)[:, None]
        bscale = np.ones((P, H), np.float32)
    else:
        bounds = np.sort(rng.integers(-127, 128, (P, H, 2, D)), axis=2).astype(np.int8)
        bscale = np.exp2(rng.integers(-4, 2, (P, H))).astype(np.float32)
    q = torch.tensor(x).to(DT[dtype])
    return dict(q=q, bounds=bounds, bscale=bscale, table=table, cu=np.cumsum([n for n, _ in reqs]).astype(np.int32),
                lens=np.array([L for _, L in reqs], np.int32), T=T, ps=ps)


def _run_select(lib, c, err, n, out=None, max_q=0, **kw):
    return lib.select_pages(c["q"].cuda(), dev(c["bounds"]), dev(c["bscale"]), i32(c["table"]), i32(c["cu"]), i32(c["lens"]), c["ps"], n,
                            max_seqlen_q=max_q, out=out, error_word=err, **kw)


def _want_select(c, n, **kw):
    return group4.select(c["q"].double().numpy()[:c["T"]], c["bounds"], c["bscale"], c["table"], c["cu"], c["lens"], c["ps"], n, **kw)


@pytest.mark.parametrize("reqs,Hq,H,D,ps,dtype,n,kw", [
    ([(1, 1)], 1, 1, 64, 16, "bf16", 1, {}), ([(1, 333)], 4, 1, 64, 16, "f16", 5, dict(first=1)),
    ([(1, 700), (1, 15), (1, 16), (1, 17), (1, 0)], 8, 2, 128, 16, "bf16", 6, dict(first=2, last=3)),
    ([(5, 900), (0, 50), (3, 3), (7, 400)], 14, 2, 128, 32, "bf16", 7, dict(last=2)), ([(1, 9000), (2, 5000)], 10, 2, 64, 16, "f16", 64, dict(first=4, last=4)),
    ([(1, 3000)], 24, 2, 64, 48, "bf16", 8, {}), ([(4, 1500)], 33, 1, 128, 16, "bf16", 9, dict(first=1)), ([(3, 2000)], 16, 8, 64, 64, "bf16", 11, {}),
    ([(40, 1000), (90, 90)], 8, 2, 128, 16, "bf16", 10, dict(window=300, first=1)), ([(30, 20)], 2, 2, 64, 16, "bf16", 3, {}),
    ([(1, 40000)], 4, 1, 64, 16, "bf16", 300, dict(window=20011)), ([(1, 2500)], 2, 1, 128, 16, "f16", 200, {}), ([(130, 2000)], 7, 1, 128, 128, "f16", 4, {}),
    ([(700, 900), (0, 9), (3, 40), (500, 450)], 8, 8, 64, 16, "bf16", 5, dict(first=1)), ([(401, 2000), (398, 1200)], 8, 4, 128, 16, "bf16", 9, dict(window=250, last=2)),
    ([(650, 650)], 8, 2, 64, 32, "f16", 6, {}), ([(350, 1800), (60, 61)], 21, 3, 128, 16, "bf16", 20, dict(first=2)),
    ([(330, 1000)], 26, 2, 64, 16, "f16", 12, {})])
@pytest.mark.parametrize("extreme", [False, True])
def test_select_pages(lib, err, reqs, Hq, H, D, ps, dtype, n, kw, extreme):
    c = _select_case(len(reqs) + n, reqs, Hq, H, D, ps, dtype, pad=2, extreme=extreme)
    want = _want_select(c, n, **kw)
    for max_q in (0, max(m for m, _ in reqs)):
        out = torch.full((c["T"] + 2, H, n), 55, dtype=torch.int32, device="cuda")
        got = _run_select(lib, c, err, n, out=out, max_q=max_q, **kw).cpu().numpy()
        assert np.array_equal(got[:c["T"]], want) and (got[c["T"]:] == 55).all()
    assert int(err) == 0


def test_select_pages_of_a_whole_table_row(lib, err):
    """More pages than a block's shared memory has places: the cluster shares them."""
    rng = np.random.default_rng(9)
    N = 100000
    bounds = np.sort(rng.integers(-127, 128, (500, 1, 2, 64)), axis=2).astype(np.int8)
    c = dict(q=torch.tensor(rng.standard_normal((1, 2, 64)).astype(np.float32)).bfloat16(), bounds=bounds, bscale=np.ones((500, 1), np.float32),
             table=rng.integers(0, 500, (1, N)).astype(np.int32), cu=np.array([1], np.int32), lens=np.array([16 * N - 5], np.int32), T=1, ps=16)
    got = _run_select(lib, c, err, 1000, first=3, last=2).cpu().numpy()
    x = c["q"].double().numpy()[0]
    code = np.rint(x * 127 / np.abs(x).max()).astype(np.int64)
    score = np.maximum(code[None] * bounds[:, 0, :1], code[None] * bounds[:, 0, 1:]).sum(-1).max(-1)[c["table"][0]].astype(float)
    score[:3] = score[-2:] = np.inf
    assert np.array_equal(got[0, 0], np.sort(np.lexsort((np.arange(N), -score))[:1000])) and int(err) == 0


def test_select_pages_with_odd_inputs(lib, err):
    """Infinite scales come first; queries that are zero, NaN or infinite score
    nothing; bad pages are no candidates, also as the newest; rows that do not fit."""
    c = _select_case(3, [(1, 500), (1, 300), (1, 300), (1, 300)], 4, 2, 64, 16, "bf16")
    c["bscale"][c["table"][0, 5]] = np.inf
    c["bscale"][c["table"][0, 20], 1] = np.inf
    c["q"][1] = 0
    c["q"][2, 1, 3] = float("nan")
    c["q"][3, 3, 3] = float("inf")
    c["table"][0, 7], c["table"][1, 18], c["table"][2, 0] = -1, 99999, -5
    for n, kw in ((3, {}), (4, dict(first=1, last=2))):
        got = _run_select(lib, c, err, n, **kw).cpu().numpy()
        want = _want_select(c, n, **kw)
        assert np.array_equal(got, want) and 5 in got[0, 0] and 5 in got[0, 1]
        assert n == 4 or 20 in got[0, 1]      # with n = 4 three places are sure and one is left, for 5
        assert int(err) == lib.DEV_ERR_BAD_PAGE
    # the same for tokens of a prompt, and queries at the ends of bf16's range
    c = _select_case(13, [(400, 900), (300, 300)], 4, 2, 64, 16, "bf16")
    c["bscale"][c["table"][0, 5]] = np.inf
    c["q"][0:700:7] = 0
    c["q"][1:700:7, 1, 3] = float("nan")
    c["q"][2:700:7, 2, 5] = float("inf")
    c["q"][3:700:7] *= 2.0 ** 122
    c["q"][4:700:7] *= 2.0 ** -124
    c["table"][0, 30], c["table"][1, 4] = -1, 99999
    for first in (0, 2):
        got = _run_select(lib, c, err, 6, first=first).cpu().numpy()
        assert np.array_equal(got, _want_select(c, 6, first=first)) and int(err) == lib.DEV_ERR_BAD_PAGE
    c = _select_case(14, [(1, 900)] * 4, 4, 2, 64, 16, "bf16")
    c["q"][0] *= 2.0 ** 122
    c["q"][1] *= 2.0 ** -124
    assert np.array_equal(_run_select(lib, c, err, 6).cpu().numpy(), _want_select(c, 6))
    err.zero_()
    c = _select_case(4, [(1, 40), (1, 40)], 2, 1, 64, 16, "bf16")
    c["lens"][0], c["cu"] = 16 * c["table"].shape[1] + 1, np.array([1, 3], np.int32)
    assert (_run_select(lib, c, err, 2).cpu().numpy() == -1).all() and int(err) == lib.DEV_ERR_BAD_LENGTH


@pytest.mark.parametrize("reqs,ps", [([(1, 500), (1, 33)], 16), ([(1, 6000)], 16), ([(400, 900), (300, 300)], 32)])
@pytest.mark.parametrize("value", [float("nan"), -float("nan"), -np.inf, np.inf])
@pytest.mark.parametrize("share", [0.05, 0.5, 1.0])
def test_select_pages_with_scales_that_are_no_numbers(lib, err, reqs, ps, value, share):
    """Scales that are NaN or infinite count as +inf: candidates before those with a
    finite score, and no more pages are written than a row has places for, with
    every place sure and with places left (one block, a cluster, prompts)."""
    H = 2
    c = _select_case(21, reqs, 4, H, 64, ps, "bf16")
    rng = np.random.default_rng(int(100 * share))
    c["bscale"][rng.random(c["bscale"].shape) < share] = value
    for n, kw in ((3, dict(first=1, last=2)), (1, {}), (6, dict(first=2, last=1))):
        room = torch.full((4096 + c["T"] * H * n + 4096,), 55, dtype=torch.int32, device="cuda")
        out = room[4096:-4096].view(c["T"], H, n)
        got = _run_select(lib, c, err, n, out=out, **kw)
        assert np.array_equal(got.cpu().numpy(), _want_select(c, n, **kw))
        assert (room[:4096] == 55).all() and (room[-4096:] == 55).all()
    assert int(err) == 0


# --------------------------------------------------------------- the attention

def _attend_case(seed, reqs, Hq, H, D, ps, dtype, slopes=False, prefix=None, mul=False, n_sel=0, pad=0, size=1.0):
    """reqs: (queries, cached tokens) per sequence.  Unused slots and pages hold
    NaN scales; unused table entries -1."""
    rng = np.random.default_rng(seed)
    n_pages = [-(-L // ps) for _, L in reqs]
    P, W = sum(n_pages) + 2, max(n_pages + [1]) + 1
    perm = rng.permutation(P)
    table = np.full((len(reqs), W), -1, np.int32)
    at = 0
    for b, n in enumerate(n_pages):
        table[b, :n] = perm[at:at + n]
        at += n
    used = np.zeros((P, ps), bool)
    for b, (_, L) in enumerate(reqs):
        for i in range(n_pages[b]):
            used[table[b, i], :min(ps, L - i * ps)] = True
    pools = []
    for _ in range(2):
        x = rng.standard_normal((P, H, ps, D)) * np.exp(0.7 * rng.standard_normal((P, H, ps, 1)))
        codes, scales = group4.encode(x.astype(np.float32))
        scales = np.where(used[:, None, :, None], scales, np.uint8(0x7F))
        pools.append(group4.pool_of(codes, scales))
    T = sum(n for n, _ in reqs)
    q = torch.tensor((size * rng.standard_normal((T + pad, Hq, D))).astype(np.float32)).to(DT[dtype])
    sel = None
    if n_sel:
        sel = np.full((T + pad, H, n_sel), -1, np.int32)
        t = 0
        for b, (n, L) in enumerate(reqs):
            for i in range(n):
                for h in range(H):
                    ids = rng.permutation(max(1, n_pages[b]))[:rng.integers(0, n_sel + 1)]
                    if L:
                        sel[t, h, :len(ids)] = np.sort(ids)
                t += 1
    c = dict(q=q, pools=pools, table=table, cu=np.cumsum([n for n, _ in reqs]).astype(np.int32), T=T, selected=sel,
             lens=np.array([L for _, L in reqs], np.int32), prefix=None if prefix is None else np.array(prefix, np.int32),
             slopes=(2.0 ** (-8.0 * (np.arange(Hq) + 1) / Hq)).astype(np.float32) if slopes else None,
             mul=[np.exp(rng.standard_normal(H)).astype(np.float32) for _ in range(2)] if mul else [None, None])
    return c


def _run_attend(lib, c, err, max_q=0, out=None, lse=None, ws=None, **kw):
    d = lambda x, f=dev: None if x is None else f(x)  # noqa: E731
    return lib.attend_group4(c["q"].cuda(), dev(c["pools"][0]), dev(c["pools"][1]), i32(c["table"]), i32(c["cu"]), i32(c["lens"]),
                             max_seqlen_q=max_q, alibi_slopes=d(c["slopes"]), prefix_lens=d(c["prefix"], i32), selected=d(c["selected"], i32),
                             k_mul=d(c["mul"][0]), v_mul=d(c["mul"][1]), out=out, lse=lse, workspace=ws, error_word=err, **kw)


def _want_attend(c, causal=True, logit_cap=0.0, window=0, sm_scale=None, bad_page=None):
    q = c["q"][:c["T"]].double().numpy()
    return group4.attend(q, c["pools"], c["table"], c["cu"], c["lens"], sm_scale or 1 / np.sqrt(q.shape[2]), causal=causal, cap=logit_cap,
                         window=window, slopes=c["slopes"], prefix=c["prefix"], selected=c["selected"], mul=c["mul"], bad_page=bad_page, sizes=True)


def _check_attend(c, got, lse, wanted=None, **kw):
    want, want_lse, size, flush = wanted or _want_attend(c, **kw)
    eps = torch.finfo(c["q"].dtype).eps / 2
    g, l = f64(got)[:c["T"]], f64(lse)[:c["T"]]
    assert np.isfinite(g).all()
    tol = eps * np.abs(want) + 2.0 ** -10 * size * (1 + eps) + 2.0 ** -32 * flush + (2.0 ** -25 if c["q"].dtype == torch.float16 else 0)
    worst = float((np.abs(g - want) / (tol + 1e-300)).max()) if g.size else 0.0
    assert worst <= 1, worst
    assert np.array_equal(np.isneginf(l), np.isneginf(want_lse))
    fin = np.isfinite(want_lse)
    spread = np.abs(want_lse[fin]).max() if fin.any() else 0.0
    off = float(np.abs(l[fin] - want_lse[fin]).max()) if fin.any() else 0.0
    assert off <= 2.0 ** -17 * (4 + 2 * spread), off


DECODE = [(1, 1), (1, 16), (1, 333), (1, 17), (1, 0), (1, 1000)]
CASES = [
    (DECODE, 4, 1, 64, 16, "bf16", {}, {}), (DECODE, 8, 2, 128, 48, "f16", dict(mul=True), {}), (DECODE, 12, 1, 128, 16, "bf16", dict(slopes=True), {}),
    (DECODE, 40, 2, 64, 32, "bf16", {}, dict(logit_cap=20.0)), (DECODE, 33, 1, 128, 16, "f16", {}, dict(window=100)), (DECODE, 3, 3, 128, 64, "bf16", {}, dict(sm_scale=0.3)),
    ([(5, 400), (0, 30), (3, 3), (8, 1000)], 16, 4, 128, 16, "bf16", dict(slopes=True, mul=True), dict(logit_cap=50.0)),
    ([(5, 400), (7, 5), (2, 90)], 8, 8, 64, 16, "f16", {}, {}), ([(4, 500)], 20, 4, 128, 32, "bf16", dict(prefix=[300]), dict(window=150)),
    ([(300, 300)], 8, 2, 128, 16, "bf16", {}, {}), ([(190, 700), (1, 90), (33, 40)], 14, 2, 128, 32, "f16", dict(prefix=[100, 0, 40]), {}),
    ([(257, 257)], 4, 4, 64, 16, "bf16", dict(mul=True), dict(window=70)), ([(100, 800)], 7, 1, 64, 48, "bf16", dict(slopes=True), dict(logit_cap=30.0)),
    ([(150, 600), (1, 5)], 5, 1, 128, 16, "bf16", {}, dict(causal=False)), ([(90, 50)], 8, 1, 128, 16, "f16", {}, {}), ([(130, 400)], 2, 2, 128, 128, "bf16", {}, dict(logit_cap=500.0)),
    ([(40, 300)], 130, 1, 64, 16, "bf16", {}, {}), ([(150, 300), (2, 50), (1, 400)], 6, 2, 128, 16, "bf16", dict(size=6.0), dict(logit_cap=5.0)),
    (DECODE, 8, 2, 64, 16, "f16", dict(size=6.0, slopes=True), dict(logit_cap=3.0))]


@pytest.mark.parametrize("reqs,Hq,H,D,ps,dtype,case_kw,kw", CASES)
def test_attend_all_keys(lib, err, reqs, Hq, H, D, ps, dtype, case_kw, kw):
    c = _attend_case(Hq + D, reqs, Hq, H, D, ps, dtype, pad=3, **case_kw)
    wanted = _want_attend(c, **kw)
    W = c["table"].shape[1]
    for max_q, width in ((0, W), (max(n for n, _ in reqs), W), (max(n for n, _ in reqs), 5000), (1, W)):   # a wide table: keys by the thousand
        c["table"] = np.concatenate([c["table"][:, :W], np.full((len(reqs), max(0, width - W)), -1, np.int32)], 1)
        out = torch.full_like(c["q"], 7.0, device="cuda")
        lse = torch.full(c["q"].shape[:2], 7.0, device="cuda")
        got = _run_attend(lib, c, err, max_q=max_q, out=out, lse=lse, **kw)
        assert got is out
        _check_attend(c, got, lse, wanted)
        assert (out[c["T"]:] == 7.0).all() and (lse[c["T"]:] == 7.0).all()
        assert torch.equal(_run_attend(lib, c, err, max_q=max_q, **kw)[:c["T"]], got[:c["T"]])    # the same again, bit for bit
    assert int(err) == 0


@pytest.mark.parametrize("reqs,Hq,H,D,ps,dtype,case_kw,kw", CASES)
@pytest.mark.parametrize("n_sel", [1, 9])
def test_attend_selected_pages(lib, err, reqs, Hq, H, D, ps, dtype, case_kw, kw, n_sel):
    c = _attend_case(Hq + D + n_sel, reqs, Hq, H, D, ps, dtype, pad=3, n_sel=n_sel, **case_kw)
    out = torch.full_like(c["q"], 7.0, device="cuda")
    lse = torch.full(c["q"].shape[:2], 7.0, device="cuda")
    _run_attend(lib, c, err, out=out, lse=lse, **kw)
    _check_attend(c, out, lse, **kw)
    assert (out[c["T"]:] == 7.0).all() and (lse[c["T"]:] == 7.0).all() and int(err) == 0


def test_attend_one_long_context(lib, err):
    """A long axis cut into hundreds of pieces; all pages listed is the same."""
    c = _attend_case(5, [(1, 30011), (1, 77)], 8, 2, 128, 64, "bf16")
    lse = torch.empty(2, 8, device="cuda")
    got = _run_attend(lib, c, err, max_q=1, lse=lse)
    wanted = _want_attend(c)
    _check_attend(c, got, lse, wanted)
    W = c["table"].shape[1]
    c["selected"] = np.stack([np.where(np.arange(W) * 64 < L, np.arange(W), -1) for L in c["lens"]])[:, None].repeat(2, 1).astype(np.int32)
    got = _run_attend(lib, c, err, lse=lse)
    _check_attend(c, got, lse, wanted)
    assert int(err) == 0


def test_attend_lists_with_odd_entries(lib, err):
    """A page twice counts twice, in any order; places without keys are skipped and
    reported; a bad page is skipped and reported."""
    c = _attend_case(6, [(2, 200)], 4, 2, 64, 16, "bf16")
    c["selected"] = np.array([[[3, 3, 0, 11], [5, -1, 1, 5]], [[12, 2, 2, 2], [0, -1, -1, -1]]], np.int32)
    lse = torch.empty(2, 4, device="cuda")
    got = _run_attend(lib, c, err, lse=lse)
    _check_attend(c, got, lse)
    assert int(err) == 0
    for bad, bit in ((13, lib.DEV_ERR_BAD_INDEX), (-2, lib.DEV_ERR_BAD_INDEX), (1 << 30, lib.DEV_ERR_BAD_INDEX)):
        c["selected"][0, 0, 3] = bad
        err.zero_()
        got = _run_attend(lib, c, err, lse=lse)
        keep, c["selected"][0, 0, 3] = c["selected"][0, 0, 3], -1
        _check_attend(c, got, lse)
        assert int(err) == bit
    err.zero_()
    bad = c["table"][0, 2] = 777
    c["pools"] = [np.concatenate([p, p[:1]]) for p in c["pools"]]
    for sel in (c["selected"], None):
        c["selected"] = sel
        got = _run_attend(lib, c, err, lse=lse)
        _check_attend(c, got, lse, bad_page=bad)
        assert int(err) == lib.DEV_ERR_BAD_PAGE
        err.zero_()


def test_attend_rows_and_lengths_that_do_not_fit(lib, err):
    c = _attend_case(7, [(2, 40), (3, 50)], 2, 1, 64, 16, "bf16")
    lse = torch.full((5, 2), 7.0, device="cuda")
    out = torch.full_like(c["q"], 7.0, device="cuda")
    keep = c["lens"].copy()
    c["lens"] = np.array([40, 16 * c["table"].shape[1] + 1], np.int32)
    _run_attend(lib, c, err, out=out, lse=lse)
    assert int(err) == lib.DEV_ERR_BAD_LENGTH and (out[2:] == 0).all() and torch.isneginf(lse[2:]).all() and (out[:2] != 7.0).all()
    err.zero_()
    c["lens"], c["cu"] = keep, np.array([2, 9], np.int32)
    out.fill_(7.0)
    _run_attend(lib, c, err, out=out)
    assert int(err) == lib.DEV_ERR_BAD_LENGTH and (out[2:] == 7.0).all() and (out[:2] != 7.0).all()


@pytest.mark.parametrize("n,D,listed", [(1, 128, False), (5, 64, False), (5, 128, False), (90, 128, False), (90, 64, False), (5, 128, True), (30, 64, True)])
def test_attend_nan_reaches_those_who_see_it(lib, err, n, D, listed):
    """A NaN scale of a key makes its rows NaN, one of a value the 16 channels of
    its rows; rows that do not see the token are as without it."""
    ps, L, H, Hq = 16, 150, 2, 4
    c = _attend_case(8, [(n, L), (n, 60)], Hq, H, D, ps, "bf16")
    if listed:
        c["selected"] = np.array([[[0, 2, 8, 9]] * H] * n + [[[0, 1, 3, -1]] * H] * n, np.int32)
    lse = torch.empty(2 * n, Hq, device="cuda")
    clean = _run_attend(lib, c, err, max_q=n, lse=lse).clone()
    clean_lse = lse.clone()
    for which, j in ((1, L - 1), (1, L - n // 2 - 1), (0, L - n // 2 - 1), (1, 3), (0, 3), (1, 35)):
        pools = [p.copy() for p in c["pools"]]
        codes, scales = group4.rows_of(pools[which])
        pg = c["table"][0, j // ps]
        scales[pg, 1, j % ps, 2] = 0x7F
        c2 = dict(c)
        c2["pools"] = list(pools)
        c2["pools"][which] = group4.pool_of(codes, scales)
        got = _run_attend(lib, c2, err, max_q=n, lse=lse)
        sees = np.array([L - n + i >= j for i in range(n)] + [False] * n)
        if listed:
            sees &= np.isin(j // ps, [0, 2, 8, 9])
        want = np.zeros((2 * n, Hq, D), bool)
        if which:
            want[sees, 2:, 32:48] = True
        else:
            want[sees, 2:] = True
        nan = torch.isnan(got).cpu().numpy()
        assert np.array_equal(nan, want)
        # the rest: sums in another order at most (a NaN where P is set moves nothing else)
        assert torch.equal(got[~torch.tensor(want).cuda()], clean[~torch.tensor(want).cuda()])
        assert np.array_equal(torch.isnan(lse).cpu().numpy(), want.all(2)) and torch.equal(lse[~torch.isnan(lse)], clean_lse[~torch.isnan(lse)])
    assert int(err) == 0


@pytest.mark.parametrize("n,D,listed", [(1, 128, False), (1, 64, True), (5, 64, False), (3, 128, True), (90, 128, False)])
def test_attend_nan_of_a_value_without_weight(lib, err, n, D, listed):
    """With a distance bias an old token's weight is zero in float32, and a NaN scale
    of its value makes its channels NaN all the same, in every form (a narrow and a
    wide table, a prompt, lists), in all rows that see it and in no others."""
    ps, L, H, Hq = 16, 900, 2, 4
    c = _attend_case(9, [(n, L), (n, 60)], Hq, H, D, ps, "bf16")
    c["slopes"] = np.array([0.5, 4.0, 0.5, 0.25], np.float32)     # times 800 tokens: e^-200 and less
    if listed:
        c["selected"] = np.array([[list(range(0, 57, 2))] * H] * n + [[list(range(4)) + [-1] * 25] * H] * n, np.int32)
    W = c["table"].shape[1]
    for width in (W, 5000):
        c["table"] = np.concatenate([c["table"][:, :W], np.full((2, width - W), -1, np.int32)], 1)
        lse = torch.empty(2 * n, Hq, device="cuda")
        clean = _run_attend(lib, c, err, max_q=n, lse=lse).clone()
        clean_lse = lse.clone()
        assert torch.isfinite(clean).all()
        for j in (0, 3, 35, 100):
            codes, scales = group4.rows_of(c["pools"][1])
            scales[c["table"][0, j // ps], 1, j % ps, 2] = 0x7F
            c2 = dict(c, pools=[c["pools"][0], group4.pool_of(codes, scales)])
            got = _run_attend(lib, c2, err, max_q=n, lse=lse)
            want = np.zeros((2 * n, Hq, D), bool)
            want[:n, 2:, 32:48] = True
            assert np.array_equal(torch.isnan(got).cpu().numpy(), want)
            rest = ~torch.tensor(want).cuda()
            assert torch.equal(got[rest], clean[rest]) and torch.equal(lse, clean_lse)
    assert int(err) == 0


@pytest.mark.parametrize("Hq,H,D,max_q", [(4, 1, 64, 1), (16, 2, 128, 1), (10, 1, 64, 2), (8, 8, 128, 3)])
def test_attend_more_queries_than_the_bound(lib, err, Hq, H, D, max_q):
    """The one-kernel form with a bound of one to three queries and sequences of many:
    a block takes row tile after row tile, whose copies land where the sums of the one
    before lay."""
    c = _attend_case(10, [(40, 700), (3, 9), (25, 400), (1, 650)], Hq, H, D, 16, "bf16", mul=True, slopes=True)
    lse = torch.empty(c["T"], Hq, device="cuda")
    wanted = _want_attend(c)
    first = None
    for _ in range(10):
        got = _run_attend(lib, c, err, max_q=max_q, lse=lse)
        first = got if first is None else first
        assert torch.equal(got, first)
    _check_attend(c, got, lse, wanted)
    assert int(err) == 0


@pytest.mark.parametrize("reqs", [[(1, 300), (1, 30)], [(5, 400), (2, 20)], [(150, 150), (1, 40)], [(60, 700)]])
@pytest.mark.parametrize("D,listed", [(128, False), (64, False), (64, True)])
def test_attend_factors_far_from_one(lib, err, reqs, D, listed):
    """Factors of V from 2^-90 to 2^60 beside each other (bf16 holds what they give),
    in every form: they scale their head's outputs and nothing else."""
    c = _attend_case(17, reqs, 8, 4, D, 16, "bf16", n_sel=7 if listed else 0)
    c["mul"] = [np.array([1.0, 0.75, 2.0, 1.0], np.float32), np.array([2.0 ** -90, 2.0 ** 60, 2.0 ** -83 * 1.3, 1e-20], np.float32)]
    wanted = _want_attend(c)
    W, T = c["table"].shape[1], c["T"]
    for width in (W, 5000):
        c["table"] = np.concatenate([c["table"][:, :W], np.full((len(reqs), width - W), -1, np.int32)], 1)
        lse = torch.empty(T, 8, device="cuda")
        got = _run_attend(lib, c, err, max_q=max(n for n, _ in reqs), lse=lse)
        _check_attend(c, got, lse, wanted)
    assert int(err) == 0


@pytest.mark.parametrize("cap", [20.0, 50.0, 500.0, 1e6, 1e20])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("scores", ["small", "mixed", "large"])
def test_capped_scores_are_good_to_a_share_of_themselves(lib, err, cap, dtype, D, scores):
    """Rows that see one key, no bias: the lse is the capped score, c = cap tanh(x / cap),
    for scores far below the cap, on both sides of half of it, and about it, in every form.

    q and K have one channel each, so the product is exact.  The score is good to 2^-19
    of itself by definition.  Then, in log2 units: m + 7 is the score y, z = y - m is
    rounded at 7 (2^-22), its exponential is good to 2^-22 (1.45 times that in the
    logarithm), log2 of it at 7 to a step (2^-21), the sum to 2^-24 |y|, ln 2 and the
    last product to 2^-24 each: 2^-19 |c| + 2^-22 |c| + ln 2 (2^-22 + 1.45 * 2^-22 +
    2^-21 = 1.07e-6) < 2^-19 |c| + 2^-22 |c| + 2^-20.  (An exponential form good to 3e-7
    of the cap is off by 6e-6 at 20, a series of six terms by 8e-6 c at x = 0.6 cap.)"""
    cap = float(np.float32(cap))
    rng = np.random.default_rng(30)
    ps, H, Hq, scale, ch = 16, 2, 8, 0.125, 5
    for reqs, max_q, width, listed in (([(1, 70), (1, 5), (1, 400)], 1, 0, False), ([(1, 70), (1, 5), (1, 400)], 1, 5000, False),
                                       ([(5, 90), (6, 6)], 6, 0, False), ([(5, 90), (6, 6)], 6, 5000, False),
                                       ([(130, 300), (70, 70)], 130, 0, False), ([(9, 200), (1, 30)], 9, 0, True)):
        c = _attend_case(31, reqs, Hq, H, D, ps, dtype)
        T = c["T"]
        k = np.zeros((len(c["pools"][0]), H, ps, D), np.float32)
        k[..., ch] = 6.0
        c["pools"][0] = group4.pool_of(*group4.encode(k))
        part = np.exp(rng.uniform(np.log(1e-5), np.log(0.45), (T, Hq)))           # of the cap
        if scores == "mixed":
            half = rng.random((T, Hq)) < 0.5
            part[half] = rng.uniform(0.4, 0.75, half.sum())
        if scores == "large":
            part = rng.uniform(0.55, 4.0, (T, Hq))
        q = np.zeros((T, Hq, D))
        q[..., ch] = part * rng.choice([-1, 1], part.shape) * cap / (6 * scale)
        if dtype == "f16":
            q = np.clip(q, -60000, 60000)
        c["q"] = torch.tensor(q).to(DT[dtype])
        x = c["q"].double().numpy()[..., ch] * 6 * scale
        want = cap * np.tanh(x / cap)
        if listed:
            at = np.concatenate([np.arange(L - n, L) for n, L in reqs])
            c["selected"] = np.stack([at // ps, np.full(T, -1)], 1)[:, None].repeat(H, 1).astype(np.int32)
        W = c["table"].shape[1]
        c["table"] = np.concatenate([c["table"], np.full((len(reqs), max(0, width - W)), -1, np.int32)], 1)
        lse = torch.empty(T, Hq, device="cuda")
        _run_attend(lib, c, err, max_q=max_q, lse=lse, sm_scale=scale, logit_cap=cap, window=1)
        off = np.abs(f64(lse) - want) / ((2.0 ** -19 + 2.0 ** -22) * np.abs(want) + 2.0 ** -20)
        assert off.max() <= 1, (reqs, width, listed, off.max())
    assert int(err) == 0


# ------------------------------------------------------------------- all of them

@pytest.mark.parametrize("D,ps,dtype", [(128, 16, "bf16"), (64, 32, "f16")])
def test_a_serving_step(lib, err, D, ps, dtype):
    """Pages assigned, tokens rotated and appended, pages chosen, attended to: a
    prompt, then steps replayed from one captured graph, each against the oracle."""
    rng = np.random.default_rng(11)
    B, Hq, H, W, n = 5, 8, 2, 12, 4
    dt, P = DT[dtype], B * W
    lens0 = [37, 5, 100, 64, 1]
    cos, sin = lib.rope_table(1e4, W * ps, D)
    ck, sk = cos.cpu().numpy(), sin.cpu().numpy()
    pools = [np.zeros((P, H, ps // 16, 9 * D), np.uint8) for _ in range(2)]
    bd, bs = np.zeros((P, H, 2, D), np.int8), np.ones((P, H), np.float32)
    dp, dbd, dbs = [dev(p) for p in pools], dev(bd), dev(bs)
    table, lens, pages, count = i32(np.full((B, W), -1)), i32([0] * B), i32(rng.permutation(P)), i32([P])
    muls = [np.exp(rng.standard_normal(H)).astype(np.float32) for _ in range(2)]
    dm = [dev(m) for m in muls]
    ws = lib.attend_group4_workspace(B, max(sum(lens0), B), Hq, H, D)

    def step(new, x, T, max_q):
        start = torch.empty_like(lens)
        _, _, _, cu, _, _ = lib.assign_pages(new, lens, table, pages, count, ps, P, T, block_table_out=table, seqlens_out=lens,
                                             free_count_out=count, start_pos=start, error_word=err)
        q, k, v = x.split([Hq, H, H], 1)
        qr = lib.write_cache_group4(k, v, cu, table, *dp, start_pos=start, rope_cos=cos, rope_sin=sin, q=q, k_bounds=dbd, bound_scale=dbs,
                                    k_mul=dm[0], v_mul=dm[1], error_word=err)
        sel = lib.select_pages(qr, dbd, dbs, table, cu, lens, ps, n, first=1, last=1, error_word=err)
        lse = torch.empty(T, Hq, device="cuda")
        o = lib.attend_group4(qr, *dp, table, cu, lens, max_seqlen_q=max_q, selected=sel if max_q == 1 else None, k_mul=dm[0], v_mul=dm[1],
                              lse=lse, workspace=ws, error_word=err)
        return cu, qr, sel, o, lse

    def check(x, start, got):
        cu, qr, sel, o, lse = got
        c, xs = cu.cpu().numpy(), x.float().cpu().numpy()
        tab = table.cpu().numpy()
        group4.write(xs[:, Hq:Hq + H], xs[:, Hq + H:], c, start, tab, pools, ck, sk, muls, bd, bs)
        assert same_pool(dp[0], pools[0]) and same_pool(dp[1], pools[1]) and np.array_equal(dbd.cpu().numpy(), bd)
        pos = np.concatenate([np.arange(s, s + m) for s, m in zip(start, np.diff(np.concatenate([[0], c])))])
        assert torch.equal(qr.cpu(), torch.tensor(group4.rotate(xs[:, :Hq], pos, ck, sk)).to(dt))
        case = dict(q=qr.cpu(), pools=pools, table=tab, cu=c, lens=lens.cpu().numpy(), T=len(xs), prefix=None, slopes=None, mul=muls,
                    selected=sel.cpu().numpy() if len(xs) == B else None)
        want = group4.select(case["q"].double().numpy(), bd, bs, tab, c, case["lens"], ps, n, first=1, last=1)
        assert np.array_equal(sel.cpu().numpy(), want)
        _check_attend(case, o, lse)

    T = sum(lens0)
    x = torch.tensor(rng.standard_normal((T, Hq + 2 * H, D)).astype(np.float32)).to(dt).cuda()
    check(x, [0] * B, step(i32(lens0), x, T, max(lens0)))
    ones, xs = i32([1] * B), torch.zeros(B, Hq + 2 * H, D, dtype=dt, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    state = [t.clone() for t in (table, lens, count, *dp, dbd, dbs)]
    with torch.cuda.stream(side):
        step(ones, xs, B, 1)                     # warm up
        for t, s in zip((table, lens, count, *dp, dbd, dbs), state):
            t.copy_(s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(ones, xs, B, 1)
    at = list(lens0)
    for _ in range(18):
        xs.copy_(torch.tensor(rng.standard_normal(xs.shape).astype(np.float32)).to(dt))
        graph.replay()
        check(xs, at, got)
        at = [a + 1 for a in at]
    assert lens.tolist() == at and int(err) == 0


def test_offsets_beyond_32_bits(lib, err):
    """A pool of 4.6 GB (and bounds to match): its last pages are written, read
    back, chosen and attended to, the first ones are left alone."""
    H, D, ps, P = 8, 128, 16, 500_000
    k, v = (torch.zeros(P, H, 1, 9 * D, dtype=torch.uint8, device="cuda") for _ in range(2))
    bd, bs = torch.zeros(P, H, 2, D, dtype=torch.int8, device="cuda"), torch.zeros(P, H, device="cuda")
    n, L = 40, 40
    table = np.array([[P - 1, P - 2, P - 3]], np.int32)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(n, 2 * H, D, generator=g, device="cuda").bfloat16()
    q = torch.randn(n, 2 * H, D, generator=g, device="cuda").bfloat16()
    lib.write_cache_group4(x[:, :H], x[:, H:], i32([n]), i32(table), k, v, k_bounds=bd, bound_scale=bs, error_word=err)
    pools = [np.zeros((3, H, 1, 9 * D), np.uint8) for _ in range(2)]
    small, sb, ss = np.array([[2, 1, 0]], np.int32), np.zeros((3, H, 2, D), np.int8), np.zeros((3, H), np.float32)
    f = x.float().cpu().numpy()
    group4.write(f[:, :H], f[:, H:], [n], [0], small, pools, bounds=sb, bscale=ss)
    assert same_pool(k[-3:], pools[0]) and same_pool(v[-3:], pools[1]) and np.array_equal(bd[-3:].cpu().numpy(), sb)
    back = lib.read_cache_group4(k, v, i32([n]), i32(table), n, error_word=err)
    assert np.array_equal(f64(back[1]), group4.tokens(pools[1], small[0], L))
    sel = lib.select_pages(q, bd, bs, i32(table), i32([n]), i32([L]), ps, 2, error_word=err)
    assert np.array_equal(sel.cpu().numpy(), group4.select(q.double().cpu().numpy(), sb, ss, small, [n], [L], ps, 2))
    case = dict(q=q.cpu(), pools=pools, table=small, cu=[n], lens=[L], T=n, prefix=None, slopes=None, mul=[None, None])
    for kw in (dict(), dict(selected=sel), dict(max_seqlen_q=n)):
        case["selected"] = sel.cpu().numpy() if kw.get("selected") is not None else None
        lse = torch.empty(n, 2 * H, device="cuda")
        _check_attend(case, lib.attend_group4(q, k, v, i32(table), i32([n]), i32([L]), lse=lse, error_word=err, **kw), lse)
    assert int(k[:-3].max()) == 0 and int(v[:-3].max()) == 0 and int(err) == 0


def test_two_streams_and_workspaces(lib, err):
    c = [_attend_case(20 + i, [(1, 900), (1, 300 + i)], 8, 2, 128, 16, "bf16") for i in range(2)]
    want = [_want_attend(x) for x in c]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for s, x in zip(streams, c):
            with torch.cuda.stream(s):
                lse = torch.empty(2, 8, device="cuda")
                ws = lib.attend_group4_workspace(2, 2, 8, 2, 128)
                got.append((_run_attend(lib, x, err, max_q=1, lse=lse, ws=ws), lse))
        torch.cuda.synchronize()
        for x, w, (o, lse) in zip(c, want, got):
            _check_attend(x, o, lse, w)
    assert int(err) == 0


def test_bindings_refuse(lib):
    H, D = 2, 64
    x = torch.zeros(4, H, D, dtype=torch.bfloat16, device="cuda")
    pool = torch.zeros(3, H, 1, 9 * D, dtype=torch.uint8, device="cuda")
    cu, table = i32([4]), i32([[0, 1]])
    cos, sin = lib.rope_table(1e4, 9, D)
    bad = [dict(rope_cos=cos), dict(k_bounds=torch.zeros(3, H, 2, D, dtype=torch.int8, device="cuda")), dict(q=x),
           dict(k_mul=torch.ones(3, device="cuda")), dict(k_mul=torch.ones(H)), dict(start_pos=i32([1, 2]))]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            lib.write_cache_group4(x, x, cu, table, pool, pool, **kw)
    for kp, xx in ((pool[..., :-1], x), (pool.int(), x), (pool, x.float()), (pool[:, :1], x), (pool.cpu(), x)):
        with pytest.raises((ValueError, TypeError)):
            lib.write_cache_group4(xx, xx, cu, table, kp, pool)
    odd = torch.zeros(4 * H * D + 1, dtype=torch.bfloat16, device="cuda")[1:].view(4, H, D)
    with pytest.raises(lib.QpkvError):
        lib.write_cache_group4(odd, x, cu, table, pool, pool)
    with pytest.raises(lib.QpkvError):
        lib.write_cache_group4(x, x, cu, table, pool, pool, rope_cos=cos[:, :24].contiguous(), rope_sin=sin[:, :24].contiguous())
    bd, bs = torch.zeros(3, H, 2, D, dtype=torch.int8, device="cuda"), torch.ones(3, H, device="cuda")
    for kw in (dict(first=2), dict(last=0), dict(window=-1)):
        with pytest.raises(lib.QpkvError):
            lib.select_pages(x, bd, bs, table, cu, cu, 16, 2, **kw)
    with pytest.raises((ValueError, TypeError)):
        lib.select_pages(x, bd.float(), bs, table, cu, cu, 16, 2)
    for kw in (dict(selected=i32(np.zeros((4, H, 0)))), dict(selected=i32(np.zeros((3, H, 2)))), dict(workspace=pool[:, :1]), dict(v_mul=bs)):
        with pytest.raises((ValueError, TypeError)):
            lib.attend_group4(x, pool, pool, table, cu, cu, **kw)
    wide = i32(np.zeros((1, 3000)))
    with pytest.raises(lib.QpkvError):
        lib.attend_group4(x, pool, pool, wide, cu, cu, workspace=pool)
    e = torch.empty(0, H, D, dtype=torch.bfloat16, device="cuda")      # nothing to do
    none, no_table = i32([]), i32(np.zeros((0, 1)))
    lib.write_cache_group4(e, e, none, no_table, pool, pool)
    assert lib.attend_group4(e, pool, pool, no_table, none, none).shape == e.shape
    assert lib.select_pages(e, bd, bs, no_table, none, none, 16, 2).shape == (0, H, 2)
    assert lib.read_cache_group4(pool, pool, none, no_table, 0)[0].shape == e.shape
