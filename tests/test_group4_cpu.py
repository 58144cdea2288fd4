"""The 4-bit cache on the CPU: argument checks of its entry points, each
refusal before anything is launched, and pins of its oracle."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import e4m3, group4, rope

FAKE = 4096      # a 16-byte aligned address that no check reads
INVALID, UNSUPPORTED, SMALL = 1, 2, 3


@pytest.fixture(scope="module")
def q():
    import os
    import quantized_paged_kv_varlen_gb300 as q
    from quantized_paged_kv_varlen_gb300 import build
    if not os.path.exists(q.LIB_PATH):
        build.build()
    q.load()
    return q


def test_struct_mirrors(q):
    lib = q.load()
    for i, c in ((7, q.WriteGroup4Params), (8, q.ReadGroup4Params), (9, q.SelectPagesParams), (10, q.AttendGroup4Params)):
        assert lib.qpkv_struct_size(i) == ctypes.sizeof(c)


def _call(fn, p, **changes):
    for n, v in changes.items():
        setattr(p, n, v)
    return fn(ctypes.byref(p), None)


def _fill(p, **ints):
    for n, t in p._fields_:
        if t is ctypes.c_void_p:
            setattr(p, n, FAKE)
    for n, v in ints.items():
        setattr(p, n, v)
    return p


def _write(q):
    return _fill(q.WriteGroup4Params(), num_seqs=2, num_tokens=5, num_heads_q=4, num_heads_kv=2, head_dim=128, page_size=16, num_pages=4,
                 bt_stride=2, rot_dim=64, rope_max_pos=40, k_stride_t=256, k_stride_h=128, v_stride_t=256, v_stride_h=128, q_stride_t=512,
                 q_stride_h=128, q_out_stride_t=512, q_out_stride_h=128)


SHARED = [(dict(num_seqs=-1), INVALID), (dict(num_tokens=-1), INVALID), (dict(num_heads_kv=0), INVALID), (dict(num_pages=0), INVALID),
          (dict(bt_stride=0), INVALID), (dict(page_size=0), INVALID), (dict(page_size=24), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED),
          (dict(dtype=2), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED), (dict(bt_stride=1 << 27), UNSUPPORTED), (dict(cu_seqlens_q=None), INVALID),
          (dict(block_table=None), INVALID), (dict(num_tokens=0), 0), (dict(num_seqs=0), 0)]


@pytest.mark.parametrize("change,want", SHARED + [
    (dict(k=None), INVALID), (dict(v=FAKE + 8), INVALID), (dict(k_pool=None), INVALID), (dict(v_pool=FAKE + 4), INVALID), (dict(rope_sin=None), INVALID),
    (dict(rope_cos=None), INVALID), (dict(k_bounds=None), INVALID), (dict(bound_scale=None), INVALID), (dict(q_out=None), INVALID),
    (dict(rope_cos=None, rope_sin=None), INVALID), (dict(rot_dim=0), INVALID), (dict(rot_dim=48), UNSUPPORTED), (dict(rot_dim=160), UNSUPPORTED),
    (dict(rope_max_pos=0), INVALID), (dict(num_heads_q=0), INVALID), (dict(k_stride_t=257), INVALID), (dict(v_stride_h=4), INVALID),
    (dict(q_stride_t=3), INVALID), (dict(q_out_stride_h=9), INVALID), (dict(k_mul=FAKE + 2), INVALID), (dict(bound_scale=FAKE + 1), INVALID),
    (dict(k_bounds=FAKE + 8), INVALID), (dict(num_heads_kv=65536), UNSUPPORTED), (dict(num_tokens=1 << 30, num_heads_kv=4096), UNSUPPORTED)])
def test_write_refuses(q, change, want):
    assert _call(q.load().qpkv_write_group4, _write(q), **change) == want
    assert q.load().qpkv_write_group4(None, None) == INVALID


def _read(q):
    return _fill(q.ReadGroup4Params(), num_seqs=2, num_tokens=5, num_heads_kv=2, head_dim=128, page_size=16, num_pages=4, bt_stride=2)


@pytest.mark.parametrize("change,want", SHARED + [
    (dict(k_pool=None), INVALID), (dict(k_out=FAKE + 8), INVALID), (dict(v_mul=FAKE + 1), INVALID), (dict(k_out=None, v_out=None), 0)])
def test_read_refuses(q, change, want):
    assert _call(q.load().qpkv_read_group4, _read(q), **change) == want


def _select(q):
    return _fill(q.SelectPagesParams(), num_seqs=2, num_tokens=5, num_heads_q=4, num_heads_kv=2, head_dim=128, page_size=16, num_pages=4,
                 bt_stride=2, num_selected=3, first=1, last=2)


@pytest.mark.parametrize("change,want", SHARED + [
    (dict(first=-1), INVALID), (dict(last=0), INVALID), (dict(num_selected=0), INVALID), (dict(first=2), INVALID), (dict(window=-1), INVALID),
    (dict(num_heads_q=0), INVALID), (dict(num_heads_q=3), UNSUPPORTED), (dict(num_heads_q=258), UNSUPPORTED), (dict(bt_stride=(1 << 18) + 1), UNSUPPORTED),
    (dict(num_selected=1 << 30), UNSUPPORTED), (dict(num_tokens=1 << 28), UNSUPPORTED), (dict(q=None), INVALID), (dict(selected=None), INVALID),
    (dict(k_bounds=FAKE + 8), INVALID), (dict(selected=FAKE + 2), INVALID), (dict(seqlens_kv=None), INVALID)])
def test_select_refuses(q, change, want):
    assert _call(q.load().qpkv_select_pages, _select(q), **change) == want


def _attend(q):
    n = q.load().qpkv_attend_group4_workspace_bytes(2, 5, 8, 2, 128)
    assert n > 0
    return _fill(q.AttendGroup4Params(), num_seqs=2, num_tokens=5, num_heads_q=8, num_heads_kv=2, head_dim=128, page_size=16,
                 num_pages=4, bt_stride=3000, num_selected=3, workspace_bytes=n)


@pytest.mark.parametrize("change,want", SHARED + [
    (dict(num_heads_q=0), INVALID), (dict(window=-1), INVALID), (dict(logit_cap=-1.0), INVALID), (dict(logit_cap=float("nan")), INVALID),
    (dict(logit_cap=float("inf")), INVALID), (dict(logit_cap=1e-30), INVALID), (dict(sm_scale=float("inf")), INVALID), (dict(num_selected=0), INVALID),
    (dict(num_selected=1 << 28), UNSUPPORTED), (dict(num_heads_q=7), UNSUPPORTED), (dict(num_pages=1 << 30), UNSUPPORTED),
    (dict(num_tokens=1 << 30), UNSUPPORTED), (dict(q=None), INVALID), (dict(o=FAKE + 4), INVALID), (dict(k_pool=FAKE + 8), INVALID),
    (dict(selected=FAKE + 1), INVALID), (dict(selected=None, workspace=None), SMALL), (dict(workspace=FAKE + 1), INVALID),
    (dict(selected=None, workspace_bytes=64), SMALL), (dict(selected=None, bt_stride=2, max_seqlen_q=9, workspace=None, num_heads_q=10), SMALL)])
def test_attend_refuses(q, change, want):
    assert _call(q.load().qpkv_attend_group4, _attend(q), **change) == want


@pytest.mark.parametrize("cap,want", [(1e20, 0), (1e-20, 0), (50.0, 0), (1.01e20, INVALID), (1e30, INVALID), (2.4e38, INVALID), (3.4e38, INVALID)])
def test_attend_takes_caps_whose_scores_stay_in_float32(q, cap, want):
    # no tokens: the checks alone
    assert _call(q.load().qpkv_attend_group4, _attend(q), logit_cap=cap, num_tokens=0) == want


def test_attend_workspace_sizes(q):
    f = q.load().qpkv_attend_group4_workspace_bytes
    assert f(-1, 5, 8, 2, 128) == f(2, -1, 8, 2, 128) == f(2, 5, 7, 2, 128) == f(2, 5, 8, 2, 96) == 0
    assert f(2, 5, 8, 2, 128) <= f(4000, 5, 8, 2, 128) and f(64, 64, 32, 8, 64) < f(64, 64, 32, 8, 128)


# ------------------------------------------------------------------- the oracle

def test_e2m1_rounds_to_the_nearest_value():
    assert group4.E2M1.tolist() == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    assert group4.encode_e2m1(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 9.0, -0.75, -5.01, 0.26])).tolist() == [
        0, 2, 2, 4, 4, 6, 6, 7, 10, 15, 1]
    x = np.random.default_rng(0).uniform(-6, 6, 4000)
    c = group4.encode_e2m1(x)
    got = np.where(c & 8, -1, 1) * group4.E2M1[c & 7]
    assert np.array_equal(np.abs(got - x), np.abs(np.concatenate([group4.E2M1, -group4.E2M1])[:, None] - x).min(0))


def test_the_corrected_quotient_gives_the_codes_of_the_division():
    """q = x r, q + (x - q s) r with r = 1 / s rounded, fused steps emulated
    exactly (24 + 4 and 24 + 24 bits fit float64): the codes of RN(x / s) for all
    significands of s and x at and around every midpoint, and at random."""
    rng = np.random.default_rng(1)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], np.float32)
    for m in range(8):
        s = np.float32((8 + m) / 8)
        near = (mids * s).astype(np.float32)
        x = np.concatenate([near] + [np.nextafter(near, np.float32(d)).astype(np.float32) for d in (0, 99)]
                           + [rng.uniform(0, 6.5, 20000).astype(np.float32) * s])
        r = np.float32(1) / s
        y = (x * r).astype(np.float32)
        rest = (x.astype(np.float64) - y.astype(np.float64) * np.float64(s)).astype(np.float32)
        y = (y.astype(np.float64) + rest.astype(np.float64) * np.float64(r)).astype(np.float32)
        assert np.array_equal(group4.encode_e2m1(y), group4.encode_e2m1((x / s).astype(np.float32)))


def test_values_are_within_half_a_step_and_exact_in_16_bits():
    rng = np.random.default_rng(2)
    x = (rng.standard_normal((50, 4, 64)) * np.exp(2 * rng.standard_normal((50, 4, 1)))).astype(np.float32)
    c, s = group4.encode(x)
    v = group4.value(c, s)
    # the largest step is 2 (4 to 6) of a scale within 2^-4 (or half its smallest step) of amax / 6
    amax = np.repeat(np.abs(x.reshape(50, 4, 4, 16)).max(-1), 16, -1)
    assert (np.abs(v - x) <= amax / 6 * (1 + 2.0 ** -4) + 6 * amax / 6 * 2.0 ** -4 + 6 * 2.0 ** -10).all()
    for t in (torch.float16, torch.bfloat16):
        assert np.array_equal(torch.tensor(v).to(t).double().numpy(), v)
    assert e4m3.decode(group4.encode(np.full((1, 16), 1e9, np.float32))[1])[0, 0] == 448
    c, s = group4.encode(np.array([[np.nan] + [1.0] * 15, [np.inf] + [1.0] * 15, [0.0] * 16], np.float32))
    assert s[:, 0].tolist() == [0x7F, 0x7F, 0] and not c.any()
    codes, scales = group4.rows_of(group4.pool_of(*group4.encode(x[:48].reshape(3, 4, 16, 64))))
    assert np.array_equal(group4.value(codes, scales), group4.value(*group4.encode(x[:48].reshape(3, 4, 16, 64))))


def test_rotation_is_the_rotation_of_the_tables():
    cos, sin = rope.cos_sin_table(50, 32, 1e4)
    x = np.random.default_rng(3).standard_normal((7, 2, 64)).astype(np.float32)
    p = np.arange(7) * 5
    y = group4.rotate(x, p, cos, sin)
    assert np.array_equal(y[..., :32], rope.rotate(x[..., :32], p, cos, sin)) and np.array_equal(y[..., 32:], x[..., 32:])


def test_bounds_hold_and_scores_bound_every_key():
    rng = np.random.default_rng(4)
    for size in (1e-3, 1.0, 300.0):
        c, s = group4.encode((size * rng.standard_normal((16, 64))).astype(np.float32))
        (lo, hi), u = group4.bounds_of(c, s)
        x = group4.value(c, s)
        assert (lo * float(u) <= x).all() and (x <= hi * float(u)).all()
        assert (x - lo * float(u)).min(0).max() < u and (hi * float(u) - x).min(0).max() < u
        q = rng.integers(-127, 128, 64)
        assert np.maximum(q * lo.astype(int), q * hi.astype(int)).sum() * float(u) >= (x @ q).max()


def test_select_takes_the_best_pages_and_the_sure_ones():
    rng = np.random.default_rng(5)
    bounds = np.sort(rng.integers(-127, 128, (9, 1, 2, 64)), axis=2).astype(np.int8)
    bscale = np.exp2(rng.integers(-3, 3, (9, 1))).astype(np.float32)
    table = np.arange(9)[None]
    x = rng.standard_normal((1, 2, 64)).astype(np.float32)
    got = group4.select(x, bounds, bscale, table, [1], [9 * 16 - 3], 16, 4, first=1, last=2)[0, 0]
    c = np.rint(x[0] * 127.0 / np.abs(x).max())
    score = [float(bscale[p, 0]) * np.maximum(c * bounds[p, 0, 0], c * bounds[p, 0, 1]).sum(1).max() for p in range(9)]
    rest = max(range(1, 7), key=lambda p: (score[p], -p))
    assert got.tolist() == sorted([0, 7, 8, rest])
    assert group4.select(x, bounds, bscale, table, [1], [20], 16, 4).tolist() == [[[0, 1, -1, -1]]]


@pytest.mark.parametrize("listed", [False, True])
def test_attention_against_sdpa(listed):
    rng = np.random.default_rng(6)
    ps, H, Hq, D, n, L = 16, 2, 6, 64, 4, 45
    pools = [group4.pool_of(*group4.encode(rng.standard_normal((5, H, ps, D)).astype(np.float32))) for _ in range(2)]
    table, q = np.array([[3, 1, 0]]), rng.standard_normal((n, Hq, D))
    sel = np.array([[[0, 2], [1, 2]]] * n) if listed else None
    o, lse = group4.attend(q, pools, table, [n], [L], 0.125, selected=sel)
    kv = [torch.tensor(group4.tokens(p, table[0], L)).transpose(0, 1).repeat_interleave(3, 0) for p in pools]
    at, j = torch.arange(n)[:, None] + L - n, torch.arange(L)[None]
    mask = (j <= at)[None].repeat(Hq, 1, 1)
    if listed:
        mask[:3, :, 16:32] = False
        mask[3:, :, :16] = False
    want = torch.nn.functional.scaled_dot_product_attention(torch.tensor(q).transpose(0, 1), kv[0], kv[1], attn_mask=mask, scale=0.125)
    assert np.abs(o - want.transpose(0, 1).numpy()).max() < 1e-12
    twice, _ = group4.attend(q, pools, table, [n], [L], 0.125, selected=np.concatenate([sel, sel], -1)) if listed else (o, 0)
    assert np.abs(o - twice).max() < 1e-12
