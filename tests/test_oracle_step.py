"""Pins of the serving step's oracle on the CPU: page assignment against a
brute-force allocator's invariants, rotary axes against one-axis RoPE and
complex rotation, the page-scaled write against its error bound, attention
against torch's scaled_dot_product_attention in float64."""
import numpy as np
import pytest
import torch

from oracle import rope, step


def _assign(seed, B=9, W=7, ps=16, free=40, T=None):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, W * ps // 2, B).astype(np.int32)
    new = rng.integers(0, W * ps // 2, B).astype(np.int32)
    perm = rng.permutation(200).astype(np.int32)
    table = np.full((B, W), -1, np.int32)
    at = 0
    for b in range(B):
        n = -(-int(lens[b]) // ps)
        table[b, :n] = perm[at:at + n]
        at += n
    pages = np.full(100, -7, np.int32)
    pages[:free] = perm[at:at + free]
    return new, lens, table, pages, free, ps, int(new.sum()) if T is None else T


@pytest.mark.parametrize("seed", range(4))
def test_assigned_pages_are_distinct_and_slots_follow_the_table(seed):
    new, lens, table, pages, free, ps, T = _assign(seed)
    out, grown, left, cu, slots, pos, refused = step.assign_pages(new, lens, table, pages, free, ps, T)
    assert not refused
    used = out[out >= 0]
    assert len(set(used.tolist())) == len(used)
    assert set(used.tolist()).isdisjoint(pages[:left].tolist())
    assert np.array_equal(grown, lens + new) and cu[-1] == T
    assert np.array_equal((out >= 0).sum(1), -(-grown // ps))
    assert len(set(slots.tolist())) == T and (slots >= 0).all()


def test_assignment_refuses_in_order_when_pages_run_out():
    new, lens, table, pages, _, ps, T = _assign(1)
    need = -(-(lens + new) // ps) + (-lens // ps)
    cum = np.cumsum(need)
    free = int(cum[4])
    out, grown, left, _, slots, _, refused = step.assign_pages(new, lens, table, pages, free, ps, T)
    assert refused == [b for b in range(5, len(new)) if need[b] > 0] and left == 0
    for b in refused:
        assert grown[b] == lens[b] and np.array_equal(out[b], table[b])


def test_rope_axes_with_equal_positions_is_one_axis_rope_and_inverse_undoes_it():
    rng = np.random.default_rng(0)
    cos, sin = rope.cos_sin_table(50, 32, 1e4)
    x = rng.standard_normal((7, 3, 32)).astype(np.float32)
    p = rng.integers(0, 50, 7)
    axis = bytes([0] * 5 + [1] * 6 + [2] * 5)
    y = step.rope_axes(x, np.stack([p, p, p]), axis, cos, sin)
    assert np.array_equal(y, rope.rotate(x, p, cos, sin))
    back = step.rope_axes(y, np.stack([p, p, p]), axis, cos, sin, inverse=True)
    assert np.abs(back - x).max() <= 8 * 2.0 ** -24 * np.abs(x).max()
    q = np.stack([p, rng.integers(0, 50, 7), rng.integers(0, 50, 7)])
    z = step.rope_axes(x, q, axis, cos, sin)
    for i, a in enumerate(axis):
        w = (x[..., i] + 1j * x[..., 16 + i]) * (cos[q[a], i] + 1j * sin[q[a], i])[:, None]
        assert np.allclose(z[..., i], w.real, atol=1e-6) and np.allclose(z[..., 16 + i], w.imag, atol=1e-6)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_page_write_keeps_values_within_its_steps(fmt):
    """One write: half a step of the code.  A rescaled code was rounded twice:
    twice half a step (in units of the final scale)."""
    rng = np.random.default_rng(3)
    ps, H, D, n0, n1 = 16, 2, 64, 5, 20
    x = rng.standard_normal((n0 + n1, H, D)).astype(np.float32)
    x[n0:] *= 4
    table = np.array([[2, 0]])
    zero = np.zeros((3, ps, H, D), np.uint8 if fmt == "e4m3" else np.int8)
    pools, scales = (zero.copy(), zero.copy()), (np.zeros((3, H), np.float32), np.zeros((3, H), np.float32))
    step.write_page8(x[:n0], x[:n0], [n0], [0], table, pools, scales, fmt)
    step.write_page8(x[n0:], x[n0:], [n1], [n0], table, pools, scales, fmt)
    s = scales[0][table[0]]
    got = (step.decode(pools[0][table[0]]) * s[:, None, :, None]).reshape(-1, H, D)[:n0 + n1]
    sc = np.repeat(s, ps, axis=0)[:n0 + n1, :, None]
    if fmt == "int8":
        half = 0.5 * sc
    else:
        half = np.maximum(np.abs(x) * 2.0 ** -4, sc * 2.0 ** -10)
    times = np.where(np.arange(n0 + n1) < n0, 2.2, 1.01)[:, None, None]   # (1 + 2^-4)^2 - 1 < 2.2 * 2^-4
    assert (np.abs(got - x) <= times * half).all()


def test_page_write_leaves_out_a_sequence_that_starts_at_minus_one():
    """A request that the page assignment refused, between two served ones."""
    rng = np.random.default_rng(4)
    ps, H, D, cu, table = 16, 1, 64, [3, 23, 28], np.array([[2, -1], [0, -1], [1, -1]])
    x = rng.standard_normal((28, H, D)).astype(np.float32)
    x[3:23] = 1e20
    pools = tuple(rng.integers(-127, 128, (3, ps, H, D)).astype(np.int8) for _ in range(2))
    scales = tuple(rng.uniform(0.01, 0.03, (3, H)).astype(np.float32) for _ in range(2))
    before = [a.copy() for a in pools + scales]
    step.write_page8(x, x, cu, [4, -1, 0], table, pools, scales, "int8")
    want = [a.copy() for a in before]
    rest = np.r_[0:3, 23:28]
    step.write_page8(x[rest], x[rest], [3, 8], [4, 0], table[[0, 2]], want[:2], want[2:], "int8")
    for got, w, old in zip(pools + scales, want, before):
        assert np.array_equal(got, w) and np.array_equal(got[0], old[0]) and not np.array_equal(got, old)


@pytest.mark.parametrize("causal,window,prefix", [(True, 0, 0), (True, 5, 0), (True, 0, 9), (False, 0, 0)])
def test_page_attention_against_sdpa(causal, window, prefix):
    rng = np.random.default_rng(5)
    ps, H, Hq, D, n, L = 16, 2, 6, 64, 4, 21
    pools = tuple(rng.integers(-127, 128, (4, ps, H, D)).astype(np.int8) for _ in range(2))
    scales = tuple(rng.uniform(0.01, 0.03, (4, H)).astype(np.float32) for _ in range(2))
    table, q = np.array([[3, 1]]), rng.standard_normal((n, Hq, D))
    o, lse = step.attend_page8(q, pools, scales, table, [n], [L], 0.125, causal=causal, window=window,
                               prefix=np.array([prefix]))
    kv = [torch.tensor((p[table[0]] * s[table[0]].astype(np.float64)[:, None, :, None]).reshape(-1, H, D)[:L])
          .transpose(0, 1).repeat_interleave(3, 0) for p, s in zip(pools, scales)]
    at, j = torch.arange(n)[:, None] + L - n, torch.arange(L)[None]
    mask = ((j <= at) | (j < prefix)) if causal else torch.ones(n, L, dtype=torch.bool)
    if window:
        mask = mask & (j > at - window)
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.tensor(q).transpose(0, 1), kv[0], kv[1], attn_mask=mask, scale=0.125)
    assert np.abs(o - want.transpose(0, 1).numpy()).max() < 1e-12
    x = torch.einsum("nhd,hld->nhl", torch.tensor(q), kv[0]) * 0.125
    x = x.masked_fill(~mask[:, None], -np.inf)
    assert np.abs(lse - torch.logsumexp(x, -1).numpy()).max() < 1e-12
