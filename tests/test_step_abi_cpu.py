"""Argument checks of the serving step's entry points on a machine without a
GPU: each refusal comes before anything is launched."""
import ctypes

import pytest

FAKE = 4096      # a 16-byte aligned address that no check reads
INVALID, UNSUPPORTED, SMALL, CUDA = 1, 2, 3, 4


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
    for i, c in ((3, q.AssignParams), (4, q.RopeAxesParams), (5, q.WritePage8Params), (6, q.AttendPage8Params)):
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


def _assign(q):
    return _fill(q.AssignParams(), num_seqs=4, num_tokens=8, page_size=16, num_pages=9, bt_stride=3, num_free=5)


@pytest.mark.parametrize("change,want", [
    (dict(num_seqs=0), INVALID), (dict(num_tokens=-1), INVALID), (dict(page_size=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(bt_stride=0), INVALID), (dict(num_free=-1), INVALID), (dict(new_lens=None), INVALID), (dict(free_pages=None), INVALID),
    (dict(positions=None), INVALID), (dict(free_count_out=None), INVALID), (dict(num_seqs=8193), UNSUPPORTED),
    (dict(bt_stride=1 << 27, page_size=16), UNSUPPORTED), (dict(num_pages=1 << 27), UNSUPPORTED)])
def test_assign_refuses(q, change, want):
    assert _call(q.load().qpkv_assign_pages, _assign(q), **change) == want
    assert q.load().qpkv_assign_pages(None, None) == INVALID


def _rope(q):
    return _fill(q.RopeAxesParams(), num_tokens=3, num_heads_q=2, num_heads_kv=1, head_dim=64, rot_dim=64, num_axes=3,
                 rope_max_pos=9, pair_axis=bytes([0, 1] * 16))


@pytest.mark.parametrize("change,want", [
    (dict(num_tokens=-1), INVALID), (dict(num_heads_q=0), INVALID), (dict(num_heads_kv=0), INVALID), (dict(rot_dim=0), INVALID),
    (dict(rope_max_pos=0), INVALID), (dict(num_axes=0), UNSUPPORTED), (dict(num_axes=5), UNSUPPORTED), (dict(rot_dim=63), UNSUPPORTED),
    (dict(rot_dim=66), UNSUPPORTED), (dict(head_dim=512, rot_dim=258, pair_axis=bytes(200)), UNSUPPORTED), (dict(dtype=3), UNSUPPORTED),
    (dict(dtype=-1), UNSUPPORTED), (dict(pair_axis=None), INVALID), (dict(pair_axis=bytes([3] * 32)), INVALID), (dict(q=None), INVALID),
    (dict(k_out=None), INVALID), (dict(q=FAKE + 1), INVALID), (dict(dtype=2, q=FAKE + 2), INVALID), (dict(num_tokens=0), 0)])
def test_rope_axes_refuses(q, change, want):
    assert _call(q.load().qpkv_rope_axes, _rope(q), **change) == want


def _write(q):
    return _fill(q.WritePage8Params(), num_seqs=2, num_tokens=5, num_heads_kv=2, head_dim=128, page_size=16, num_pages=4, bt_stride=2,
                 k_stride_t=256, k_stride_h=128, v_stride_t=256, v_stride_h=128)


@pytest.mark.parametrize("change,want", [
    (dict(num_seqs=-1), INVALID), (dict(num_tokens=-1), INVALID), (dict(num_heads_kv=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(page_size=0), INVALID), (dict(page_size=24), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
    (dict(format=2), UNSUPPORTED), (dict(kv_layout=2), UNSUPPORTED), (dict(bt_stride=1 << 27), UNSUPPORTED), (dict(v=None), INVALID),
    (dict(k=FAKE + 8), INVALID), (dict(k_stride_t=257), INVALID), (dict(v_stride_h=4), INVALID), (dict(v_scale=None), INVALID),
    (dict(num_tokens=0), 0), (dict(num_seqs=0), 0)])
def test_write_page8_refuses(q, change, want):
    assert _call(q.load().qpkv_write_page8, _write(q), **change) == want


def _attend(q):
    n = q.load().qpkv_attend_page8_workspace_bytes(2, 5, 8, 2, 128)
    assert n > 0
    return _fill(q.AttendPage8Params(), num_seqs=2, num_tokens=5, num_heads_q=8, num_heads_kv=2, head_dim=128, page_size=16,
                 num_pages=4, bt_stride=2, workspace_bytes=n)


@pytest.mark.parametrize("change,want", [
    (dict(num_seqs=-1), INVALID), (dict(num_tokens=-1), INVALID), (dict(num_heads_q=0), INVALID), (dict(window=-1), INVALID),
    (dict(logit_cap=-1.0), INVALID), (dict(logit_cap=float("nan")), INVALID), (dict(logit_cap=float("inf")), INVALID), (dict(logit_cap=1e-30), INVALID),
    (dict(sm_scale=float("nan")), INVALID), (dict(num_heads_q=7), UNSUPPORTED), (dict(head_dim=80), UNSUPPORTED),
    (dict(page_size=8), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(format=-1), UNSUPPORTED), (dict(kv_layout=5), UNSUPPORTED),
    (dict(bt_stride=1 << 27), UNSUPPORTED), (dict(num_tokens=1 << 30), UNSUPPORTED), (dict(q=None), INVALID), (dict(o=FAKE + 4), INVALID),
    (dict(workspace=None), INVALID), (dict(workspace=FAKE + 1), INVALID), (dict(workspace_bytes=64), SMALL), (dict(num_tokens=0), 0),
    (dict(num_seqs=0), 0)])
def test_attend_page8_refuses(q, change, want):
    assert _call(q.load().qpkv_attend_page8, _attend(q), **change) == want


def test_attend_workspace_sizes(q):
    f = q.load().qpkv_attend_page8_workspace_bytes
    assert f(-1, 5, 8, 2, 128) == f(2, -1, 8, 2, 128) == f(2, 5, 7, 2, 128) == f(2, 5, 8, 2, 96) == 0
    assert f(2, 5, 8, 2, 128) <= f(4000, 5, 8, 2, 128) and f(64, 64, 32, 8, 64) < f(64, 64, 32, 8, 128)


def test_axis_sections(q):
    assert q.axis_sections((2, 1, 3)) == bytes([0, 0, 1, 2, 2, 2])
    assert q.axis_sections((4, 2, 1), interleaved=True) == bytes([0, 1, 2, 0, 1, 0, 0])
    assert q.axis_sections((1, 3), interleaved=True) == bytes([0, 1, 1, 1])
    for bad in ((), (1, 2, 3, 4, 5), (2, -1)):
        with pytest.raises(ValueError):
            q.axis_sections(bad)
