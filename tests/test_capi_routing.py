"""Refusals of the routed-rows entry points: argument errors of the C calls and
of the binding, with no GPU (every call fails validation or is empty)."""
import ctypes
import os

import pytest
import torch

import gemm_wq_quantize_amd as g


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(g.LIB_PATH):
        from gemm_wq_quantize_amd import build
        build.build()
    return g.load_library()


P = ctypes.c_void_p
FAKE, ODD, HALF = P(0x1000), P(0x1001), P(0x1002)


def z(shape, dtype):
    return torch.zeros(shape, dtype=dtype)


def test_sort_refusals(lib):
    ws = lib.wq_sort_rows_workspace
    assert ws(1, 8, 64) == 0 and ws(0, 8, 64) == 0
    assert ws(1 << 16, 8, 64) > 0
    assert ws(-1, 8, 64) == g.WQ_EINVAL
    assert ws(1, 8, 0) == g.WQ_ESHAPE and ws(1, 8, 1025) == g.WQ_ESHAPE and ws(1, 8, 1024) == 0
    assert ws(1 << 24, 2, 64) == g.WQ_ESHAPE and ws(1 << 62, 1 << 62, 64) == g.WQ_ESHAPE
    sort = lambda t, k, b, ids=FAKE, off=FAKE, order=FAKE, place=FAKE, w=FAKE, n=1 << 40: lib.wq_sort_rows(
        ids, t, k, b, off, order, place, w, n, None)
    assert sort(4, 2, 0) == g.WQ_ESHAPE
    assert sort(4, 2, 8, ids=None) == g.WQ_EINVAL
    assert sort(4, 2, 8, off=None) == g.WQ_EINVAL
    assert sort(4, 2, 8, place=HALF) == g.WQ_EALIGN
    assert sort(1 << 16, 8, 8, n=4) == g.WQ_EINVAL      # workspace too small
    assert sort(1 << 16, 8, 8, w=None) == g.WQ_EINVAL
    assert sort(1 << 16, 8, 8, w=ODD) == g.WQ_EALIGN


def test_move_refusals(lib):
    d = lambda t, k, h, dt=2, x=FAKE, pl=FAKE, o=FAKE: lib.wq_dispatch_rows(x, dt, pl, t, k, h, o, None)
    c = lambda t, k, h, dt=2, x=FAKE, pl=FAKE, w=FAKE, o=FAKE: lib.wq_combine_rows(x, dt, pl, w, t, k, h, o, None)
    r = lambda t, k, h, dt=2, w=FAKE, dw=FAKE, x=FAKE: lib.wq_combine_rows_grad(x, FAKE, dt, FAKE, w, t, k, h, FAKE, dw,
                                                                               None)
    for f in (d, c):
        assert f(0, 2, 8, x=None, pl=None, o=None) == g.WQ_OK
        assert f(4, 2, 0, x=None, pl=None, o=None) == g.WQ_OK
        assert f(4, 2, 8, x=None) == g.WQ_EINVAL and f(4, 2, 8, o=None) == g.WQ_EINVAL
        assert f(4, 2, 8, pl=None) == g.WQ_EINVAL
        assert f(-4, 2, 8) == g.WQ_EINVAL and f(4, 2, 8, dt=3) == g.WQ_EINVAL
        assert f(1 << 23, 4, 8) == g.WQ_ESHAPE and f(4, 2, 1 << 31) == g.WQ_ESHAPE
        assert f(1 << 23, 1, (1 << 31) - 1) == g.WQ_ESHAPE   # more workgroups than a grid holds
        assert f(4, 2, 8, x=ODD) == g.WQ_EALIGN and f(4, 2, 8, dt=0, o=HALF) == g.WQ_EALIGN
        assert f(4, 2, 8, pl=HALF) == g.WQ_EALIGN
    assert d(4, 0, 8) == g.WQ_OK and c(4, 0, 8) == g.WQ_ESHAPE
    assert c(4, 2, 8, w=HALF) == g.WQ_EALIGN
    assert r(0, 2, 8) == g.WQ_OK and r(4, 0, 8) == g.WQ_OK and r(4, 2, 0) == g.WQ_ESHAPE
    assert r(4, 2, 8, w=None) == g.WQ_EINVAL and r(4, 2, 8, dw=None) == g.WQ_EINVAL
    assert r(4, 2, 8, dt=0, x=HALF) == g.WQ_EALIGN and r(4, 2, 8, dw=HALF) == g.WQ_EALIGN


def test_binding_refusals():
    i32, f32, bf = torch.int32, torch.float32, torch.bfloat16
    ids = z((4, 2), i32)
    with pytest.raises(ValueError, match="offsets"):
        g.wq_sort_rows(ids, 3, z(3, i32), z(8, i32), z(8, i32))
    with pytest.raises(ValueError, match="order and place"):
        g.wq_sort_rows(ids, 3, z(4, i32), z(7, i32), z(8, i32))
    with pytest.raises(ValueError, match="int32"):
        g.wq_sort_rows(ids.long(), 3, z(4, i32), z(8, i32), z(8, i32))
    with pytest.raises(ValueError, match="sorted rows"):
        g.wq_dispatch_rows(z((4, 16), bf), ids, z((7, 16), bf))
    with pytest.raises(ValueError, match="one dtype"):
        g.wq_dispatch_rows(z((4, 16), bf), ids, z((8, 16), f32))
    with pytest.raises(ValueError, match="place"):
        g.wq_combine_rows(z((8, 16), bf), z((3, 2), i32), None, z((4, 16), bf))
    with pytest.raises(ValueError, match="weights"):
        g.wq_combine_rows(z((8, 16), bf), ids, z((4, 2), bf), z((4, 16), bf))
    with pytest.raises(ValueError, match="weights"):
        g.wq_combine_rows_grad(z((4, 16), bf), z((8, 16), bf), ids, z((4, 2), f32), z((8, 16), bf), z((4, 1), f32))
    with pytest.raises(ValueError, match="sorted rows"):
        g.wq_combine_rows_grad(z((4, 16), bf), z((8, 16), bf), ids, z((4, 2), f32), z((8, 15), bf), z((4, 2), f32))
