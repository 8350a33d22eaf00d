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


def test_experts_refusals(lib):
    def f(a=FAKE, rows=4, order=FAKE, topk=2, off=FAKE, slots=8, e=3, b=FAKE, layout=1, s=FAKE, zr=None, group=128,
          n=40, k=256, c=FAKE):
        return lib.wq_gemm_w4a16_experts(a, rows, order, topk, off, slots, e, b, layout, s, zr, group, 8.0, n, k, c,
                                         None)
    assert f(a=None, off=None, slots=0, rows=0) == g.WQ_OK and f(a=None, n=0) == g.WQ_OK
    for kw in (dict(a=None), dict(off=None), dict(b=None), dict(s=None), dict(c=None), dict(rows=-1), dict(e=-1),
               dict(layout=2), dict(k=-64)):
        assert f(**kw) == g.WQ_EINVAL, kw
    for kw in (dict(e=0), dict(e=1025), dict(k=0), dict(k=96, group=96), dict(k=(1 << 22) + 64), dict(group=96),
               dict(group=512), dict(rows=3), dict(topk=0), dict(order=None, rows=4), dict(n=1 << 30),
               dict(rows=1 << 23, slots=1 << 24), dict(rows=1 << 24, topk=2, slots=1 << 25)):
        assert f(**kw) == g.WQ_ESHAPE, kw
    assert f(order=None, rows=1 << 25, slots=1 << 25) == g.WQ_ESHAPE
    assert f(rows=(1 << 31) // (2 * 8192), topk=1, slots=(1 << 31) // (2 * 8192), k=8192) == g.WQ_ESHAPE
    assert f(layout=0) == g.WQ_EUNSUPPORTED and f(group=32) == g.WQ_EUNSUPPORTED
    for kw in (dict(a=ODD), dict(b=P(0x1008)), dict(c=P(0x1008)), dict(s=HALF), dict(zr=HALF), dict(order=HALF),
               dict(off=HALF)):
        assert f(**kw) == g.WQ_EALIGN, kw


def test_experts_binding_refusals():
    i32, bf, u8 = torch.int32, torch.bfloat16, torch.uint8
    args = dict(a=z((4, 256), bf), order=z(8, i32), topk=2, offsets=z(4, i32), b=z((3, 40, 128), u8), layout=1,
                scales=z((3, 40, 2), bf), zeros=None, group=128, zero_const=8.0, c_out=z((8, 40), bf))
    for kw, match in ((dict(a=z((4, 256), torch.float32)), "bf16"), (dict(b=z((3, 40, 127), u8)), "b is uint8"),
                      (dict(c_out=z((8, 39), bf)), "c_out"), (dict(scales=z((3, 40, 1), bf)), "scales"),
                      (dict(scales=z((3, 40, 2), torch.float32)), "scales"), (dict(group=0), "scales"),
                      (dict(zeros=z((3, 40, 1), bf)), "zeros"), (dict(offsets=z(3, i32)), "offsets"),
                      (dict(offsets=z(4, torch.int64)), "int32"), (dict(order=z(7, i32)), "order"),
                      (dict(topk=1), "order"), (dict(order=None), "without order")):
        with pytest.raises(ValueError, match=match):
            g.wq_gemm_w4a16_experts(**{**args, **kw})


def test_lora_refusals(lib):
    ws = lib.wq_lora_workspace
    assert ws(1, 4096, 8, 16) > 0 and ws(0, 64, 1, 8) == 0
    assert ws(-1, 64, 1, 8) == g.WQ_EINVAL
    for t, k, l, r in ((4, 48, 1, 8), (4, 0, 1, 8), (4, (1 << 24) + 32, 1, 8), (4, 64, 0, 8), (4, 64, 1025, 8),
                       (4, 64, 1, 0), (4, 64, 1, 12), (4, 64, 1, 136), ((1 << 24) + 1, 64, 1, 8)):
        assert ws(t, k, l, r) == g.WQ_ESHAPE

    def f(x=FAKE, t=4, k=64, order=FAKE, off=FAKE, l=3, a=FAKE, b=FAKE, r=16, s=FAKE, base=FAKE, out=FAKE, dt=2, n=40,
          w=FAKE, nb=1 << 40):
        return lib.wq_lora(x, t, k, order, off, l, a, b, r, s, base, out, dt, n, w, nb, None)
    assert f(t=0, x=None, out=None) == g.WQ_OK and f(n=0, out=None) == g.WQ_OK
    for kw in (dict(x=None), dict(order=None), dict(off=None), dict(a=None), dict(b=None), dict(s=None),
               dict(out=None), dict(w=None), dict(dt=1), dict(n=-1), dict(t=-1), dict(nb=255)):
        assert f(**kw) == g.WQ_EINVAL, kw
    for kw in (dict(k=40), dict(r=20), dict(r=256), dict(l=0), dict(n=1 << 31), dict(t=1 << 24, n=(1 << 31) - 1)):
        assert f(**kw) == g.WQ_ESHAPE, kw
    for kw in (dict(x=P(0x1008)), dict(a=HALF), dict(b=P(0x1008)), dict(w=P(0x1008)), dict(order=HALF), dict(off=ODD),
               dict(s=HALF), dict(base=ODD), dict(out=ODD), dict(dt=0, out=HALF)):
        assert f(**kw) == g.WQ_EALIGN, kw


def test_lora_binding_refusals():
    i32, bf, f32 = torch.int32, torch.bfloat16, torch.float32
    args = dict(x=z((4, 64), bf), order=z(4, i32), offsets=z(4, i32), a=z((3, 16, 64), bf), b=z((3, 40, 16), bf),
                scales=z(3, f32), base=z((4, 40), bf), out=z((4, 40), bf))
    for kw, match in ((dict(x=z((4, 64), f32)), "bf16"), (dict(a=z((3, 16, 32), bf)), "a is"),
                      (dict(b=z((2, 40, 16), bf)), "a is"), (dict(b=z((3, 40, 8), bf)), "a is"),
                      (dict(out=z((4, 39), bf)), "out is"), (dict(base=z((4, 40), f32)), "base"),
                      (dict(scales=z(2, f32)), "scales"), (dict(scales=z(3, bf)), "scales"),
                      (dict(order=z(5, i32)), "order"), (dict(offsets=z(3, i32)), "offsets"),
                      (dict(order=z(4, torch.int64)), "int32")):
        with pytest.raises(ValueError, match=match):
            g.wq_lora(**{**args, **kw})


def test_more_workgroups_than_a_launch_holds(lib):
    """2^32 lanes and more: refused before anything is enqueued."""
    d = lambda t, h, dt=2: lib.wq_dispatch_rows(FAKE, dt, FAKE, t, 1, h, FAKE, None)
    c = lambda t, h, dt=2, w=FAKE: lib.wq_combine_rows(FAKE, dt, FAKE, w, t, 1, h, FAKE, None)
    for f in (d, c):
        assert f(1 << 20, 32768) == g.WQ_ESHAPE            # 2^24 pieces of 4 KiB
        assert f(1 << 24, 1025) == g.WQ_ESHAPE             # a workgroup a row
        assert f(1 << 24, 2048, dt=1) == g.WQ_ESHAPE
        assert f(1 << 20, 16384, dt=0) == g.WQ_ESHAPE
    assert c(1 << 20, 32768, w=None) == g.WQ_ESHAPE
    for dt, h in ((2, 1025), (1, 4096), (0, 513)):
        assert lib.wq_combine_rows_grad(FAKE, FAKE, dt, FAKE, FAKE, 1 << 24, 1, h, FAKE, FAKE, None) == g.WQ_ESHAPE
    e = lambda slots, experts, n: lib.wq_gemm_w4a16_experts(FAKE, slots, None, 1, FAKE, slots, experts, FAKE, 1, FAKE,
                                                            None, 64, 8.0, n, 64, FAKE, None)
    assert e(1024, 1024, (1 << 21) - 1) == g.WQ_ESHAPE     # 1024 row tiles x 2^15 of 64 columns
    assert e(1 << 24, 1, 40000) == g.WQ_ESHAPE             # 2^17 row tiles x 157 of 256 columns
    lo = lambda t, adapters, n: lib.wq_lora(FAKE, t, 64, FAKE, FAKE, adapters, FAKE, FAKE, 16, FAKE, FAKE, FAKE, 2, n,
                                            FAKE, 1 << 40, None)
    assert lo(1 << 24, 1, 1 << 15) == g.WQ_ESHAPE          # (2^19 + 2) row tiles x 32 of 1024 columns
    assert lo(1 << 10, 1024, 1 << 25) == g.WQ_ESHAPE       # 1024 row tiles x 2^15 of 1024 columns
