"""GPU parity of the sort by bin and the moves with the oracle, with their
gradients, repeatability, streams and graphs."""
import numpy as np
import pytest
import torch

import gemm_wq_quantize_amd as g
from oracle import routing
from test_gpu_graphs import replay_matches_eager

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def say(*a):
    print("[case]", *a, flush=True)


def sort(ids, bins, **kw):
    offsets = torch.full((bins + 1,), -7, dtype=torch.int32, device="cuda")
    order = torch.full((ids.numel(),), -7, dtype=torch.int32, device="cuda")
    place = torch.full(tuple(ids.shape), -7, dtype=torch.int32, device="cuda")
    g.wq_sort_rows(ids, bins, offsets, order, place, **kw)
    return offsets, order, place


def check_sort(ids, bins):
    got = sort(torch.from_numpy(ids).int().cuda(), bins)
    torch.cuda.synchronize()
    for a, b in zip(got, routing.sort_rows(ids, bins)):
        assert np.array_equal(a.cpu().numpy(), b)


@pytest.mark.parametrize("t,topk,bins", [(0, 4, 5), (1, 1, 1), (1, 8, 128), (7, 9, 3), (64, 1, 2), (513, 8, 1024),
                                         (4096, 1, 64), (4097, 1, 64), (3001, 7, 257), (20000, 2, 1), (9000, 6, 513),
                                         (262145, 2, 100)])
def test_sort(t, topk, bins):
    say("sort", t, topk, bins)
    rng = np.random.default_rng(1000 * t + bins)
    check_sort(rng.integers(-1 - bins // 8, bins + bins // 8 + 1, size=(t, topk)), bins)


def test_sort_one_bin_all_dropped_and_extremes():
    say("sort extremes")
    check_sort(np.full((700, 8), 5), 9)
    check_sort(np.full((700, 8), -1), 9)
    check_sort(np.array([[2 ** 31 - 1, -2 ** 31, 0, 8, 9]] * 3), 9)
    check_sort(np.arange(9000)[::-1].reshape(-1, 1) % 1024, 1024)


def plan(t, topk, bins, drop, seed):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, bins, size=(t, topk))
    ids[rng.random(size=ids.shape) < drop] = -1
    return routing.sort_rows(ids, bins)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def close(got, ref, dtype, terms, magnitude):
    """One rounding to dtype (half a step; half the least subnormal of fp16) of a
    float32 sum of ``terms`` products, each step off by 2^-24 of ``magnitude`` =
    the sum of the absolute products."""
    got, ref = got.double().cpu().numpy(), np.asarray(ref)
    bound = (half_step(dtype) + 2.0 ** -24) * np.abs(ref) + (terms + 1) * 2.0 ** -23 * magnitude + 2.0 ** -25
    bad = np.abs(got - ref) > bound
    assert not bad.any(), f"{int(bad.sum())} of {bad.size}; worst {float((np.abs(got - ref) / bound).max()):.3g}x"


MOVES = [(1, 1, 1, "bf16"), (1, 8, 4096, "bf16"), (5, 2, 7, "f16"), (33, 8, 2048, "bf16"), (33, 3, 2056, "f32"),
         (64, 5, 64, "f16"), (17, 9, 1411, "f16"), (300, 6, 129, "bf16"), (19, 17, 515, "f32"), (6, 4, 8191, "bf16")]


@pytest.mark.parametrize("t,topk,h,dt", MOVES)
@pytest.mark.parametrize("drop", [0.0, 0.4])
def test_moves_and_gradients(t, topk, h, dt, drop):
    say("moves", t, topk, h, dt, drop)
    dtype = DT[dt]
    gen = torch.Generator().manual_seed(t * 31 + h)
    _, _, place = plan(t, topk, 11, drop, t + h)
    pl = torch.from_numpy(place).cuda()
    x = torch.randn((t, h), generator=gen).to(dtype)
    rows = torch.randn((t * topk, h), generator=gen).to(dtype)
    w = torch.randn((t, topk), generator=gen)
    # dispatch: bits, rows behind the kept ones as they were
    out = torch.full((t * topk, h), 3.0, dtype=dtype, device="cuda")
    g.wq_dispatch_rows(x.cuda(), pl, out)
    ref = routing.dispatch_rows(x.double().numpy(), place, np.full((t * topk, h), 3.0))
    assert np.array_equal(out.double().cpu().numpy(), ref)
    # combine, weighted and not
    r64, w64 = rows.double().numpy(), w.double().numpy()
    back = torch.full((t, h), float("nan"), dtype=dtype, device="cuda")
    for weights in (w, None):
        g.wq_combine_rows(rows.cuda(), pl, None if weights is None else w.cuda(), back)
        ww = None if weights is None else w64
        mag = routing.combine_rows(np.abs(r64), place, None if ww is None else np.abs(ww))
        close(back, routing.combine_rows(r64, place, ww), dtype, topk, mag)
    # gradients of the weighted combine
    d_rows = torch.full((t * topk, h), 5.0, dtype=dtype, device="cuda")
    d_w = torch.full((t, topk), float("nan"), device="cuda")
    g.wq_combine_rows_grad(x.cuda(), rows.cuda(), pl, w.cuda(), d_rows, d_w)
    rd, rw = routing.combine_rows_grad(x.double().numpy(), r64, place, w64, np.full((t * topk, h), 5.0))
    close(d_rows, rd, dtype, 1, np.abs(rd))
    _, mag = routing.combine_rows_grad(np.abs(x.double().numpy()), np.abs(r64), place, w64, np.zeros((t * topk, h)))
    # a lane's chain is at most h / 64 products long, then 8 sums across lanes and waves
    close(d_w, rw, torch.float32, h / 64 + 8, mag)
    # in place over the rows
    inplace = rows.cuda()
    g.wq_combine_rows_grad(x.cuda(), inplace, pl, w.cuda(), inplace, d_w)
    kept = place[place >= 0]
    assert torch.equal(inplace[kept], d_rows[kept])


def test_gradients_by_differences():
    """<d_out, combine> is linear in rows and weights: float32 differences of
    whole steps agree with the gradients."""
    say("differences")
    t, topk, h = 6, 3, 40
    gen = torch.Generator().manual_seed(3)
    _, _, place = plan(t, topk, 4, 0.2, 3)
    pl = torch.from_numpy(place).cuda()
    rows, w = torch.randn((t * topk, h), generator=gen).cuda(), torch.randn((t, topk), generator=gen).cuda()
    d = torch.randn((t, h), generator=gen).cuda()
    d_rows, d_w = torch.zeros_like(rows), torch.empty_like(w)
    g.wq_combine_rows_grad(d, rows, pl, w, d_rows, d_w)

    def value(rows, w):
        out = torch.empty_like(d)
        g.wq_combine_rows(rows, pl, w, out)
        return (out.double() * d.double()).sum()
    for i in range(t):
        for j in range(topk):
            step = torch.zeros_like(w)
            step[i, j] = 1.0
            diff = float(value(rows, w + step) - value(rows, w - step)) / 2
            # both values carry float32 sums of topk terms of size < 2^4 over h outputs
            assert abs(diff - float(d_w[i, j])) < h * 2.0 ** -24 * 2 ** 8
    for i in (0, 5, t * topk - 1):
        step = torch.zeros_like(rows)
        step[i] = 1.0
        diff = float(value(rows + step, w) - value(rows - step, w)) / 2
        assert abs(diff - float(d_rows[i].double().sum())) < h * 2.0 ** -24 * 2 ** 8


def test_dropped_rows_and_non_finite_values():
    say("non-finite")
    place = torch.tensor([[0, -1], [-1, -1], [1, 2]], dtype=torch.int32, device="cuda")
    rows = torch.ones((6, 24), dtype=torch.bfloat16, device="cuda")
    rows[3:] = float("nan")                     # rows that no slot goes to
    w = torch.tensor([[2.0, float("inf")], [float("nan"), 1.0], [1.0, 1.0]], device="cuda")
    out = torch.empty((3, 24), dtype=torch.bfloat16, device="cuda")
    g.wq_combine_rows(rows, place, w, out)
    assert torch.equal(out.float().cpu(), torch.tensor([[2.0], [0.0], [2.0]]).expand(3, 24))
    rows[1, 3], rows[2, 5] = float("inf"), float("nan")
    g.wq_combine_rows(rows, place, w, out)
    assert torch.isinf(out[2, 3]) and torch.isnan(out[2, 5]) and float(out[2, 4]) == 2.0
    # float32 beyond the type's range rounds to infinity
    big = torch.full((6, 24), 60000.0, dtype=torch.float16, device="cuda")
    half = torch.empty((3, 24), dtype=torch.float16, device="cuda")
    g.wq_combine_rows(big, place, w, half)
    assert torch.isinf(half[0]).all() and torch.isinf(half[2]).all() and (half[1] == 0).all()


def test_positions_outside_the_rows_are_skipped():
    say("positions outside")
    place = torch.tensor([[0, 99], [2 ** 31 - 1, 3]], dtype=torch.int32, device="cuda")
    x = torch.randn((2, 40), device="cuda")
    out = torch.zeros((4, 40), device="cuda")
    g.wq_dispatch_rows(x, place, out)
    assert torch.equal(out[0], x[0]) and torch.equal(out[3], x[1]) and (out[1:3] == 0).all()
    back = torch.empty_like(x)
    g.wq_combine_rows(out, place, None, back)
    assert torch.equal(back, x)


def test_misaligned_rows_and_streams():
    """Views that start one element in, on a stream of their own."""
    say("misaligned, stream")
    t, topk, h = 9, 4, 1000
    _, _, place = plan(t, topk, 5, 0.1, 1)
    pl = torch.from_numpy(place).cuda()
    buf = torch.randn(t * h + 1, device="cuda").bfloat16()
    x = buf[1:].view(t, h)
    space = torch.zeros(t * topk * h + 3, dtype=torch.bfloat16, device="cuda")
    out = space[3:].view(t * topk, h)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g.wq_dispatch_rows(x, pl, out, stream=st)
    ids = torch.randint(-1, 9, (70000, 1), dtype=torch.int32).cuda()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = sort(ids, 9)
    torch.cuda.current_stream().wait_stream(st)
    ref = routing.dispatch_rows(x.double().cpu().numpy(), place, np.zeros((t * topk, h)))
    assert np.array_equal(out.double().cpu().numpy(), ref) and (space[:3] == 0).all()
    for a, b in zip(got, routing.sort_rows(ids.cpu().numpy(), 9)):
        assert np.array_equal(a.cpu().numpy(), b)


def test_large_offsets():
    """Rows whose byte offsets pass 2^32."""
    say("large offsets")
    t, topk, h = 4200, 64, 8192           # 268800 rows of 16 KiB: 4.4 GB
    ids = torch.randint(0, 100, (t, topk), dtype=torch.int32, generator=torch.Generator().manual_seed(2)).cuda()
    _, _, place = sort(ids, 100)
    x = torch.randn((t, h), device="cuda").bfloat16()
    out = torch.empty((t * topk, h), dtype=torch.bfloat16, device="cuda")
    g.wq_dispatch_rows(x, place, out)
    back = torch.empty_like(x)
    g.wq_combine_rows(out, place, torch.full((t, topk), 1.0 / 64, device="cuda"), back)
    assert torch.equal(back, x)           # 64 equal terms of weight 2^-6: exact
    assert torch.equal(out[place[-1].long()], x[-1:].expand(topk, -1))


@pytest.mark.parametrize("t", [1, 2500])
def test_graphs_and_repeatability(t):
    say("graphs", t)
    topk, h, bins = 4, 1000, 37
    gen = torch.Generator().manual_seed(t)
    ids = torch.randint(-1, bins, (t, topk), dtype=torch.int32, generator=gen).cuda()

    def ints(*shape):
        return torch.empty(shape, dtype=torch.int32, device="cuda")
    outs = [(ints(bins + 1), ints(t * topk), ints(t, topk)) for _ in range(2)]
    replay_matches_eager(lambda o: g.wq_sort_rows(ids, bins, *o), *outs)
    ids.clamp_(min=0)
    place = sort(ids, bins)[2]
    x, rows = torch.randn((t, h), generator=gen).cuda().half(), torch.randn((t * topk, h), generator=gen).cuda().half()
    w = torch.randn((t, topk), generator=gen).cuda()
    replay_matches_eager(lambda o: g.wq_dispatch_rows(x, place, o), torch.empty_like(rows), torch.empty_like(rows))
    replay_matches_eager(lambda o: g.wq_combine_rows(rows, place, w, o), torch.empty_like(x), torch.empty_like(x))
    replay_matches_eager(lambda o: g.wq_combine_rows_grad(x, rows, place, w, *o),
                         (torch.empty_like(rows), torch.empty_like(w)), (torch.empty_like(rows), torch.empty_like(w)))


def test_workspace_of_the_caller():
    say("workspace")
    t, topk, bins = 5000, 3, 40
    need = g.wq_sort_rows_workspace(t, topk, bins)
    assert need > 0
    ids = torch.randint(-1, bins, (t, topk), dtype=torch.int32).cuda()
    ws = torch.full((need + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    got = sort(ids, bins, workspace=ws[:need])
    for a, b in zip(got, routing.sort_rows(ids.cpu().numpy(), bins)):
        assert np.array_equal(a.cpu().numpy(), b)
    assert (ws[need:] == 0x5A).all()
    with pytest.raises(ValueError, match="workspace"):
        sort(ids, bins, workspace=ws[:need - 4])
