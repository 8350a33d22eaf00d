"""GPU parity of the experts' int4 products with the oracle: one row an expert to
many, ragged sizes, gathered and sorted rows, group and column scales, zeros."""
import numpy as np
import pytest
import torch

import gemm_wq_quantize_amd as g
from oracle import routing
from test_gpu_graphs import replay_matches_eager
from tolerances import check_bf16_rows

pytestmark = pytest.mark.gpu


def say(*a):
    print("[case]", *a, flush=True)


def case(t, topk, e, n, k, group, gather=True, zeros=False, drop=0.0, seed=0, ids=None, zero_const=8.0):
    rng = np.random.default_rng(seed + t + n)
    if ids is None:
        ids = rng.integers(0, e, size=(t, topk))
        ids[rng.random(size=ids.shape) < drop] = -1
    offsets, order, _ = routing.sort_rows(ids, e)
    gen = torch.Generator().manual_seed(seed + k)
    c = dict(topk=topk, group=group, zero_const=zero_const)
    c["a"] = torch.randn((t if gather else t * topk, k), generator=gen).bfloat16()
    c["b"] = torch.randint(0, 256, (e, n, k // 2), dtype=torch.uint8, generator=gen)
    c["scales"] = (0.002 + 0.018 * torch.rand((e, n, k // group), generator=gen)).bfloat16()
    c["zeros"] = (6 + 3 * torch.rand((e, n, k // group), generator=gen)).bfloat16() if zeros else None
    c["order"] = torch.from_numpy(order) if gather else None
    c["offsets"] = torch.from_numpy(offsets)
    return c


def run(c, out, stream=None):
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    g.wq_gemm_w4a16_experts(d["a"], d["order"], d["topk"], d["offsets"], d["b"], g.LAYOUT_GFX950, d["scales"], d["zeros"],
                            d["group"], d["zero_const"], out, stream=stream)
    return out


def reference(c, slots, n, bf16_weights):
    f = lambda t: None if t is None else t.double().numpy()
    return routing.gemm_experts(f(c["a"]), None if c["order"] is None else c["order"].numpy(), c["topk"],
                                c["offsets"].numpy(), c["b"].numpy(), f(c["scales"]), f(c["zeros"]), c["zero_const"],
                                c["group"], np.full((slots, n), 2.0), bf16_weights)


def check(c, slots, n):
    """Within the bf16 bars of one of the two definitions as a whole: weights
    unrounded, or each rounded to bf16; rows behind the kept ones untouched."""
    got = run(c, torch.full((slots, n), 2.0, dtype=torch.bfloat16, device="cuda"))
    got = got.double().cpu().numpy()
    kept = int(c["offsets"][-1])
    assert np.all(got[kept:] == 2.0)
    if kept == 0:
        return
    try:
        check_bf16_rows(got[:kept], reference(c, slots, n, False)[:kept])
    except AssertionError:
        check_bf16_rows(got[:kept], reference(c, slots, n, True)[:kept])


# t, topk, experts, n, k, group
SMALL = [(1, 1, 1, 1, 64, 64), (1, 8, 64, 176, 512, 128), (3, 2, 5, 17, 192, 192), (16, 1, 1, 33, 256, 256),
         (17, 1, 1, 100, 128, 64), (40, 3, 7, 250, 384, 128), (9, 4, 130, 64, 1024, 512), (70, 1, 3, 257, 640, 640)]
LARGE = [(200, 2, 2, 300, 512, 128), (700, 2, 3, 130, 320, 64), (1000, 1, 9, 513, 256, 256), (300, 8, 4, 264, 1024, 1024),
         (1030, 4, 16, 96, 448, 448), (513, 3, 2, 1000, 2048, 2048)]


@pytest.mark.parametrize("t,topk,e,n,k,group", SMALL + LARGE)
@pytest.mark.parametrize("gather,zeros,drop", [(True, False, 0.0), (False, True, 0.3), (True, True, 0.1)])
def test_parity(t, topk, e, n, k, group, gather, zeros, drop):
    say("experts", t, topk, e, n, k, group, gather, zeros, drop)
    check(case(t, topk, e, n, k, group, gather, zeros, drop), t * topk, n)


@pytest.mark.parametrize("zero_const", [0.0, 7.5, 7.3, -3.0])
@pytest.mark.parametrize("t", [4, 400])
def test_zero_constants(t, zero_const):
    say("zero constant", t, zero_const)
    check(case(t, 2, 3, 72, 256, 128, zero_const=zero_const), t * 2, 72)


def test_empty_experts_and_dropped_rows():
    say("empty experts")
    for t in (6, 300):
        check(case(t, 2, 9, 48, 128, 128, ids=np.full((t, 2), 8)), t * 2, 48)         # all in the last
        check(case(t, 2, 9, 48, 128, 128, ids=np.full((t, 2), -1)), t * 2, 48)        # none kept
        check(case(t, 2, 700, 48, 128, 128), t * 2, 48)                               # mostly empty
        ids = np.full((t, 2), 4)
        ids[0, 1] = 2
        check(case(t, 2, 9, 48, 128, 128, ids=ids), t * 2, 48)                        # one row, and the rest


@pytest.mark.parametrize("t,e", [(5, 3), (600, 3)])
def test_integer_inputs_are_exact(t, e):
    """Small integers and power-of-two scales: every product and sum is exact in
    float32, and the result below 2^8 steps of bf16."""
    say("integers", t)
    n, k = 80, 256
    c = case(t, 1, e, n, k, 128)
    gen = torch.Generator().manual_seed(9)
    a = torch.zeros(t, k)
    at = torch.randint(0, k, (t, 4), generator=gen)
    a.scatter_(1, at, torch.randint(-2, 3, (t, 4), generator=gen).float())
    c["a"] = a.bfloat16()
    c["scales"] = torch.full_like(c["scales"], 0.5)
    got = run(c, torch.empty((t, n), dtype=torch.bfloat16, device="cuda"))
    assert np.array_equal(got.double().cpu().numpy(), reference(c, t, n, False))


@pytest.mark.parametrize("t", [3, 500])
def test_repeatable_on_a_stream_and_in_graphs(t):
    say("stream, graph", t)
    n, k = 200, 512
    c = case(t, 2, 5, n, k, 128, zeros=True)
    a = run(c, torch.empty((2 * t, n), dtype=torch.bfloat16, device="cuda"))
    st = torch.cuda.Stream()
    d = {x: v.cuda() if isinstance(v, torch.Tensor) else v for x, v in c.items()}
    out = torch.empty_like(a)
    st.wait_stream(torch.cuda.current_stream())
    call = lambda o, s=None: g.wq_gemm_w4a16_experts(d["a"], d["order"], 2, d["offsets"], d["b"], g.LAYOUT_GFX950,
                                                     d["scales"], d["zeros"], 128, 8.0, o, stream=s)
    call(out, st)
    st.synchronize()
    assert torch.equal(a, out)
    replay_matches_eager(call, out, torch.empty_like(out))


def test_large_weight_offsets():
    """The last expert's weights lie past 2^32 bytes."""
    say("large weights")
    e, n, k = 140, 8192, 8192                     # 4.7 GB of codes
    b = torch.zeros((e, n, k // 2), dtype=torch.uint8, device="cuda")
    gen = torch.Generator().manual_seed(1)
    last = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, generator=gen)
    b[-1] = last.cuda()
    scales = torch.ones((e, n, 1), dtype=torch.bfloat16, device="cuda")
    for t in (2, 300):
        a = torch.zeros((t, k)).bfloat16()
        a[:, 7] = 1.0
        a[:, 8001] = -1.0
        offsets = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
        offsets[-1] = t
        out = torch.empty((t, n), dtype=torch.bfloat16, device="cuda")
        g.wq_gemm_w4a16_experts(a.cuda(), None, 1, offsets, b, g.LAYOUT_GFX950, scales, None, k, 8.0, out)
        # element 7 of a word is nibble 7, element 1 (8001 = 8 * 1000 + 1) nibble 4
        want = (last[:, 3] >> 4).float() - (last[:, 4002] & 15).float()
        assert torch.equal(out.float().cpu(), want.expand(t, n))


@pytest.mark.parametrize("t", [4, 40, 300])
def test_rows_do_not_mix(t):
    """A row with NaN or infinity leaves the other rows' bits alone."""
    say("rows do not mix", t)
    n, k = 136, 512
    c = case(t, 1, 2, n, k, 128, gather=False)
    out = run(c, torch.empty((t, n), dtype=torch.bfloat16, device="cuda"))
    c["a"][t // 2, 7] = float("nan")
    c["a"][t - 1, 100] = float("inf")
    bad = run(c, torch.empty((t, n), dtype=torch.bfloat16, device="cuda"))
    keep = [i for i in range(t) if i not in (t // 2, t - 1)]
    assert torch.equal(out[keep], bad[keep])
    assert not torch.isfinite(bad[t // 2].float()).any() and not torch.isfinite(bad[t - 1].float()).any()


def test_a_bad_plan_stays_in_its_buffers():
    """Offsets and an order that were never written: whatever comes out, nothing
    is read or written outside, and the rows behind the output are untouched."""
    say("bad plan")
    for t in (8, 200):
        c = case(t, 2, 4, 64, 128, 128)
        c["offsets"] = torch.tensor([-5, 3, 10 ** 9, 2, 2 ** 31 - 1], dtype=torch.int32)
        c["order"] = torch.full((2 * t,), 2 ** 31 - 1, dtype=torch.int32)
        c["order"][::3] = -2 ** 31
        space = torch.zeros((2 * t + 64, 64), dtype=torch.bfloat16, device="cuda")
        run(c, space[:2 * t])
        torch.cuda.synchronize()
        assert (space[2 * t:] == 0).all()


def test_large_output_offsets():
    """Rows of the output past 2^32 bytes."""
    say("large output")
    slots, n, k, e = 300000, 8192, 64, 3
    gen = torch.Generator().manual_seed(4)
    b = torch.randint(0, 256, (e, n, k // 2), dtype=torch.uint8, generator=gen)
    a = torch.zeros((slots, k), dtype=torch.bfloat16, device="cuda")
    a[:, 3] = 2.0
    offsets = torch.tensor([0, 5, slots - 7, slots], dtype=torch.int32, device="cuda")
    out = torch.empty((slots, n), dtype=torch.bfloat16, device="cuda")
    g.wq_gemm_w4a16_experts(a, None, 1, offsets, b.cuda(), g.LAYOUT_GFX950,
                            torch.ones((e, n, 1), dtype=torch.bfloat16, device="cuda"), None, k, 8.0, out)
    for i, x in ((0, 0), (5, 1), (slots - 8, 1), (slots - 7, 2), (slots - 1, 2)):
        want = 2.0 * ((b[x, :, 2] >> 4).float() - 8.0)    # element 3 is nibble 5
        assert torch.equal(out[i].float().cpu(), want)


def test_two_streams_at_once():
    """Two calls in flight on streams of their own give what each gives alone."""
    say("two streams")
    n, k = 264, 1024
    cases = [case(t, 2, 6, n, k, 128, seed=t) for t in (500, 7)]
    alone = [run(c, torch.empty((2 * t, n), dtype=torch.bfloat16, device="cuda")) for c, t in zip(cases, (500, 7))]
    outs = [torch.empty_like(a) for a in alone]
    dev = [{x: v.cuda() if isinstance(v, torch.Tensor) else v for x, v in c.items()} for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        for d, o, st in zip(dev, outs, streams):
            g.wq_gemm_w4a16_experts(d["a"], d["order"], 2, d["offsets"], d["b"], g.LAYOUT_GFX950, d["scales"], d["zeros"],
                                    128, 8.0, o, stream=st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, o) for a, o in zip(alone, outs))
