"""GPU parity of the low-rank adapters with the oracle, and the operators run
together: a mixture layer on int4 experts, and adapters beside an int4 projection."""
import numpy as np
import pytest
import torch

import gemm_wq_quantize_amd as g
from oracle import int4, routing
from test_gpu_graphs import replay_matches_eager

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def say(*a):
    print("[case]", *a, flush=True)


def case(t, k, n, adapters, rank, dt="bf16", drop=0.2, base=True, seed=0, ids=None):
    rng = np.random.default_rng(seed + t + n)
    if ids is None:
        ids = rng.integers(0, adapters, size=t)
        ids[rng.random(size=t) < drop] = -1
    offsets, order, _ = routing.sort_rows(ids.reshape(-1, 1), adapters)
    gen = torch.Generator().manual_seed(seed + k)
    rand = lambda *s: torch.randn(s, generator=gen)
    c = dict(x=rand(t, k).bfloat16(), order=torch.from_numpy(order), offsets=torch.from_numpy(offsets),
             a=(rand(adapters, rank, k) * k ** -0.5).bfloat16(), b=(0.3 * rand(adapters, n, rank)).bfloat16(),
             scales=rand(adapters), base=rand(t, n).to(DT[dt]) if base else None)
    return c, ids


def run(c, out, **kw):
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in c.items()}
    g.wq_lora(d["x"], d["order"], d["offsets"], d["a"], d["b"], d["scales"], d["base"], out, **kw)
    return out


def check(c, ids, dt):
    t, n, k = c["x"].shape[0], c["b"].shape[1], c["x"].shape[1]
    got = run(c, torch.full((t, n), float("nan"), dtype=DT[dt], device="cuda")).double().cpu().numpy()
    f = lambda v: v.double().numpy()
    base = np.zeros((t, n)) if c["base"] is None else f(c["base"])
    ref = routing.lora(f(c["x"]), ids, f(c["a"]), f(c["b"]), f(c["scales"]), base)
    # one rounding to the output's type; float32 sums whose roundings (2^-24 of the
    # absolute products' sum each) walk at random: eight deviations of sqrt(k)
    # steps; a[l] x carried to the second product within 2^-17 (bf16 out) or 2^-24
    mag = routing.lora(np.abs(f(c["x"])), ids, np.abs(f(c["a"])), np.abs(f(c["b"])), np.abs(f(c["scales"])), 0 * base)
    low = np.zeros((t, n))
    a, b, x = f(c["a"]), np.abs(f(c["b"])), f(c["x"])
    for i, l in enumerate(ids):
        if 0 <= l < a.shape[0]:
            low[i] = abs(float(c["scales"][l])) * (b[l] @ np.abs(a[l] @ x[i]))
    bound = torch.finfo(DT[dt]).eps / 2 * (np.abs(ref) + np.abs(ref - base) * 2.0 ** -8)
    bound += 8 * np.sqrt(k) * 2.0 ** -24 * mag + 2.0 ** (-17 if dt == "bf16" else -24) * low + 2.0 ** -24 * np.abs(base)
    bad = np.abs(got - ref) > bound
    assert not bad.any(), f"{int(bad.sum())} of {bad.size}; worst {np.nanmax(np.abs(got - ref) / (bound + 1e-300)):.3g}x"
    none = (ids < 0) | (ids >= c["a"].shape[0])
    assert np.array_equal(got[none], base[none])


SIZES = [(1, 32, 1, 1, 8), (1, 4096, 5120, 64, 16), (7, 96, 33, 3, 24), (33, 512, 260, 40, 16), (64, 1024, 1000, 2, 64),
         (100, 320, 127, 5, 128), (40, 2560, 136, 600, 32), (1025, 256, 257, 3, 8), (1500, 512, 384, 30, 64),
         (2000, 288, 200, 1000, 40), (1100, 608, 130, 2, 104),
         (4100, 96, 100, 5, 24), (8200, 160, 72, 40, 128)]


@pytest.mark.parametrize("t,k,n,adapters,rank", SIZES)
@pytest.mark.parametrize("dt,base,drop", [("bf16", True, 0.2), ("f32", True, 0.0), ("bf16", False, 0.5)])
def test_parity(t, k, n, adapters, rank, dt, base, drop):
    say("lora", t, k, n, adapters, rank, dt, base, drop)
    c, ids = case(t, k, n, adapters, rank, dt, drop, base)
    check(c, ids, dt)


def test_all_or_none_have_an_adapter():
    say("one adapter, none")
    for t in (5, 1200):
        for fill in (0, 2, -1, 99):
            c, ids = case(t, 64, 72, 3, 16, ids=np.full(t, fill))
            check(c, ids, "bf16")


@pytest.mark.parametrize("t", [9, 1300])
def test_base_in_place_and_its_bits(t):
    say("in place", t)
    c, ids = case(t, 128, 77, 4, 16, drop=0.5)
    none = torch.from_numpy(ids < 0)
    c["base"][none] = -0.0
    c["base"][none, 3] = float("nan")
    c["base"][none, 4] = float("inf")
    c["x"][none] = float("nan")               # rows that no product reads
    out = run(c, torch.empty((t, 77), dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(out.cpu()[none].view(torch.int16), c["base"][none].view(torch.int16))
    assert torch.isfinite(out.cpu()[~none]).all()
    d = c["base"].cuda()
    c["base"] = d
    run(c, d)
    assert torch.equal(d.view(torch.int16), out.view(torch.int16))


@pytest.mark.parametrize("t", [12, 1100])
def test_streams_workspace_and_graphs(t):
    say("stream, workspace, graph", t)
    c, _ = case(t, 512, 264, 6, 32)
    d = {k: v.cuda() for k, v in c.items()}
    ref = run(c, torch.empty((t, 264), dtype=torch.bfloat16, device="cuda"))
    need = g.wq_lora_workspace(t, 512, 6, 32)
    ws = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    call = lambda o, **kw: g.wq_lora(d["x"], d["order"], d["offsets"], d["a"], d["b"], d["scales"], d["base"], o, **kw)
    out = torch.empty_like(ref)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    call(out, workspace=ws[:need], stream=st)
    st.synchronize()
    assert torch.equal(out, ref) and (ws[need:] == 0x5A).all()
    out.zero_()
    st.wait_stream(torch.cuda.current_stream())
    call(out, stream=st)                       # workspace from the allocator, on that stream
    st.synchronize()
    assert torch.equal(out, ref)
    with pytest.raises(ValueError, match="workspace"):
        call(out, workspace=ws[:need - 4])
    replay_matches_eager(call, out, torch.empty_like(out))


def test_large_offsets():
    """Adapters and rows past 2^32 bytes."""
    say("large offsets")
    k, n, rank, adapters, t = 16384, 16384, 128, 1024, 4
    a = torch.zeros((adapters, rank, k), dtype=torch.bfloat16, device="cuda")   # 4.3 GB each
    b = torch.zeros((adapters, n, rank), dtype=torch.bfloat16, device="cuda")
    a[-1, 5, 9000] = 2.0
    b[-1, :, 5] = torch.arange(n, device="cuda") % 64
    x = torch.ones((t, k), dtype=torch.bfloat16, device="cuda")
    offsets = torch.zeros(adapters + 1, dtype=torch.int32, device="cuda")
    offsets[-1] = t
    order = torch.arange(t, dtype=torch.int32, device="cuda")
    out = torch.empty((t, n), dtype=torch.float32, device="cuda")
    g.wq_lora(x, order, offsets, a, b, torch.ones(adapters, device="cuda"), None, out)
    assert torch.equal(out, (2.0 * (torch.arange(n, device="cuda") % 64)).expand(t, n))


def test_a_bad_plan_stays_in_its_buffers():
    say("bad plan")
    for t in (9, 1500):
        c, _ = case(t, 64, 40, 3, 16)
        c["offsets"] = torch.tensor([-7, 10 ** 9, 3, 2 ** 31 - 1], dtype=torch.int32)
        c["order"] = torch.full((t,), 2 ** 31 - 1, dtype=torch.int32)
        c["order"][::2] = -5
        space = torch.zeros((t + 64, 40), dtype=torch.bfloat16, device="cuda")
        run(c, space[:t])
        torch.cuda.synchronize()
        assert (space == 0).all()              # no row of the order exists


def test_refusals_on_the_device():
    say("refusals")
    c, _ = case(5, 64, 40, 3, 16)
    d = {k: v.cuda() for k, v in c.items()}
    out = torch.zeros((5, 40), dtype=torch.bfloat16, device="cuda")
    call = lambda **kw: g.wq_lora(**{**d, "out": out, **kw})
    with pytest.raises(ValueError, match="on the GPU"):
        call(x=c["x"])
    with pytest.raises(ValueError, match="contiguous"):
        call(base=torch.zeros((40, 5), dtype=torch.bfloat16, device="cuda").T)
    with pytest.raises(g.WqError, match="ESHAPE"):
        call(a=torch.zeros((3, 20, 64), dtype=torch.bfloat16, device="cuda"),
             b=torch.zeros((3, 40, 20), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(g.WqError, match="EALIGN"):
        call(workspace=torch.zeros(4096, dtype=torch.uint8, device="cuda")[4:])
    assert (out == 0).all()


def weights(e, n, k, gen):
    w = (0.02 * torch.randn((e * n, k), generator=gen)).half().cuda()
    packed = torch.empty((e * n, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((e * n, k // 128), dtype=torch.bfloat16, device="cuda")
    g.wq_quantize_pack_int4(w, 128, g.LAYOUT_GFX950, packed, scales)
    return packed.view(e, n, k // 2), scales.view(e, n, k // 128)


@pytest.mark.parametrize("t", [1, 3, 300])
def test_mixture_layer(t):
    """Router choices -> sort -> experts (gate and up) -> gated product -> experts
    (down) -> combine, on weights from the library's own quantiser."""
    say("mixture layer", t)
    e, topk, h, inter = 6, 2, 512, 384
    gen = torch.Generator().manual_seed(t)
    w1, s1 = weights(e, 2 * inter, h, gen)
    w2, s2 = weights(e, h, inter, gen)
    x = torch.randn((t, h), generator=gen).bfloat16().cuda()
    chosen = torch.topk(torch.randn((t, e), generator=gen), topk, dim=1)
    ids, router = chosen.indices.int().cuda(), torch.softmax(chosen.values, 1).cuda()
    ints = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")
    offsets, order, place = ints(e + 1), ints(t * topk), ints(t, topk)
    up = torch.empty((t * topk, 2 * inter), dtype=torch.bfloat16, device="cuda")
    down = torch.empty((t * topk, h), dtype=torch.bfloat16, device="cuda")

    def layer(out):
        g.wq_sort_rows(ids, e, offsets, order, place)
        g.wq_gemm_w4a16_experts(x, order, topk, offsets, w1, g.LAYOUT_GFX950, s1, None, 128, 8.0, up)
        act = torch.nn.functional.silu(up[:, :inter].float()) * up[:, inter:].float()
        g.wq_gemm_w4a16_experts(act.bfloat16(), None, topk, offsets, w2, g.LAYOUT_GFX950, s2, None, 128, 8.0, down)
        g.wq_combine_rows(down, place, router, out)
    out = torch.empty((t, h), dtype=torch.bfloat16, device="cuda")
    layer(out)
    # the oracle on the same packed weights, each bf16 step rounded as the layer rounds it
    f = lambda v: v.double().cpu().numpy()
    bf = lambda v: torch.from_numpy(v).bfloat16().double().numpy()
    off, od, pl = routing.sort_rows(ids.cpu().numpy(), e)
    u = bf(routing.gemm_experts(f(x), od, topk, off, w1.cpu().numpy(), f(s1), None, 8.0, 128, np.zeros(up.shape)))
    gate = u[:, :inter]
    act = bf(gate / (1 + np.exp(-gate)) * u[:, inter:])
    dn = bf(routing.gemm_experts(act, None, topk, off, w2.cpu().numpy(), f(s2), None, 8.0, 128, np.zeros(down.shape)))
    ref = routing.combine_rows(dn, pl, f(router))
    # four bf16 roundings on the way and up to two of weights, each at most 2^-8
    # of its value and of either sign: 1e-2 of the row's norm holds their root sum
    err = np.linalg.norm(f(out) - ref, axis=1) / np.linalg.norm(ref, axis=1)
    assert err.max() <= 1e-2
    replay_matches_eager(layer, out, torch.empty_like(out))


@pytest.mark.parametrize("t", [4, 200])
def test_adapters_beside_an_int4_projection(t):
    say("projection with adapters", t)
    k, n, adapters, rank = 512, 640, 5, 16
    gen = torch.Generator().manual_seed(t)
    w, s = weights(1, n, k, gen)
    c, ids = case(t, k, n, adapters, rank, seed=3)
    d = {x: v.cuda() for x, v in c.items()}
    out = torch.empty((t, n), dtype=torch.bfloat16, device="cuda")
    if t <= 32:
        g.wq_gemv_w4(w[0], g.LAYOUT_GFX950, s[0], None, 8.0, k, 128, d["x"], out)
    else:
        g.wq_gemm_w4a16(d["x"], w[0], g.LAYOUT_GFX950, s[0], 128, 8.0, out)
    offsets, order, place = (torch.empty(m, dtype=torch.int32, device="cuda") for m in (adapters + 1, t, t))
    g.wq_sort_rows(torch.from_numpy(ids).int().cuda(), adapters, offsets, order, place)
    g.wq_lora(d["x"], order, offsets, d["a"], d["b"], d["scales"], out, out)
    f = lambda v: v.double().cpu().numpy()
    codes = int4.gemm_w4a16_rows(f(d["x"]), w[0].cpu().numpy(), 1, f(s[0]), 8.0, 128)
    base = torch.from_numpy(codes).bfloat16().double().numpy()
    ref = routing.lora(f(d["x"]), ids, f(d["a"]), f(d["b"]), f(d["scales"]), base)
    # two roundings to bf16 (base and sum) of values below base's and the sum's size
    err = np.linalg.norm(f(out) - ref, axis=1) / np.linalg.norm(np.abs(ref) + np.abs(base), axis=1)
    assert err.max() <= 1e-2
