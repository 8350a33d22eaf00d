"""Pins of the routed-rows oracle: hand-worked cases, brute force and
invariants (the definitions are not on the pages)."""
import numpy as np
import pytest

from oracle import int4, routing


def test_sort_hand_worked():
    # slots 0..7 of four tokens; bin 1 stays empty, -1 and 3 are dropped
    ids = np.array([[2, 0], [0, -1], [2, 2], [3, 0]])
    offsets, order, place = routing.sort_rows(ids, 3)
    assert offsets.tolist() == [0, 3, 3, 6]
    assert order.tolist() == [1, 2, 7, 0, 4, 5, 3, 6]
    assert place.tolist() == [[3, 0], [1, -1], [4, 5], [-1, 2]]


@pytest.mark.parametrize("t,topk,bins", [(0, 2, 3), (1, 1, 1), (5, 8, 2), (200, 3, 17)])
def test_sort_invariants(t, topk, bins):
    rng = np.random.default_rng(t + topk)
    ids = rng.integers(-2, bins + 2, size=(t, topk))
    offsets, order, place = routing.sort_rows(ids, bins)
    flat = ids.reshape(-1)
    assert sorted(order.tolist()) == list(range(t * topk))
    assert offsets[0] == 0 and offsets[-1] == np.count_nonzero((flat >= 0) & (flat < bins))
    for b in range(bins):
        mine = order[offsets[b]:offsets[b + 1]]
        assert np.array_equal(mine, np.flatnonzero(flat == b))
        assert np.array_equal(place.reshape(-1)[mine], np.arange(offsets[b], offsets[b + 1]))
    assert np.all(place.reshape(-1)[order[offsets[-1]:]] == -1)


def test_moves_hand_worked():
    x = np.array([[1.0, 2.0], [3.0, 4.0]])
    place = np.array([[1, -1], [0, 2]])
    out = routing.dispatch_rows(x, place, np.full((4, 2), 9.0))
    assert out.tolist() == [[3, 4], [1, 2], [3, 4], [9, 9]]
    back = routing.combine_rows(out, place, np.array([[2.0, 5.0], [0.5, -1.0]]))
    assert back.tolist() == [[2, 4], [-1.5, -2]]
    assert routing.combine_rows(out, place, None).tolist() == [[1, 2], [6, 8]]
    d_rows, d_w = routing.combine_rows_grad(np.array([[1.0, 1.0], [1.0, 0.0]]), out, place,
                                            np.array([[2.0, 5.0], [0.5, -1.0]]), np.full((4, 2), 7.0))
    assert d_rows.tolist() == [[0.5, 0], [2, 2], [-1, 0], [7, 7]]
    assert d_w.tolist() == [[3, 0], [3, 3]]


def test_gradients_by_differences():
    # combine is linear in the rows and in the weights: a central difference of
    # <d_out, combine> is its gradient up to rounding
    rng = np.random.default_rng(0)
    t, topk, h = 4, 3, 5
    _, _, place = routing.sort_rows(rng.integers(-1, 4, size=(t, topk)), 4)
    rows, w, d = rng.normal(size=(t * topk, h)), rng.normal(size=(t, topk)), rng.normal(size=(t, h))
    d_rows, d_w = routing.combine_rows_grad(d, rows, place, w, np.zeros((t * topk, h)))

    def value(rows, w):
        return float(np.sum(d * routing.combine_rows(rows, place, w)))
    eps = 1e-3
    for i in range(t * topk):
        for k in range(h):
            step = np.zeros_like(rows)
            step[i, k] = eps
            assert abs((value(rows + step, w) - value(rows - step, w)) / (2 * eps) - d_rows[i, k]) < 1e-9
    for i in range(t):
        for j in range(topk):
            step = np.zeros_like(w)
            step[i, j] = eps
            assert abs((value(rows, w + step) - value(rows, w - step)) / (2 * eps) - d_w[i, j]) < 1e-9
    # dispatch's gradient is the unweighted combine: <r, dispatch(x)> = <combine(r), x>
    x = rng.normal(size=(t, h))
    moved = routing.dispatch_rows(x, place, np.zeros((t * topk, h)))
    assert abs(np.sum(moved * rows) - np.sum(x * routing.combine_rows(rows, place, None))) < 1e-9


@pytest.mark.parametrize("topk,gather,zeros", [(1, True, False), (2, True, True), (3, False, False)])
def test_experts_brute_force(topk, gather, zeros):
    rng = np.random.default_rng(topk)
    t, e, n, k, group = 5, 4, 3, 128, 64
    offsets, order, _ = routing.sort_rows(rng.integers(-1, e, size=(t, topk)), e)
    codes = rng.integers(0, 16, size=(e, n, k)).astype(np.uint8)
    packed = np.stack([int4.pack(c, int4.LAYOUT_GFX950) for c in codes])
    scales = rng.uniform(0.5, 2, size=(e, n, k // group))
    z = rng.uniform(6, 9, size=scales.shape) if zeros else None
    a = rng.normal(size=(t if gather else t * topk, k))
    got = routing.gemm_experts(a, order if gather else None, topk, offsets, packed, scales, z, 8.0, group,
                               np.full((t * topk, n), 4.0))
    for i in range(t * topk):
        if i >= offsets[e]:
            assert np.all(got[i] == 4.0)
            continue
        b = [x for x in range(e) if offsets[x] <= i < offsets[x + 1]][0]
        src = order[i] // topk if gather else i
        for j in range(n):
            want = sum(a[src, x] * (int(codes[b, j, x]) - (z[b, j, x // group] if zeros else 8.0)) *
                       scales[b, j, x // group] for x in range(k))
            assert abs(got[i, j] - want) < 1e-9


def test_lora_hand_worked():
    x = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    a = np.array([[[1.0, 0.0]], [[0.0, 1.0]]])          # rank 1: picks x[0], x[1]
    b = np.array([[[10.0], [20.0]], [[1.0], [-1.0]]])
    base = np.array([[0.5, 0.5], [0.0, 0.0], [7.0, 8.0]])
    got = routing.lora(x, np.array([1, 0, -1]), a, b, np.array([0.5, 3.0]), base)
    assert got.tolist() == [[6.5, -5.5], [15.0, 30.0], [7.0, 8.0]]
