"""Oracle for rows that go to different weights: the sort by bin, the moves
there and back with their gradients, the experts' int4 products and the
low-rank adapters.

TEST INFRASTRUCTURE (see ``oracle/__init__``): plain loops over the
definitions in float64, written apart from the HIP path.  The pages do not
define these operators (parity unpinned); the definitions are this library's,
pinned by hand-worked cases and invariants in ``tests/test_oracle_routing.py``.
"""
from __future__ import annotations

import numpy as np

from . import int4


def sort_rows(ids: np.ndarray, bins: int):
    """ids [t][topk] -> (offsets [bins + 1], order [slots], place [t][topk]):
    slot = i * topk + j; slots of one bin ascending, bins in order, dropped
    slots (id outside [0, bins)) behind them in ascending order with place -1."""
    flat = np.asarray(ids).reshape(-1)
    lists = [[] for _ in range(bins + 1)]
    for slot, b in enumerate(flat.tolist()):
        lists[b if 0 <= b < bins else bins].append(slot)
    offsets = np.zeros(bins + 1, dtype=np.int32)
    for b in range(bins):
        offsets[b + 1] = offsets[b] + len(lists[b])
    order = np.array([s for one in lists for s in one], dtype=np.int32).reshape(-1)
    place = np.full(flat.size, -1, dtype=np.int32)
    for i in range(int(offsets[bins])):
        place[order[i]] = i
    return offsets, order, place.reshape(np.asarray(ids).shape)


def dispatch_rows(x: np.ndarray, place: np.ndarray, out: np.ndarray) -> np.ndarray:
    """A copy of ``out`` with out[place[i][j]] = x[i] for every kept slot."""
    out = np.array(out)
    for i, row in enumerate(place):
        for p in row:
            if p >= 0:
                out[p] = x[i]
    return out


def combine_rows(rows: np.ndarray, place: np.ndarray, weights) -> np.ndarray:
    """out[i] = sum_j weights[i][j] * rows[place[i][j]] (weights None: 1)."""
    t, topk = place.shape
    out = np.zeros((t, rows.shape[1]), dtype=np.float64)
    for i in range(t):
        for j in range(topk):
            if place[i, j] >= 0:
                w = 1.0 if weights is None else float(weights[i, j])
                out[i] += w * rows[place[i, j]].astype(np.float64)
    return out


def combine_rows_grad(d_out, rows, place, weights, d_rows):
    """(d_rows, d_weights): a copy of ``d_rows`` with d_rows[place[i][j]] =
    weights[i][j] * d_out[i], and d_weights[i][j] = <d_out[i], rows[place[i][j]]>
    (0 for a dropped slot)."""
    d_rows = np.array(d_rows, dtype=np.float64)
    d_w = np.zeros(place.shape, dtype=np.float64)
    for i, row in enumerate(place):
        d = d_out[i].astype(np.float64)
        for j, p in enumerate(row):
            if p >= 0:
                d_rows[p] = float(weights[i, j]) * d
                d_w[i, j] = float(np.dot(d, rows[p].astype(np.float64)))
    return d_rows, d_w


def gemm_experts(a, order, topk, offsets, packed, scales, zeros, zero_const, group, out, bf16_weights=False):
    """A copy of ``out`` [slots][n] whose rows offsets[e] .. offsets[e + 1] - 1
    hold a[src(i)] times expert e's weights (packed [e][n][k/2] in the gfx950
    layout); src(i) = order[i] // topk, or i without ``order``.
    ``bf16_weights``: each weight rounded to bf16 first."""
    out = np.array(out, dtype=np.float64)
    for e in range(packed.shape[0]):
        lo, hi = int(offsets[e]), int(offsets[e + 1])
        if lo == hi:
            continue
        src = np.arange(lo, hi) if order is None else np.asarray(order[lo:hi]) // topk
        z = None if zeros is None else zeros[e]
        rows = int4.gemm_w4a16_rows_bf16w if bf16_weights else int4.gemm_w4a16_rows
        out[lo:hi] = rows(a[src], packed[e], int4.LAYOUT_GFX950, scales[e], zero_const, group, zeros=z)
    return out


def lora(x, ids, a, b, scales, base):
    """out[i] = base[i] + scales[l] * b[l] (a[l] x[i]) with l = ids[i]; base[i]
    alone where ids[i] names no adapter."""
    out = np.array(base, dtype=np.float64)
    flat = np.asarray(ids).reshape(-1)
    for l in range(a.shape[0]):
        rows = np.flatnonzero(flat == l)
        low = x[rows].astype(np.float64) @ a[l].astype(np.float64).T
        out[rows] += float(scales[l]) * (low @ b[l].astype(np.float64).T)
    return out
