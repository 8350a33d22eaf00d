"""Measured cases of the routed-rows operators: rows sorted by expert and moved
there and back (with gradients), the experts' int4 products, and low-rank
adapters beside a shared projection.

``run`` computes a case either in plain torch operations (``own`` false) or by
the library's entry points (``own`` true); ``exact`` gives the same outputs
from the definitions in float64.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# nibble p of a packed 32-bit word holds element NIBBLE[p] of its eight codes
NIBBLE = (0, 2, 4, 6, 1, 3, 5, 7)


# --------------------------------------------------------------------- cases

def listed():
    return [
        # one decoded token's choice of experts: pure latency
        dict(name="sort one token", kind="sort", t=1, topk=8, bins=128, drop=0.0),
        # the router's choices of a long prompt, some slots over capacity
        dict(name="sort long prompt", kind="sort", t=16384, topk=8, bins=256, drop=0.03),
        # a decode step of 32 sequences: rows to their experts and back
        dict(name="move decode step", kind="move", t=32, topk=8, h=4096, bins=64, dtype="bf16", drop=0.0),
        # a prompt's rows to their experts and back
        dict(name="move prompt", kind="move", t=4096, topk=8, h=5120, bins=64, dtype="bf16", drop=0.0),
        # odd row count and length: rows that no 16-byte access divides
        dict(name="move odd rows", kind="move", t=3001, topk=3, h=1411, bins=17, dtype="f16", drop=0.05),
        # a training step's backward pass of the same movement
        dict(name="move back prompt", kind="move_grad", t=4096, topk=8, h=4096, bins=64, dtype="bf16", drop=0.0),
        # float32 rows, two experts each, some dropped
        dict(name="move back f32", kind="move_grad", t=777, topk=2, h=1000, bins=8, dtype="f32", drop=0.1),
        # one token through its eight of 64 experts (gate and up rows together)
        dict(name="experts one token", kind="experts", t=1, topk=8, bins=64, k=4096, n=2816, group=128,
             gather=True, zeros=False, drop=0.0),
        # a small batch's second product: sorted rows as they lie, stored zeros, ragged n
        dict(name="experts small batch", kind="experts", t=48, topk=4, bins=32, k=2560, n=5112, group=128,
             gather=False, zeros=True, drop=0.02),
        # a prompt through all experts
        dict(name="experts prompt", kind="experts", t=4096, topk=8, bins=64, k=4096, n=2816, group=128,
             gather=True, zeros=False, drop=0.0),
        # 32 requests, nearly each with an adapter of its own, one token each
        dict(name="adapters decode", kind="lora", t=32, adapters=64, runs=32, rank=16, k=5120, n=17280,
             dtype="bf16", drop=0.1),
        # packed prompts of ten requests, two of them without an adapter
        dict(name="adapters prompts", kind="lora", t=4096, adapters=8, runs=10, rank=64, k=5120, n=5120,
             dtype="bf16", drop=0.2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["sort", "move", "move_grad", "experts", "experts", "lora", "lora"])
    drop = rng.choice([0.0, 0.0, 0.02, 0.1])
    if kind == "sort":
        topk = rng.randint(1, 8)
        return dict(kind=kind, t=_log(rng, 1, 16384), topk=topk, bins=_log(rng, max(topk, 2), 256), drop=drop)
    if kind in ("move", "move_grad"):
        topk = rng.randint(1, 8)
        h = _log(rng, 64, 5120)
        if rng.random() < 0.7:
            h = (h + 7) // 8 * 8
        return dict(kind=kind, t=_log(rng, 1, 3500), topk=topk, h=h, bins=_log(rng, max(topk, 2), 128),
                    dtype=rng.choice(["bf16", "bf16", "f16", "f32"]) if h <= 2560 else rng.choice(["bf16", "f16"]),
                    drop=drop)
    if kind == "experts":
        topk = rng.randint(1, 8)
        group = rng.choice([64, 128, 128, 256, 0])  # 0: one scale a column
        step = group or 64
        k = max(1, round(_log(rng, 256, 4096) / step)) * step
        return dict(kind=kind, t=_log(rng, 1, 4096), topk=topk, bins=_log(rng, max(topk, 4), 64), k=k,
                    n=_log(rng, 100, 2816), group=group or k, gather=rng.random() < 0.5,
                    zeros=rng.random() < 0.3, drop=drop)
    return dict(kind=kind, t=_log(rng, 1, 4096), adapters=_log(rng, 1, 64), runs=_log(rng, 1, 64),
                rank=rng.choice([8, 16, 16, 32, 64, 128]), k=32 * _log(rng, 8, 160), n=_log(rng, 100, 5120),
                dtype=rng.choice(["bf16", "bf16", "f32"]), drop=drop)


# -------------------------------------------------------------------- inputs

def _choices(c, gen):
    """Router choices int32 [t][topk]: distinct experts of a skewed router, some slots dropped (-1)."""
    lean = 0.7 * torch.randn(c["bins"], device=DEV, generator=gen)
    noise = -torch.log(-torch.log(torch.rand(c["t"], c["bins"], device=DEV, generator=gen).clamp(1e-6, 1 - 1e-6)))
    ids = torch.topk(lean + noise, c["topk"], dim=1).indices.to(torch.int32)
    return torch.where(torch.rand(ids.shape, device=DEV, generator=gen) < c["drop"], -1, ids)


def _plan(ids, bins):
    """offsets, order and place of the rows sorted by bin, as wq_sort_rows defines them."""
    flat = ids.reshape(-1)
    key = torch.where(flat < 0, bins, flat).long()
    key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(bins + 1, device=DEV)).to(torch.int32)
    place = torch.empty_like(order)
    place[order] = torch.arange(order.numel(), device=DEV)
    place = torch.where(flat < 0, -1, place)
    return offsets, order.to(torch.int32), place.to(torch.int32).reshape(ids.shape)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device=DEV).manual_seed(seed)
    kind = c["kind"]

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return (scale * torch.randn(*shape, device=DEV, generator=gen)).to(dtype)

    def zeros(*shape, dtype):
        return torch.zeros(*shape, dtype=dtype, device=DEV)

    s = {"case": dict(c)}
    if kind == "sort":
        s["ids"] = _choices(c, gen)
        slots = c["t"] * c["topk"]
        s["offsets"] = zeros(c["bins"] + 1, dtype=torch.int32)
        s["order"], s["place"] = zeros(slots, dtype=torch.int32), zeros(c["t"], c["topk"], dtype=torch.int32)
        return s
    if kind in ("move", "move_grad"):
        dt, slots = DTYPES[c["dtype"]], c["t"] * c["topk"]
        ids = _choices(c, gen)
        s["offsets"], s["order"], s["place"] = _plan(ids, c["bins"])
        s["weights"] = torch.softmax(randn(c["t"], c["topk"]), dim=1)
        s["rows"] = randn(slots, c["h"], dtype=dt)
        s["token_out"] = zeros(c["t"], c["h"], dtype=dt)
        s["row_out"] = zeros(slots, c["h"], dtype=dt)
        if kind == "move":
            s["x"] = randn(c["t"], c["h"], dtype=dt)
        else:
            s["d_out"] = randn(c["t"], c["h"], dtype=dt)
            s["d_sorted"] = randn(slots, c["h"], dtype=dt)
            s["d_weights"] = zeros(c["t"], c["topk"], dtype=torch.float32)
        return s
    if kind == "experts":
        slots, e, n, k, groups = c["t"] * c["topk"], c["bins"], c["n"], c["k"], c["k"] // c["group"]
        ids = _choices(c, gen)
        s["offsets"], s["order"], _ = _plan(ids, e)
        s["a"] = randn(c["t"] if c["gather"] else slots, k, dtype=torch.bfloat16)
        s["b"] = torch.randint(0, 256, (e, n, k // 2), dtype=torch.uint8, device=DEV, generator=gen)
        s["scales"] = (0.002 + 0.018 * torch.rand(e, n, groups, device=DEV, generator=gen)).bfloat16()
        s["zeros"] = None
        if c["zeros"]:
            s["zeros"] = torch.randint(6, 10, (e, n, groups), device=DEV, generator=gen).bfloat16()
        s["out"] = zeros(slots, n, dtype=torch.bfloat16)
        return s
    # lora: `runs` packed requests of random lengths, each with one adapter or none
    t, runs = c["t"], min(c["runs"], c["t"])
    cuts = torch.randperm(t - 1, device=DEV, generator=gen)[:runs - 1] + 1 if t > 1 else torch.empty(0, device=DEV)
    request = torch.zeros(t, dtype=torch.long, device=DEV)
    request[cuts.long()] = 1
    request = torch.cumsum(request, 0)
    of_request = torch.randint(0, c["adapters"], (runs,), device=DEV, generator=gen)
    of_request = torch.where(torch.rand(runs, device=DEV, generator=gen) < c["drop"], -1, of_request)
    s["offsets"], s["order"], _ = _plan(of_request[request].to(torch.int32).reshape(t, 1), c["adapters"])
    dt = DTYPES[c["dtype"]]
    s["x"] = randn(t, c["k"], dtype=torch.bfloat16)
    s["a"] = randn(c["adapters"], c["rank"], c["k"], dtype=torch.bfloat16, scale=c["k"] ** -0.5)
    s["b"] = randn(c["adapters"], c["n"], c["rank"], dtype=torch.bfloat16, scale=0.2)
    s["scales"] = 0.5 + 1.5 * torch.rand(c["adapters"], device=DEV, generator=gen)
    s["base"] = randn(t, c["n"], dtype=dt)
    s["out"] = zeros(t, c["n"], dtype=dt)
    return s


# ----------------------------------------------------------------- operators

def run(state):
    return (_run_own if own else _run_plain)(state, state["case"])


def _run_own(s, c):
    import gemm_wq_quantize_amd as wq
    kind = c["kind"]
    if kind == "sort":
        wq.wq_sort_rows(s["ids"], c["bins"], s["offsets"], s["order"], s["place"])
        return s["offsets"], s["order"], s["place"]
    if kind == "move":
        wq.wq_dispatch_rows(s["x"], s["place"], s["row_out"])
        wq.wq_combine_rows(s["rows"], s["place"], s["weights"], s["token_out"])
        return s["row_out"], s["token_out"]
    if kind == "move_grad":
        wq.wq_combine_rows_grad(s["d_out"], s["rows"], s["place"], s["weights"], s["row_out"], s["d_weights"])
        wq.wq_combine_rows(s["d_sorted"], s["place"], None, s["token_out"])
        return s["row_out"], s["d_weights"], s["token_out"]
    if kind == "experts":
        wq.wq_gemm_w4a16_experts(s["a"], s["order"] if c["gather"] else None, c["topk"], s["offsets"], s["b"],
                                 wq.LAYOUT_GFX950, s["scales"], s["zeros"], c["group"], 8.0, s["out"])
        return s["out"]
    wq.wq_lora(s["x"], s["order"], s["offsets"], s["a"], s["b"], s["scales"], s["base"], s["out"])
    return s["out"]


def _picked(rows, place):
    """rows[place] in float32 as [t][topk][h], zero where place is -1."""
    got = rows.float()[place.clamp(min=0).long()]
    return torch.where((place >= 0)[..., None], got, 0.0)


def _placed(values, place, like):
    """values [t][topk][h] at rows `place` of a tensor like `like`; other rows zero."""
    out = torch.zeros((like.shape[0] + 1, like.shape[1]), dtype=like.dtype, device=DEV)
    out[torch.where(place < 0, like.shape[0], place).reshape(-1).long()] = values.reshape(-1, like.shape[1]).to(like.dtype)
    return out[:-1]


def _weights(b, scales, zeros, zero_const):
    """Packed codes [..][n][k/2] -> float32 (q - z) * s, [..][n][k]."""
    words = b.view(torch.int32)
    back = [NIBBLE.index(i) for i in range(8)]
    shifts = torch.tensor([4 * p for p in back], dtype=torch.int32, device=DEV)
    q = ((words[..., None] >> shifts) & 15).flatten(-2)
    q = q.unflatten(-1, (scales.shape[-1], -1)).float()
    z = zero_const if zeros is None else zeros.float()[..., None]
    return ((q - z) * scales.float()[..., None]).flatten(-2)


def _bin_of_rows(offsets, count):
    """Bin of each sorted row; the number of bins for rows behind the last one."""
    return torch.searchsorted(offsets[1:].contiguous().long(), torch.arange(count, device=DEV), right=True)


def _by_bin(rows, offsets, weights):
    """rows [r][k] times their bin's weights [bins][n][k] transposed: [r][n], zero behind the last bin."""
    bins, count = weights.shape[0], rows.shape[0]
    which = _bin_of_rows(offsets, count)
    most = int((offsets[1:] - offsets[:-1]).max())
    at = torch.arange(count, device=DEV) - torch.cat([offsets, offsets[-1:]]).long()[which]
    at = torch.where(which == bins, 0, at)
    padded = torch.zeros((bins + 1, max(most, 1), rows.shape[1]), device=DEV)
    padded[which, at] = torch.where((which < bins)[:, None], rows.float(), 0.0)
    out = torch.bmm(padded[:bins], weights.transpose(1, 2))
    return torch.where((which < bins)[:, None], out[which.clamp(max=bins - 1), at], 0.0)


def _run_plain(s, c):
    kind = c["kind"]
    if kind == "sort":
        return _plan(s["ids"], c["bins"])
    if kind == "move":
        to = _placed(s["x"][:, None, :].expand(-1, c["topk"], -1), s["place"], s["row_out"])
        back = (s["weights"][..., None] * _picked(s["rows"], s["place"])).sum(1)
        return to, back.to(s["rows"].dtype)
    if kind == "move_grad":
        d = s["d_out"].float()[:, None, :]
        d_rows = _placed(s["weights"][..., None] * d, s["place"], s["row_out"])
        d_weights = (d * _picked(s["rows"], s["place"])).sum(-1)
        return d_rows, d_weights, _picked(s["d_sorted"], s["place"]).sum(1).to(s["rows"].dtype)
    if kind == "experts":
        slots = c["t"] * c["topk"]
        rows = s["a"][s["order"].long() // c["topk"]] if c["gather"] else s["a"]
        if slots < c["bins"]:  # few rows: only the weights that they meet
            which = _bin_of_rows(s["offsets"], slots)
            one = which.clamp(max=c["bins"] - 1)
            w = _weights(s["b"][one], s["scales"][one], None if s["zeros"] is None else s["zeros"][one], 8.0)
            out = torch.bmm(w, rows.float()[..., None])[..., 0]
            out = torch.where((which < c["bins"])[:, None], out, 0.0)
        else:
            out = _by_bin(rows, s["offsets"], _weights(s["b"], s["scales"], s["zeros"], 8.0))
        return out.to(torch.bfloat16)
    order = s["order"].long()
    rows = s["x"][order].float()
    which = _bin_of_rows(s["offsets"], c["t"])
    scale = torch.cat([s["scales"], torch.zeros(1, device=DEV)])[which]
    if c["t"] < c["adapters"]:
        one = which.clamp(max=c["adapters"] - 1)
        low = torch.bmm(s["a"][one].float(), rows[..., None])
        add = torch.bmm(s["b"][one].float(), low)[..., 0]
        add = torch.where((which < c["adapters"])[:, None], add, 0.0)
    else:
        low = _by_bin(rows, s["offsets"], s["a"].float())
        add = _by_bin(low, s["offsets"], s["b"].float())
    out = s["base"].float()
    out[order] += scale[:, None] * add
    return out.to(s["base"].dtype)


# --------------------------------------------------------------------- work

def _met(c, bins, topk):
    """Bins that t tokens with topk choices each are expected to meet."""
    return bins * (1.0 - (1.0 - topk / bins) ** c["t"])


def work(case):
    c = case
    t, kind = c["t"], c["kind"]
    if kind == "sort":
        slots = t * c["topk"]
        return {"bytes": 4 * (3 * slots + c["bins"] + 1), "flops": slots}
    if kind in ("move", "move_grad"):
        es, rows = (4 if c["dtype"] == "f32" else 2), t * c["topk"] * (1 - c["drop"])
        small = 8 * t * c["topk"]
        if kind == "move":
            return {"bytes": es * c["h"] * (2 * t + 2 * rows) + small, "flops": 2 * rows * c["h"]}
        return {"bytes": es * c["h"] * (2 * t + 3 * rows) + small + 4 * t * c["topk"], "flops": 4 * rows * c["h"]}
    if kind == "experts":
        rows = t * c["topk"] * (1 - c["drop"])
        per = c["n"] * (c["k"] / 2 + (4 if c["zeros"] else 2) * (c["k"] // c["group"]))
        a = 2 * c["k"] * (t if c["gather"] else rows)
        return {"bytes": _met(c, c["bins"], min(c["topk"], c["bins"])) * per + a + 2 * rows * c["n"],
                "flops": 2 * rows * c["n"] * c["k"]}
    es, rows, runs = (4 if c["dtype"] == "f32" else 2), t * (1 - c["drop"]), min(c["runs"], t)
    met = c["adapters"] * (1.0 - (1.0 - 1.0 / c["adapters"]) ** (runs * (1 - c["drop"])))
    return {"bytes": 2 * met * c["rank"] * (c["k"] + c["n"]) + 2 * rows * c["k"] + 2 * es * t * c["n"],
            "flops": 2 * rows * c["rank"] * (c["k"] + c["n"])}


# -------------------------------------------------------------------- exact

def exact(case, seed):
    """The definitions in float64; None for the sort, whose outputs are whole numbers."""
    c = case
    kind = c["kind"]
    if kind == "sort":
        return None
    s = prepare(c, seed)
    if kind in ("move", "move_grad"):
        t, topk, h = c["t"], c["topk"], c["h"]
        place = s["place"].long()
        rows64, w64 = s["rows"].double(), s["weights"].double()
        moved = torch.zeros(t * topk, h, dtype=torch.float64, device=DEV)
        token = torch.zeros(t, h, dtype=torch.float64, device=DEV)
        dots = torch.zeros(t, topk, dtype=torch.float64, device=DEV)
        source = s["x"].double() if kind == "move" else s["d_out"].double()
        back = rows64 if kind == "move" else s["d_sorted"].double()
        for j in range(topk):
            live = (place[:, j] >= 0).nonzero()[:, 0]
            at = place[live, j]
            wj = w64[live, j][:, None]
            moved[at] = source[live] if kind == "move" else wj * source[live]
            token[live] += (wj if kind == "move" else 1.0) * back[at]
            if kind == "move_grad":
                dots[live, j] = (source[live] * rows64[at]).sum(1)
        return (moved, token) if kind == "move" else (moved, dots, token)
    offsets = s["offsets"].tolist()
    if kind == "experts":
        out = torch.zeros(c["t"] * c["topk"], c["n"], dtype=torch.float64, device=DEV)
        for e in range(c["bins"]):
            lo, hi = offsets[e], offsets[e + 1]
            if lo == hi:
                continue
            codes = torch.empty(c["n"], c["k"], dtype=torch.float64, device=DEV)
            b = s["b"][e]
            for p in range(8):  # nibble p: byte p // 2 of each word, low nibble first
                byte = b[:, p // 2::4]
                codes[:, NIBBLE[p]::8] = ((byte >> 4) if p % 2 else (byte & 15)).double()
            g = c["group"]
            scale = s["scales"][e].double().repeat_interleave(g, dim=1)
            zero = s["zeros"][e].double().repeat_interleave(g, dim=1) if c["zeros"] else 8.0
            rows = s["a"][s["order"][lo:hi].long() // c["topk"]] if c["gather"] else s["a"][lo:hi]
            out[lo:hi] = rows.double() @ ((codes - zero) * scale).T
        return out
    out = s["base"].double().clone()
    for e in range(c["adapters"]):
        at = s["order"][offsets[e]:offsets[e + 1]].long()
        if at.numel():
            low = s["x"][at].double() @ s["a"][e].double().T
            out[at] += s["scales"][e].double() * (low @ s["b"][e].double().T)
    return out
