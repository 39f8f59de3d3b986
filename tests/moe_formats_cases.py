"""Inputs and float64 references of the router and of the 8-bit and 16-bit expert-grouped products.

The references share no code with the library: expert by expert, row by row of the definition, in float64 on the CPU.
"""
import numpy as np
import torch

import moe_token_int8_amd as L

DEV = "cuda"


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def w8_inputs(seed, counts, K, N, src_rows=None, k=1, extra_rows=0):
    """Codes, scales, gather and offsets for experts with the given row counts; `extra_rows` rows belong to nobody."""
    g = np.random.default_rng(seed)
    rows = int(sum(counts)) + extra_rows
    src = rows if src_rows is None else src_rows
    gather = None if src_rows is None else g.integers(0, src_rows * k, size=rows).astype(np.int32)
    return dict(Xq=g.integers(-127, 128, size=(src, K), dtype=np.int8),
                sx=(g.random(src, dtype=np.float32) + 0.5) * np.float32(0.03),
                codes=g.integers(-127, 128, size=(len(counts), K, N), dtype=np.int8),
                sw=((g.random((len(counts), N), dtype=np.float32) + 0.5) * np.float32(1e-3)).astype(np.float32),
                gather=gather, k=k, offsets=offsets_of(counts), rows=rows)


def w8_reference(c):
    """float64 [rows, N]; rows of nobody are NaN (callers compare owned rows only)."""
    out = np.full((c["rows"], c["sw"].shape[1]), np.nan)
    for e in range(len(c["sw"])):
        a, b = c["offsets"][e], c["offsets"][e + 1]
        r = np.arange(a, b)
        src = r if c["gather"] is None else c["gather"][r] // c["k"]
        ok = (src >= 0) & (src < len(c["Xq"])) & (True if c["gather"] is None else c["gather"][r] >= 0)
        s = np.where(ok, src, 0)
        y = (c["Xq"][s].astype(np.float64) @ c["codes"][e].astype(np.float64)) * c["sx"][s].astype(np.float64)[:, None]
        out[a:b] = np.where(ok[:, None], y * c["sw"][e].astype(np.float64)[None, :], 0.0)
    return out


def w8_device(c):
    """Packs the experts on the host; returns (desc, DeviceWeights, device tensors of the call)."""
    E, K, N = c["codes"].shape
    d = L.desc(K, N, K, False, bits=8)
    blobs = [L.w4a8_pack_codes(d, c["codes"][e], c["sw"][e][None, :], None) for e in range(E)]
    t = {n: None if c[n] is None else torch.from_numpy(c[n]).to(DEV) for n in ("Xq", "sx", "gather", "offsets")}
    return d, L.to_device(d, blobs, DEV), t


def w16_inputs(seed, dtype, counts, K, N, src_rows=None, k=1, extra_rows=0, std=0.05):
    """CPU tensors X [src, K], W [E, N, K] of `dtype`."""
    g = torch.Generator().manual_seed(seed)
    rows = int(sum(counts)) + extra_rows
    src = rows if src_rows is None else src_rows
    gather = None if src_rows is None else torch.randint(0, src_rows * k, (rows,), generator=g, dtype=torch.int32)
    return dict(X=torch.randn(src, K, generator=g).to(dtype), W=(torch.randn(len(counts), N, K, generator=g) * std).to(dtype),
                gather=gather, k=k, offsets=torch.from_numpy(offsets_of(counts)), rows=rows)


def w16_reference(c):
    """(sums, sums of the absolute products) in float64 [rows, N]; rows of nobody are NaN."""
    N = c["W"].shape[1]
    y = torch.full((c["rows"], N), float("nan"), dtype=torch.float64)
    mag = torch.zeros(c["rows"], N, dtype=torch.float64)
    off = c["offsets"].tolist()
    for e in range(len(off) - 1):
        r = torch.arange(off[e], off[e + 1])
        if not len(r):
            continue
        src = r if c["gather"] is None else torch.div(c["gather"][r].long(), c["k"], rounding_mode="floor")
        ok = (src >= 0) & (src < len(c["X"]))
        x, w = c["X"][torch.where(ok, src, 0)].double(), c["W"][e].double()
        y[r] = torch.where(ok[:, None], x @ w.t(), 0.0)
        mag[r] = torch.where(ok[:, None], x.abs() @ w.abs().t(), 0.0)
    return y, mag


def half_step(dtype, y):
    """Bound of one rounding of y to `dtype`: half a step, and half the least subnormal of float16 near zero."""
    if dtype == torch.float32:
        return 0 * y.abs()
    return y.abs() * (torch.finfo(dtype).eps / 2) + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def w16_bound(dtype_out, K, y, mag):
    """|got - y|: a float32 sum of K exact products, whatever its order, is within K 2^-23 sum|x w| (each of at most K
    additions rounds or truncates by at most one unit, 2^-23, of a partial sum that sum|x w| bounds); then one rounding
    to the output type of a value that is at most that much larger."""
    e = K * 2.0 ** -23 * mag
    return e + half_step(dtype_out, y.abs() + e) + 1e-38


def silu_reference(c):
    """(h, bound of |got - h|) for W [E, 2I, K]: with g, u off by eg, eu, and |silu'| <= 1.1, silu(g) u is off by
    1.1 eg (|u| + eu) + |silu(g)| eu; the float32 evaluation (an exponential good to 4 units, one addition, one division,
    one product) adds 8 2^-23 |h|; then the output rounding."""
    y, mag = w16_reference(c)
    I = y.shape[1] // 2
    K = c["X"].shape[1]
    g, u = y[:, :I], y[:, I:]
    e = K * 2.0 ** -23 * mag
    sg = g * torch.sigmoid(g)
    h = sg * u
    b = 1.1 * e[:, :I] * (u.abs() + e[:, I:]) + sg.abs() * e[:, I:]
    b = b + 8 * 2.0 ** -23 * (h.abs() + b)
    return h, b + half_step(c["X"].dtype, h.abs() + b) + 1e-38


def assert_within(got, want, bound, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - bound
    i = int(torch.argmax(over))
    assert float(over.reshape(-1)[i]) <= 0, (what, float(got.reshape(-1)[i]), float(want.reshape(-1)[i]),
                                             float(bound.reshape(-1)[i]))


# ----------------------------------------------------------------------------------------------- router
def route_reference(x, bias, E, k, score, renorm, scale, groups, keep):
    """Float64 by the definition, token by token and choice by choice.  Returns (ids, weights)."""
    T = len(x)
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    size = E // groups
    for t in range(T):
        v = x[t].astype(np.float64)
        masked = np.isneginf(v)
        bad = np.isnan(v).any() or (score == "softmax" and np.isposinf(v).any())
        with np.errstate(all="ignore"):
            if score == "softmax":
                p = np.where(masked, 0.0, np.exp(v - (0.0 if masked.all() else v[~masked].max())))
                p = p / p.sum() if p.sum() > 0 else p
            else:
                p = np.where(masked, 0.0, 1 / (1 + np.exp(-v)))
            rank = np.where(masked, -np.inf, v if bias is None else p + bias.astype(np.float64))
        if bad or np.isnan(rank).any():
            ids[t], w[t] = np.arange(k), np.nan
            continue
        if groups > 1:
            by = -np.sort(-rank.reshape(groups, size), axis=1)
            best = by[:, 0].copy()
            if bias is not None and size > 1:
                best += np.where(np.isneginf(by[:, 1]), 0.0, by[:, 1])
            kept = np.argsort(-best, kind="stable")[:keep]
            rank = np.where(np.isin(np.arange(E) // size, kept), rank, -np.inf)
        order = np.argsort(-rank, kind="stable")[:k]
        there = ~np.isneginf(rank[order])
        ids[t] = np.where(there, order, -1)
        c = np.where(there, p[order], 0.0)
        if renorm:
            c = c / c.sum() if c.sum() > 0 else c * 0.0
        w[t] = c * scale
    return ids, w
