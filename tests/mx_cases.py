"""Inputs and float64 references of the microscaled (MX) calls and of the norm around a block.

The references share no code with the library: elements by a search over the formats' values, products expert by expert in
float64 on the CPU."""
import math

import numpy as np
import torch

import moe_token_int8_amd as L

DEV = "cuda"
FP4, FP8 = L.W4A8_MX_FP4, L.W4A8_MX_FP8
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)][:-1])


def up(x, unit):
    return -(-x // unit) * unit


def encode(x, fmt):
    """(codes [M, Kp] one to a byte, scale bytes [M, Kp / 32]) of rows x (numpy or torch, exact in float64), by the definition:
    elements and scales behind K are zero."""
    x = np.asarray(torch.as_tensor(x).double())
    M, K = x.shape
    Kp = up(K, 128)
    full = np.zeros((M, Kp))
    full[:, :K] = x
    blocks = full.reshape(M, Kp // 32, 32)
    with np.errstate(all="ignore"):
        amax = np.abs(blocks).max(2)
        bad = ~np.isfinite(blocks).all(2)
        e = np.frexp(np.where(bad, 1.0, amax))[1] - 1
        b = np.where(amax == 0, 0, np.maximum(e + 127 - (2 if fmt == FP4 else 8), 0))
        y = np.where(bad[..., None], 0.0, blocks) * np.exp2(127.0 - b)[..., None]
    grid = E2M1 if fmt == FP4 else E4M3
    mid = (grid[1:] + grid[:-1]) / 2
    a = np.minimum(np.abs(y), grid[-1])
    i = np.searchsorted(mid, a, side="left")                        # a tie goes down here: odd indices go up
    tie = (i < len(mid)) & (a == mid[np.minimum(i, len(mid) - 1)]) & (i % 2 == 1)
    code = np.where(tie, i + 1, i) | np.where(np.signbit(y), 8 if fmt == FP4 else 128, 0)
    code = np.where(bad[..., None], 0, code)
    return code.astype(np.uint8).reshape(M, Kp), np.where(bad, 255, b).astype(np.uint8)


def stored(code, fmt):
    return code[:, 0::2] | (code[:, 1::2] << 4) if fmt == FP4 else code


def unstored(q, fmt):
    if fmt == FP8:
        return q
    out = np.empty((q.shape[0], 2 * q.shape[1]), np.uint8)
    out[:, 0::2], out[:, 1::2] = q & 15, q >> 4
    return out


def values(code, s, fmt, K):
    """float64 [M, K] of codes one to a byte."""
    grid, half = (E2M1, 8) if fmt == FP4 else (np.append(E4M3, np.nan), 128)
    v = grid[code % half] * np.where(code >= half, -1.0, 1.0)
    with np.errstate(all="ignore"):
        scale = np.where(s == 255, np.nan, np.exp2(s.astype(np.float64) - 127))
    return (v.reshape(len(v), s.shape[1], 32) * scale[..., None]).reshape(len(v), 32 * s.shape[1])[:, :K]


def same_codes(got, want, fmt):
    """Codes that stand for the same values (a zero's sign counts too)."""
    return np.array_equal(unstored(got, fmt), want)


def random_codes(g, M, K, fmt, spread=3):
    """Stored codes and scales of M rows as any producer may leave them: all finite codes, scales around 1; zeros behind K."""
    Kp = up(K, 128)
    code = g.integers(0, 16 if fmt == FP4 else 256, size=(M, Kp), dtype=np.uint8)
    if fmt == FP8:
        code[(code & 127) == 127] ^= 1
    s = g.integers(127 - spread, 128 + spread, size=(M, Kp // 32), dtype=np.uint8)
    code[:, K:] = 0
    s[:, up(K, 32) // 32:] = 0
    return code, s


def pack(code, s, N, K):
    """Packed weights by the documented places."""
    K1, blob = up(K, 128) // 128, np.zeros(L.w4a8_mx_packed_size(K, N), np.uint8)
    n, k = np.arange(N)[:, None], np.arange(K1 * 128)[None, :]
    at = ((n // 16 * K1 + k // 128) * 64 + k % 128 // 32 * 16 + n % 16) * 16 + k % 32 // 2
    np.bitwise_or.at(blob, at.reshape(-1), (code << (4 * (k % 2)).astype(np.uint8)).reshape(-1))
    base = up(up(N, 16) * K1 * 64, 256)
    b = np.arange(K1 * 4)[None, :]
    blob[base + ((n // 64 * K1 + b // 4) * 64 + b % 4 * 16 + n % 16) * 4 + n % 64 // 16] = s
    return blob


def offsets_of(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def moe_inputs(seed, counts, K, N, fmt, src_rows=None, k=1, extra_rows=0, spread=3):
    g = np.random.default_rng(seed)
    rows = int(sum(counts)) + extra_rows
    src = rows if src_rows is None else src_rows
    x, sx = random_codes(g, src, K, fmt, spread)
    w = [random_codes(g, N, K, FP4, spread) for _ in counts]
    gather = None if src_rows is None else g.integers(0, src_rows * k, size=rows).astype(np.int32)
    return dict(x=x, sx=sx, w=w, gather=gather, k=k, offsets=offsets_of(counts), rows=rows, K=K, N=N, fmt=fmt)


def moe_reference(c):
    """(sums, sums of magnitudes) in float64 [rows, N]; rows of nobody are NaN, rows whose gather names nothing zeros."""
    y, mag = np.full((c["rows"], c["N"]), np.nan), np.zeros((c["rows"], c["N"]))
    x = values(c["x"], c["sx"], c["fmt"], c["K"])
    off = c["offsets"]
    for e in range(len(off) - 1):
        r = np.arange(off[e], off[e + 1])
        if not len(r):
            continue
        src = r if c["gather"] is None else np.where(c["gather"][r] < 0, -1, c["gather"][r] // c["k"])
        ok = (src >= 0) & (src < len(x))
        xe, we = x[np.where(ok, src, 0)], values(*c["w"][e], FP4, c["K"])
        with np.errstate(all="ignore"):
            y[r] = np.where(ok[:, None], xe @ we.T, 0.0)
            mag[r] = np.where(ok[:, None], np.abs(xe) @ np.abs(we).T, 0.0)
    return y, mag


def moe_device(c):
    t = {"Xq": stored(c["x"], c["fmt"]), "sx": c["sx"], "gather": c["gather"], "offsets": c["offsets"],
         "W": np.stack([pack(*w, c["N"], c["K"]) for w in c["w"]])}
    return {n: None if v is None else torch.from_numpy(np.ascontiguousarray(v)).to(DEV) for n, v in t.items()}


def half_step(dtype, y):
    """Bound of one rounding of y to `dtype`: half a step, and half the least subnormal of float16 near zero."""
    if dtype == torch.float32:
        return np.zeros_like(y)
    return np.abs(y) * (torch.finfo(dtype).eps / 2) + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def sum_bound(K, mag, fmt, exact):
    """|float32 sum - y|: a float32 sum of K exact products, whatever its order, is within K 2^-23 sum|x w| (each of at most K
    additions rounds or truncates by at most 2^-23 of a partial sum that sum|x w| bounds).  MXFP8 products, unless the output is
    float32, lose up to 2^-13 of the power of two of the largest of 8 neighbours each: 8 2^-13 of that one at most, and no
    more than 2^-10 of the 8 magnitudes' sum."""
    return (up(K, 128) * 2.0 ** -23 + (0 if exact or fmt == FP4 else 2.0 ** -10)) * mag


def product_bound(dtype, K, y, mag, fmt):
    """|got - y|: the sum's bound and one rounding to the output type."""
    e = sum_bound(K, mag, fmt, dtype == torch.float32)
    return e + half_step(dtype, np.abs(y) + e) + 1e-37


def silu_bound(K, y, mag, fmt):
    """(h, bound in float32) of silu(g) u: g, u off by eg, eu and |silu'| <= 1.1; the evaluation (an exponential good to |g| + 4 units
    of 2^-24, an addition, a reciprocal, two products) adds (8 + |g|) 2^-23 |h|."""
    I = y.shape[1] // 2
    g, u = y[:, :I], y[:, I:]
    e = sum_bound(K, mag, fmt, False)
    with np.errstate(all="ignore"):
        sg = g / (1 + np.exp(-g))
    h = sg * u
    b = 1.1 * e[:, :I] * (np.abs(u) + e[:, I:]) + np.abs(sg) * e[:, I:]
    return h, b + (8 + np.abs(g)) * 2.0 ** -23 * (np.abs(h) + b) + 1e-37


def assert_within(got, want, bound, what):
    """float16 results whose exact value rounds past 65504, at 65520 and more, are infinite; within the bound of that, either."""
    if isinstance(got, torch.Tensor):
        if got.dtype == torch.float16:
            got = got.double().cpu().numpy()
            far, near = np.abs(want) - bound >= 65520, np.abs(want) + bound >= 65520
            assert (got[far] == np.copysign(np.inf, want[far])).all(), what
            over = far | (near & (got == np.copysign(np.inf, want)))
            got = np.where(over, want, got)
        else:
            got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    over = np.abs(got - want) - bound
    i = int(np.argmax(over))
    assert over.reshape(-1)[i] <= 0, (what, got.reshape(-1)[i], want.reshape(-1)[i], bound.reshape(-1)[i])


def quant_bound(h, b, fmt):
    """|values of the codes - h| where the library quantizes values within b of h: b, and either half a step of the value's element
    or what saturating cuts (values past 6 or 448 units).  The unit follows from the block's largest magnitude, which is known
    within b: where a power of two lies between, either unit may be taken."""
    M, N = h.shape
    a, worst = np.abs(h) + b, np.zeros_like(h)
    for largest in (np.abs(h) + b, np.maximum(np.abs(h) - b, 0)):
        pad = np.zeros((M, up(N, 32)))
        pad[:, :N] = largest
        amax = pad.reshape(M, -1, 32).max(2)
        unit = np.exp2(np.floor(np.log2(np.maximum(amax, 1e-300))) - (2 if fmt == FP4 else 8))
        unit = np.repeat(unit, 32, 1)[:, :N]
        man, least = (1, 0) if fmt == FP4 else (3, -6)
        step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(a / unit, 1e-300))), least) - man) * unit
        cut = np.maximum(a - (6 if fmt == FP4 else 448) * unit, 0.0)
        worst = np.maximum(worst, np.maximum(step / 2, cut))
    return b + worst
