"""silu(g) u of the MX gate/up products over the whole range of g: every value is formed exactly from two E4M3 elements with a weight of 1."""
import math

import numpy as np
import pytest
import torch

import moe_token_int8_amd as L
from mx_cases import DEV, FP4, FP8, half_step, pack, stored

pytestmark = pytest.mark.gpu
GATES = [-math.inf, -3e38, -1e30, -1024.0, -200.0, -104.0, -100.0, -90.0, -89.0, -88.75, -88.0, -87.75, -87.5, -87.25, -87.0, -80.5, -60.0, -30.0,
         -17.0, -16.5, -5.0, -1.25, -1.0, -0.5, -2.0 ** -10, -2.0 ** -40, 0.0, 2.0 ** -40, 2.0 ** -10, 0.5, 1.0, 3.0, 16.5, 17.0, 60.0, 88.0, 89.0, 1024.0,
         1e30]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.lib()


def element(v):
    """(E4M3 code, scale byte) of the power of two and the four highest bits of v, and what is left of v."""
    if v == 0:
        return 0, 127, 0.0
    if math.isinf(v):
        return (0x7e if v > 0 else 0xfe), 254, 0.0                # 448 2^127
    m, e = math.frexp(abs(v))
    man = int(m * 16)                                             # 8 .. 15: 1.mmm
    code = (7 << 3) | (man - 8) | (0x80 if v < 0 else 0)          # exponent 0
    return code, 127 + e - 1, v - math.copysign(man / 16 * 2.0 ** e, v)


def problem(rows, I, u):
    """Rows of each gate in turn: x = its two elements in blocks 0 and 1 and u in block 2; gate weights 1 there, up weights 1 in block 2."""
    x, sx = np.zeros((rows, 128), np.uint8), np.full((rows, 4), 127, np.uint8)
    g = np.zeros(rows)
    for r in range(rows):
        v = GATES[r % len(GATES)]
        c0, b0, rest = element(v)
        c1, b1, rest = element(rest)
        x[r, 0], sx[r, 0], x[r, 32], sx[r, 1] = c0, b0, c1, b1
        g[r] = v - rest
        x[r, 64], sx[r, 2], _ = element(u)
    w = np.zeros((2 * I, 128), np.uint8)
    w[:I, 0] = w[:I, 32] = w[I:, 64] = 2                          # E2M1 1
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    W = dev(pack(w, np.full((2 * I, 4), 127, np.uint8), 2 * I, 128))
    off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    return g, (dev(stored(x, FP8)), dev(sx), FP8, None, 1, off, 1, W, W.numel(), 128)


def silu(g):
    """silu(g) in float64 as documented: 0 where exp(g) < 2^-126."""
    with np.errstate(all="ignore"):
        return np.where(np.exp(g) < 2.0 ** -126, 0.0, g / (1 + np.exp(-g)))


@pytest.mark.parametrize("u", [1.0, 2.0 ** 60, -(2.0 ** 100)])
@pytest.mark.parametrize("rows,I", [(39, 16), (400, 272), (2100, 2064)])
def test_silu_over_its_range(rows, I, u):
    g, args = problem(rows, I, u)
    H = torch.empty(rows, I, dtype=torch.bfloat16, device=DEV)
    L.w4a8_moe_gemm_silu_mx(*args, H)
    got = H.double().cpu().numpy()
    s = silu(g)
    want = s * u
    assert np.array_equal(got, np.repeat(got[:, :1], I, 1), equal_nan=True)
    got = got[:, 0]
    fits = np.abs(want) < 3.3e38
    bound = (2.0 ** -22 + np.where(np.isfinite(g), np.abs(g), 0) * 2.0 ** -24) * np.abs(want)
    bound = np.where(fits, bound + half_step(torch.bfloat16, np.abs(want) + bound) + 1e-37, 0)
    bad = [(a, b, c) for a, b, c, d, f in zip(g, got, want, bound, fits) if (not abs(b - c) <= d if f else b != math.copysign(math.inf, c))]
    assert not bad, bad[:20]
    for fmt in (FP4, FP8):
        q, sc = L.mx_empty(fmt, rows, I, DEV)
        L.w4a8_moe_gemm_silu_mx_quant(*args, I, fmt, q, sc)
        h = torch.empty(rows, I, device=DEV)
        L.w4a8_mx_dequant(q, sc, fmt, h)
        h = h.double().cpu().numpy()
        # equal values of a block: E2M1 keeps 1, 1.5, 2, 3, 4 (past 6 of a block's unit it saturates), E4M3 eighths
        near = np.abs(h - want[:, None]) <= np.abs(want[:, None]) * (1 / 3 if fmt == FP4 else 1 / 8) + 1e-37
        assert (near | ~(np.abs(want) < 3e38)[:, None]).all()
