"""Edge values and odd calls of the grouped products in the MFMA-tile kernel, at sizes that tests/test_moe_formats_dispatch.py
holds to the tile size they are named for: gather entries that name no row, scales that are no numbers, the largest codes, float16's
ends, silu's ends, and graphs."""
import numpy as np
import pytest
import torch

import moe_token_int8_amd as L
from moe_formats_cases import (DEV, assert_within, half_step, offsets_of, silu_reference, w16_bound, w16_inputs, w16_reference,
                               w8_device, w8_inputs)
from test_gpu_moe_formats import SENTINEL, check_w8, run_w16, run_w8
from test_gpu_moe_tiles import LARGE

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16

# tile size -> columns of the plain products (K 1152 in 8, 1096 in 16 bits) and of the paired one, with LARGE rows
TILES = {"128 x 128": (2306, 1156), "256 x 256": (4102, 2312)}
SPLITS = [[2415, 0, 0, 0, 0], [300, 129, 70, 1815, 101], [0, 16, 33, 64, 2000], [483] * 5]     # of the rows of a graph


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.lib()


@pytest.mark.parametrize("tile", list(TILES))
def test_w8_gather_entries_that_name_no_row(tile):
    c = w8_inputs(81, LARGE, 1152, TILES[tile][0], src_rows=11, k=2)
    c["gather"][::5] = -1
    c["gather"][1::7] = 22                                      # token 11 of 11
    c["gather"][2::9] = 2 ** 31 - 1
    check_w8(c)


@pytest.mark.parametrize("tile", list(TILES))
@pytest.mark.parametrize("gathered", [False, True])
def test_w8_nan_and_zero_scales_stay_in_their_rows(tile, gathered):
    """Rows whose scale is NaN (marked non-finite when they were quantized) are NaN, rows of scale 0 and -0 zero, and no others."""
    c = w8_inputs(82, LARGE, 1152, TILES[tile][0], src_rows=sum(LARGE) if gathered else None)
    if gathered:
        c["gather"] = np.random.default_rng(83).permutation(sum(LARGE)).astype(np.int32)
    src = np.arange(sum(LARGE)) if c["gather"] is None else c["gather"]
    nan, zero = [2, 128, 129, 500, 2414], [0, 300, 1400]
    c["sx"][nan] = np.nan
    c["sx"][zero] = np.array([0.0, -0.0, 0.0], np.float32)
    Y = run_w8(c, torch.float32).cpu()
    isnan, iszero = torch.isnan(Y), Y == 0
    bad, none = torch.from_numpy(np.isin(src, nan)), torch.from_numpy(np.isin(src, zero))
    assert isnan[bad].all() and not isnan[~bad].any() and int(bad.sum()) == 5
    assert iszero[none].all() and int(none.sum()) == 3


@pytest.mark.parametrize("tile", list(TILES))
def test_w8_largest_codes_sum_exactly(tile):
    c = w8_inputs(84, LARGE, 1152, TILES[tile][0])
    c["codes"][:] = 127
    c["Xq"][:] = np.where(c["Xq"] >= 0, 127, -127)
    c["Xq"][::2] = 127
    check_w8(c)


@pytest.mark.parametrize("tile", list(TILES))
def test_float16_subnormals_and_overflow(tile):
    c = w16_inputs(85, F16, LARGE, 1096, TILES[tile][0])
    c["X"][1] *= 2.0 ** -14                                     # subnormal activations, and weights
    c["W"][0, 3] *= 2.0 ** -14
    y, mag = w16_reference(c)
    for out in (F16, torch.float32):
        assert_within(run_w16(c, out), y, w16_bound(out, 1096, y, mag), (tile, out))
    c["X"][:], c["W"][:] = 200.0, 100.0
    assert torch.isinf(run_w16(c)).all()                        # 1096 * 20000 is past 65504
    assert (run_w16(c, torch.float32) == 1096 * 20000.0).all()


@pytest.mark.parametrize("tile", list(TILES))
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_silu_gather_entries_that_name_no_row(tile, dtype):
    c = w16_inputs(86, dtype, LARGE, 1096, 2 * TILES[tile][1], src_rows=50, k=2, std=1096 ** -0.5)
    c["gather"][::5] = -1
    c["gather"][1::7] = 100
    c["gather"][2::9] = 2 ** 31 - 1
    c["X"][0] = float("nan")                                    # such rows must not pick up row 0 either
    src = torch.div(c["gather"].long(), 2, rounding_mode="floor")
    zero = (src < 0) | (src >= 50)
    fine = ~zero & (src != 0)
    H = run_w16(c, silu=True).cpu()
    assert (H[zero] == 0).all() and torch.isnan(H[src == 0]).all()
    c["X"][0] = 0
    h, bound = silu_reference(c)
    assert_within(H[fine], h[fine], bound[fine], (tile, dtype))


@pytest.mark.parametrize("tile", list(TILES))
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_silu_at_the_ends_of_the_range(tile, dtype):
    """h = g / (1 + exp(-g)) u for every pair of edge values, each made by one product with 1; the bounds are those of the same test
    of the streaming kernel: 8 units of float32, 2^-126 |g u| where exp(g) may count as 0, one rounding, and with an infinite u and
    g < -87.3 either an infinity or the NaN of 0 times infinity."""
    inf, nan, big = float("inf"), float("nan"), torch.finfo(dtype).max
    v = torch.tensor([0.0, -0.0, 1.0, -1.0, 5.5, -5.5, 88.0, -88.0, 104.0, -104.0, 250.0, -250.0, big, -big, inf, -inf, nan]).to(dtype)
    g, u = (t.reshape(-1) for t in torch.meshgrid(v, v, indexing="ij"))
    I, K, rows = TILES[tile][1], 1096, sum(LARGE)
    n = I // len(g)
    assert n * len(g) == I
    g, u = g.repeat(n), u.repeat(n)
    W = torch.zeros(len(LARGE), 2 * I, K, dtype=dtype)
    W[:, :, 0] = torch.cat([g, u])
    X = torch.zeros(rows, K, dtype=dtype)
    X[:, 0] = 1
    H = run_w16(dict(X=X, W=W, gather=None, k=1, offsets=torch.from_numpy(offsets_of(LARGE)), rows=rows), silu=True).cpu()
    # every row holds the same products, so one row against the definition, and the others against it bit by bit
    assert torch.equal(H.view(torch.int16), H[:1].view(torch.int16).expand(rows, -1))
    H = H[0]
    want = g.double() / (1 + torch.exp(-g.double())) * u.double()
    under = torch.isinf(u) & (g < -87.3)
    assert torch.equal(torch.isnan(H)[~under], torch.isnan(want)[~under]) and not torch.isfinite(H[under]).any()
    want = torch.where(under & torch.isnan(H), float("nan"), want)
    fit = want.abs() < torch.finfo(dtype).max
    top = ~torch.isnan(want) & ~fit
    assert (H[top].double().abs() >= torch.finfo(dtype).max).all() and torch.equal(torch.sign(H[top]).double(), torch.sign(want[top]))
    e = 8 * 2.0 ** -23 * want[fit].abs() + 2.0 ** -126 * (g.double() * u.double()).abs()[fit].nan_to_num(posinf=0)
    assert_within(H[fit], want[fit], e + half_step(dtype, want[fit].abs() + e) + 1e-38, "silu edges")


@pytest.mark.parametrize("tile", list(TILES))
def test_tiles_in_a_graph(tile):
    """Every product captured at this tile size, replayed on other splits of the rows with eager calls between."""
    rows, E, (N, I) = sum(SPLITS[0]), 5, TILES[tile]
    c8 = w8_inputs(87, SPLITS[0], 1152, N, src_rows=200, k=3)
    c16 = w16_inputs(88, BF16, SPLITS[0], 1096, max(N, 2 * I))
    d, w, t = w8_device(c8)
    X, W, off = c16["X"].to(DEV), c16["W"].to(DEV), t["offsets"]
    Y = [torch.zeros(rows, n, dtype=BF16, device=DEV) for n in (N, N, I)]

    def step():
        L.w4a8_moe_gemm_w8a8(t["Xq"], t["sx"], t["gather"], 3, off, E, rows, w.blob, w.stride, d, Y[0])
        L.w4a8_moe_gemm_w16a16(X, None, 1, off, W[:, :N], Y[1])
        L.w4a8_moe_gemm_silu_w16a16(X, None, 1, off, W[:, :2 * I], Y[2])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for counts in SPLITS:
        off.copy_(torch.from_numpy(offsets_of(counts)))
        for y in Y:
            y.fill_(SENTINEL)
        step()
        torch.cuda.synchronize()
        want = [y.clone() for y in Y]
        for y in Y:
            y.fill_(SENTINEL)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(Y, want))
        assert all((y[sum(counts):] == SENTINEL).all() for y in Y)


LEAST, MOST = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("tile", list(TILES))
@pytest.mark.parametrize("off,owner", [
    ([600, 1300, LEAST, LEAST, 600, 600], {0: (600, 1300), 3: (0, 600)}),       # an end so low that its difference to a start overflows
    ([0, 500, 500, -7, LEAST, 500], {0: (0, 500), 4: (0, 500)}),
    ([LEAST, 129, MOST, LEAST, -1, 0], {0: (0, 129), 1: (129, 2415)}),
    ([MOST, MOST, LEAST, LEAST, LEAST, LEAST], {}),
])
def test_malformed_offsets_stay_inside_the_rows(tile, off, owner):
    """An expert owns the rows between its two offsets, each clamped to the rows of the call, and none where they do not ascend."""
    rows, (N, I) = sum(LARGE), TILES[tile]
    o = torch.tensor(off, dtype=torch.int32)
    written = torch.zeros(rows, dtype=torch.bool)
    for a, b in owner.values():
        written[a:b] = True
    print("malformed", tile, off, flush=True)
    c = w16_inputs(89, BF16, LARGE, 1096, N)
    if off[1] == 500:
        c["W"][4] = c["W"][0]                                   # two experts own the same rows: let them say the same
    buf = torch.full((rows + 2, N), SENTINEL, dtype=BF16, device=DEV)
    run_w16(dict(c, offsets=o), Y=buf[1:-1])
    assert (buf[0] == SENTINEL).all() and (buf[-1] == SENTINEL).all() and (buf[1:-1][~written.to(DEV)] == SENTINEL).all()
    for e, (a, b) in owner.items():
        one = dict(X=c["X"][a:b], W=c["W"][e:e + 1], gather=None, k=1, offsets=torch.tensor([0, b - a]), rows=b - a)
        y, mag = w16_reference(one)
        assert_within(buf[1 + a:1 + b], y, w16_bound(BF16, 1096, y, mag), (tile, e))
    c8 = w8_inputs(90, LARGE, 1152, N)
    c8["offsets"] = np.array(off, np.int64).astype(np.int32)
    if off[1] == 500:
        c8["codes"][4], c8["sw"][4] = c8["codes"][0], c8["sw"][0]
    Y = run_w8(c8).cpu()
    assert (Y[~written] == SENTINEL).all()
    for e, (a, b) in owner.items():
        s = (c8["Xq"][a:b].astype(np.float64) @ c8["codes"][e].astype(np.float64)) * c8["sx"][a:b, None].astype(np.float64)
        want = torch.from_numpy(s * c8["sw"][e].astype(np.float64))
        bound = 4 * 2.0 ** -24 * want.abs()
        assert_within(Y[a:b], want, bound + half_step(BF16, want.abs() + bound) + 1e-38, (tile, e))
    H = run_w16(dict(c, W=c["W"][:, :2 * I] if 2 * I <= N else torch.cat([c["W"], c["W"]], 1)[:, :2 * I], offsets=o), silu=True)
    assert (H[~written.to(DEV)] == SENTINEL).all()
