"""Expert-grouped products on 8-bit per-channel blobs and on 16-bit weights against float64.

Row counts are chosen around the 16-, 32-, 64-, 128- and 256-row tiles; bounds are derived in moe_formats_cases."""
import numpy as np
import pytest
import torch

import moe_token_int8_amd as L
from moe_formats_cases import (DEV, assert_within, half_step, silu_reference, w16_bound, w16_inputs, w16_reference,
                               w8_device, w8_inputs, w8_reference)

pytestmark = pytest.mark.gpu
SENTINEL = 7.0


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.lib()


COUNTS = {
    "one": [1],
    "few": [1, 0, 2, 16, 0, 17, 3],
    "edges": [15, 16, 17, 31, 32, 33, 63, 64, 65],
    "tiles": [127, 128, 129, 0, 255, 256, 257],
    "large": [0, 0, 700, 5, 0, 1031, 0],
    "empty": [0, 0, 0],
}


# ------------------------------------------------------------------------------------------- W8A8
def run_w8(c, out=torch.bfloat16, dw=None, Y=None):
    d, w, t = dw or w8_device(c)
    E, _, N = c["codes"].shape
    Y = torch.full((c["rows"], N), SENTINEL, dtype=out, device=DEV) if Y is None else Y
    L.w4a8_moe_gemm_w8a8(t["Xq"], t["sx"], t["gather"], c["k"], t["offsets"], E, c["rows"], w.blob, w.stride, d, Y,
                         L.W4A8_OUT_F32 if out == torch.float32 else L.W4A8_OUT_BF16)
    torch.cuda.synchronize()
    return Y


def check_w8(c, outs=(torch.float32, torch.bfloat16)):
    """The int32 sum is exact; its conversion and the two products round once each: 3 2^-24 relative, bounded by 4 2^-24."""
    want = torch.from_numpy(w8_reference(c))
    owned = int(c["offsets"][-1])
    dw = w8_device(c)
    for out in outs:
        Y = run_w8(c, out, dw)
        assert (Y[owned:] == SENTINEL).all()
        w = want[:owned]
        e = 4 * 2.0 ** -24 * w.abs()
        if owned:
            assert_within(Y[:owned], w, e + half_step(out, w.abs() + e) + 1e-38, (out, c["codes"].shape))


@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("K,N", [(128, 64), (256, 1), (384, 17), (1408, 300)])
def test_w8_sizes(counts, K, N):
    print("w8", counts, K, N, flush=True)
    check_w8(w8_inputs(1, COUNTS[counts], K, N))
    check_w8(w8_inputs(2, COUNTS[counts], K, N, src_rows=40, k=3, extra_rows=5), outs=(torch.bfloat16,))


@pytest.mark.parametrize("K,N", [(4096, 257), (7168, 48), (2048, 1026)])
def test_w8_deep(K, N):
    print("w8 deep", K, N, flush=True)
    check_w8(w8_inputs(3, [3, 40, 0, 300], K, N, src_rows=64, k=6))


def test_w8_extreme_codes_sum_exactly():
    """All codes at +-127: the largest int32 sum of K = 4096, past 2^24 where a float32 sum would round."""
    c = w8_inputs(4, [5, 70, 300], 4096, 48)
    c["Xq"][:] = np.where(c["Xq"] >= 0, 127, -127)
    c["codes"][:] = 127
    c["Xq"][::2] = 127
    check_w8(c)


def test_w8_gather_entries_that_name_no_row():
    c = w8_inputs(5, [20, 3, 150], 256, 70, src_rows=11, k=2)
    c["gather"][::5] = -1
    c["gather"][1::7] = 22                                      # token 11 of 11
    c["gather"][2::9] = 2 ** 31 - 1
    check_w8(c)


def test_w8_nan_scale_stays_in_its_row():
    """A row that quantization marked non-finite (scale NaN, codes 0) gives NaN outputs in that row only."""
    c = w8_inputs(6, [4, 140], 256, 33)
    for r in (2, 50, 143):
        c["sx"][r], c["Xq"][r] = np.nan, 0
    Y = run_w8(c, torch.float32).cpu()
    bad = torch.isnan(Y)
    assert bad[[2, 50, 143]].all() and int(bad.sum()) == 3 * 33


def test_w8_guards_around_the_output():
    c = w8_inputs(7, [3, 20, 200], 256, 37)
    buf = torch.full((c["rows"] + 8, 37), SENTINEL, dtype=torch.bfloat16, device=DEV)
    run_w8(c, Y=buf[4:-4])
    assert (buf[:4] == SENTINEL).all() and (buf[-4:] == SENTINEL).all() and (buf[4:-4] != SENTINEL).any()


def test_w8_same_result_twice():
    c = w8_inputs(8, [9, 33, 90, 400], 1024, 200, src_rows=100, k=4)
    dw = w8_device(c)
    assert torch.equal(run_w8(c, dw=dw), run_w8(c, dw=dw))


# ------------------------------------------------------------------------------------------- W16A16
def strided(t, pad, fill=float("nan")):
    """The same values with `pad` elements of `fill` behind every row (device tensor)."""
    full = torch.full((*t.shape[:-1], t.shape[-1] + pad), fill, dtype=t.dtype, device=DEV)
    full[..., : t.shape[-1]] = t.to(DEV)
    return full[..., : t.shape[-1]]


def run_w16(c, out=None, pad=0, silu=False, Y=None):
    X, W = strided(c["X"], pad), strided(c["W"], pad)
    N = W.shape[1] // (2 if silu else 1)
    if Y is None:
        Y = torch.full((c["rows"], N + pad), SENTINEL, dtype=out or X.dtype, device=DEV)[:, :N]
    gather = None if c["gather"] is None else c["gather"].to(DEV)
    f = L.w4a8_moe_gemm_silu_w16a16 if silu else L.w4a8_moe_gemm_w16a16
    f(X, gather, c["k"], c["offsets"].to(DEV), W, Y)
    torch.cuda.synchronize()
    return Y


def check_w16(c, outs, pad=0):
    y, mag = w16_reference(c)
    owned = int(c["offsets"][-1])
    for out in outs:
        Y = run_w16(c, out, pad)
        assert (Y[owned:] == SENTINEL).all()
        if owned:
            assert_within(Y[:owned], y[:owned], w16_bound(out, c["X"].shape[1], y[:owned], mag[:owned]), (out, c["W"].shape))


def check_silu(c, pad=0):
    h, bound = silu_reference(c)
    owned = int(c["offsets"][-1])
    H = run_w16(c, silu=True, pad=pad)
    assert (H[owned:] == SENTINEL).all()
    if owned:
        assert_within(H[:owned], h[:owned], bound[:owned], ("silu", c["W"].shape))


@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("K,N", [(8, 64), (64, 1), (136, 17), (1408, 300)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_w16_sizes(counts, K, N, dtype):
    print("w16", counts, K, N, dtype, flush=True)
    check_w16(w16_inputs(1, dtype, COUNTS[counts], K, N), (dtype, torch.float32))
    check_w16(w16_inputs(2, dtype, COUNTS[counts], K, N, src_rows=40, k=3, extra_rows=5), (dtype,), pad=8)


@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("K,I", [(8, 32), (72, 1), (328, 45), (1024, 176)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_silu_sizes(counts, K, I, dtype):
    print("silu", counts, K, I, dtype, flush=True)
    check_silu(w16_inputs(3, dtype, COUNTS[counts], K, 2 * I, std=K ** -0.5))
    check_silu(w16_inputs(4, dtype, COUNTS[counts], K, 2 * I, src_rows=40, k=3, extra_rows=5, std=K ** -0.5), pad=16)


@pytest.mark.parametrize("K,N", [(4096, 258), (7168, 48), (2040, 1026)])
def test_w16_deep(K, N):
    print("w16 deep", K, N, flush=True)
    c = w16_inputs(5, torch.bfloat16, [3, 40, 0, 300], K, N, src_rows=64, k=6, std=0.02)
    check_w16(c, (torch.bfloat16, torch.float32))
    check_silu(c)


def test_w16_gather_entries_that_name_no_row():
    for silu in (False, True):
        c = w16_inputs(6, torch.bfloat16, [20, 3, 150], 256, 70, src_rows=11, k=2)
        c["gather"][::5] = -1
        c["gather"][1::7] = 22
        c["gather"][2::9] = 2 ** 31 - 1
        c["X"][0] = float("nan")                                # such rows must not pick up row 0 either
        src = torch.div(c["gather"].long(), 2, rounding_mode="floor")
        zero = (src < 0) | (src >= 11)
        Y = run_w16(c, silu=silu).cpu()
        assert (Y[zero] == 0).all()
        assert torch.isnan(Y[src == 0]).all() and torch.isfinite(Y[~zero & (src != 0)]).all()


@pytest.mark.parametrize("counts", [[5], [300]])
def test_w16_infinities_and_nans_stay_where_they_are(counts):
    """K = 40 ends inside a 128-byte unit: an infinity in the last values of a row or of a weight must not meet the zeros
    that stand behind K, and touches its own row or column only."""
    c = w16_inputs(7, torch.bfloat16, counts, 40, 50)
    c["X"][3, 39] = float("inf")
    c["X"][3, 0] = 1.0
    c["W"][0, 7, 38] = float("-inf")
    y = c["X"].double() @ c["W"][0].double().t()                # the same infinities and NaNs by IEEE arithmetic
    Y = run_w16(c, torch.float32, pad=8).cpu().double()
    assert torch.equal(torch.isnan(Y), torch.isnan(y))
    assert torch.equal(torch.isinf(Y), torch.isinf(y)) and torch.equal(Y[torch.isinf(Y)], y[torch.isinf(y)])


def test_w16_float16_subnormals_and_overflow():
    c = w16_inputs(8, torch.float16, [4, 130], 64, 32)
    c["X"][1] *= 2.0 ** -14                                     # subnormal activations
    c["W"][0, 3] *= 2.0 ** -14
    check_w16(c, (torch.float16, torch.float32))
    c["X"][:] = 200.0
    c["W"][:] = 100.0
    assert torch.isinf(run_w16(c)).all()                        # 64 * 20000 is past 65504
    assert (run_w16(c, torch.float32) == 64 * 20000.0).all()


@pytest.mark.parametrize("rows", [6, 200])
def test_w16_rows_and_experts_past_4_gib(rows):
    """Activation rows and experts that start beyond 2^32 bytes from the first."""
    c = w16_inputs(9, torch.bfloat16, [rows // 2, rows - rows // 2], 128, 48)
    ldx = (((1 << 32) // 2) // (rows // 2) + 127) // 8 * 8
    X = torch.empty(rows * ldx, dtype=torch.bfloat16, device=DEV).as_strided((rows, 128), (ldx, 1))
    X.copy_(c["X"])
    stride = (1 << 31) + 64
    W = torch.empty(stride + 48 * 128, dtype=torch.bfloat16, device=DEV).as_strided((2, 48, 128), (stride, 128, 1))
    W.copy_(c["W"])
    Y = torch.empty(rows, 48, dtype=torch.bfloat16, device=DEV)
    L.w4a8_moe_gemm_w16a16(X, None, 1, c["offsets"].to(DEV), W, Y)
    torch.cuda.synchronize()
    y, mag = w16_reference(c)
    assert_within(Y, y, w16_bound(torch.bfloat16, 128, y, mag), "far rows")


def test_w16_output_views():
    """Output rows that are not a multiple of four apart, and that start off an 8-byte boundary."""
    c = w16_inputs(10, torch.bfloat16, [3, 20, 200], 256, 44)
    want = run_w16(c)
    buf = torch.full((c["rows"] + 2, 51), SENTINEL, dtype=torch.bfloat16, device=DEV)
    got = run_w16(c, Y=buf[1:-1, 3:47])
    assert torch.equal(got, want)
    buf[1:-1, 3:47] = SENTINEL
    assert (buf == SENTINEL).all()


def test_streams_and_graph():
    """Both formats captured on one graph, replayed on other routings with eager calls between."""
    c8 = w8_inputs(11, [9, 0, 140, 33], 512, 96, src_rows=60, k=3)
    c16 = w16_inputs(12, torch.bfloat16, [9, 0, 140, 33], 96, 64)
    d, w, t = w8_device(c8)
    X16, W16, off = c16["X"].to(DEV), c16["W"].to(DEV), t["offsets"]
    Y8 = torch.zeros(182, 96, dtype=torch.bfloat16, device=DEV)
    Y16 = torch.zeros(182, 64, dtype=torch.bfloat16, device=DEV)
    H16 = torch.zeros(182, 32, dtype=torch.bfloat16, device=DEV)

    def step():
        L.w4a8_moe_gemm_w8a8(t["Xq"], t["sx"], t["gather"], 3, off, 4, 182, w.blob, w.stride, d, Y8)
        L.w4a8_moe_gemm_w16a16(X16, None, 1, off, W16, Y16)
        L.w4a8_moe_gemm_silu_w16a16(X16, None, 1, off, W16, H16)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for counts in ([9, 0, 140, 33], [182, 0, 0, 0], [1, 2, 3, 0], [0, 60, 61, 61]):
        off.copy_(torch.tensor([0, *np.cumsum(counts)], dtype=torch.int32))
        for y in (Y8, Y16, H16):
            y.fill_(SENTINEL)
        step()
        torch.cuda.synchronize()
        want = [y.clone() for y in (Y8, Y16, H16)]
        for y in (Y8, Y16, H16):
            y.fill_(SENTINEL)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((Y8, Y16, H16), want))


def test_malformed_offsets_stay_inside_the_output():
    """Offsets past the rows of the call are clamped to them."""
    c = w16_inputs(13, torch.bfloat16, [10, 30], 64, 40)
    X, W = c["X"].to(DEV), c["W"].to(DEV)
    buf = torch.full((48, 40), SENTINEL, dtype=torch.bfloat16, device=DEV)
    L.w4a8_moe_gemm_w16a16(X, None, 1, torch.tensor([0, 10, 47], dtype=torch.int32, device=DEV), W, buf[4:44])
    torch.cuda.synchronize()
    assert (buf[:4] == SENTINEL).all() and (buf[44:] == SENTINEL).all()
    y, mag = w16_reference(c)
    assert_within(buf[4:44], y, w16_bound(torch.bfloat16, 64, y, mag), "clamped")


@pytest.mark.parametrize("silu", [False, True])
def test_w16_single_entries_with_any_stride(silu):
    """One row, one expert, one column: their strides say nothing."""
    c = w16_inputs(14, torch.bfloat16, [1], 64, 2 if silu else 1)
    want = run_w16(c, silu=silu)
    X, W = c["X"].to(DEV).as_strided((1, 64), (0, 1)), c["W"].to(DEV)
    W = W.as_strided(W.shape, (3, 64, 1))
    Y = torch.zeros(1, 1, dtype=torch.bfloat16, device=DEV).as_strided((1, 1), (0, 1))
    f = L.w4a8_moe_gemm_silu_w16a16 if silu else L.w4a8_moe_gemm_w16a16
    f(X, None, 1, c["offsets"].to(DEV), W, Y)
    assert torch.equal(Y, want)
