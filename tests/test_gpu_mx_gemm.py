"""Products of MX activations with packed MXFP4 weights, dense and by expert, against float64.

Row counts lie around the 16-, 32-, 64-, 128- and 256-row tiles; bounds are derived in mx_cases."""
import numpy as np
import pytest
import torch

import moe_token_int8_amd as L
from mx_cases import (DEV, FP4, FP8, assert_within, encode, half_step, moe_device, moe_inputs, moe_reference, product_bound, quant_bound,
                      silu_bound, stored, unstored, up, values)

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


def run_moe(c, out=torch.float32, t=None, Y=None):
    t = t or moe_device(c)
    Y = torch.full((c["rows"], c["N"]), SENTINEL, dtype=out, device=DEV) if Y is None else Y
    L.w4a8_moe_gemm_mx(t["Xq"], t["sx"], c["fmt"], t["gather"], c["k"], t["offsets"], len(c["w"]), t["W"], t["W"].shape[1], c["K"], Y)
    torch.cuda.synchronize()
    return Y


def check_moe(c, outs=(torch.float32, torch.bfloat16)):
    y, mag = moe_reference(c)
    owned = int(c["offsets"][-1])
    t = moe_device(c)
    for out in outs:
        Y = run_moe(c, out, t)
        assert (Y[owned:] == SENTINEL).all()
        if owned:
            assert_within(Y[:owned], y[:owned], product_bound(out, c["K"], y[:owned], mag[:owned], c["fmt"]), (out, c["K"], c["N"]))


@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("K,N", [(32, 64), (128, 1), (300, 17), (1408, 300)])
def test_moe_sizes(counts, K, N, fmt):
    check_moe(moe_inputs(K + N + fmt, COUNTS[counts], K, N, fmt))


@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("T,k,E,K,N", [(1, 6, 64, 512, 96), (33, 4, 9, 1000, 130), (300, 3, 8, 640, 272)])
def test_moe_gather(T, k, E, K, N, fmt):
    g = np.random.default_rng(T)
    counts = np.bincount(g.integers(0, E, size=T * k), minlength=E)
    c = moe_inputs(T, counts, K, N, fmt, src_rows=T, k=k, extra_rows=5)
    check_moe(c, (torch.float32, torch.float16))


@pytest.mark.parametrize("fmt", [FP4, FP8])
def test_gather_entries_that_name_no_row(fmt):
    for counts, T in (([5, 9], 7), ([100, 300], 200)):
        c = moe_inputs(1, counts, 256, 80, fmt, src_rows=T, k=2)
        c["gather"][::5] = -1
        c["gather"][1::7] = 2 * T
        c["gather"][2::7] = 2 ** 31 - 1
        check_moe(c)


@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("M,K,N", [(1, 128, 16), (1, 4096, 130), (8, 1024, 1024), (16, 96, 48), (17, 2048, 64), (32, 257, 255), (64, 1408, 200),
                                   (100, 512, 512), (129, 1280, 300), (256, 768, 256), (513, 640, 770), (1500, 256, 96)])
def test_dense(M, K, N, fmt):
    c = moe_inputs(M + K, [M], K, N, fmt)
    y, mag = moe_reference(c)
    t = moe_device(c)
    for out in (torch.float32, torch.bfloat16, torch.float16):
        Y = torch.full((M, N + 5), SENTINEL, dtype=out, device=DEV)
        L.w4a8_mx_gemm(t["Xq"], t["sx"], fmt, t["W"][0], K, N, Y[:, :N])
        assert (Y[:, N:] == SENTINEL).all()
        assert_within(Y[:, :N], y, product_bound(out, K, y, mag, fmt), (out, M, K, N))
        assert torch.equal(Y, _again(lambda Z: L.w4a8_mx_gemm(t["Xq"], t["sx"], fmt, t["W"][0], K, N, Z[:, :N]), Y))


def _again(call, like):
    Z = torch.full_like(like, SENTINEL)
    call(Z)
    return Z


@pytest.mark.parametrize("M", [8, 200, 600])
def test_sums_that_float32_holds_are_exact(M):
    """E2M1 products are multiples of 1/4 up to 36; with block scales of 1/2 to 2 on both sides (multiples of 1/16, up to 144) 1024
    of them stay below 2^18 = 2^22 sixteenths: every partial sum is a float32."""
    c = moe_inputs(M, [M], 1024, 160, FP4, spread=1)
    y, _ = moe_reference(c)
    assert np.array_equal(run_moe(c).double().cpu().numpy(), y)


@pytest.mark.parametrize("M", [3, 40, 300])
@pytest.mark.parametrize("fmt", [FP4, FP8])
def test_scales_far_apart(M, fmt):
    """Blocks whose scales differ by up to 2^60 in one row."""
    c = moe_inputs(M, [M], 640, 90, fmt, spread=30)
    check_moe(c, (torch.float32,))


@pytest.mark.parametrize("M", [5, 50, 400])
@pytest.mark.parametrize("fmt", [FP4, FP8])
def test_nan_blocks_stay_in_their_row(M, fmt):
    c = moe_inputs(M, [M], 300, 70, fmt)
    c["sx"][M // 2, 3] = 255
    c["w"][0][1][66, 2] = 255
    y, _ = moe_reference(c)
    got = run_moe(c).cpu().numpy()
    bad = np.zeros((M, 70), bool)
    bad[M // 2], bad[:, 66] = True, True
    assert np.array_equal(np.isnan(got), bad)


@pytest.mark.parametrize("M", [2, 33, 300])
def test_unused_rows_and_malformed_offsets(M):
    """Offsets past the rows of the call, or going down, move nothing outside Y."""
    c = moe_inputs(M, [M, 0, 0], 128, 32, FP4)
    t = moe_device(c)
    for off in ([0, M, M + 1000, 5], [-7, M // 2, M // 2, 2 ** 31 - 1], [0, 0, 0, 0]):
        t["offsets"] = torch.tensor(off, dtype=torch.int32, device=DEV)
        big = torch.full((M + 64, 32), SENTINEL, device=DEV)
        run_moe(c, t=t, Y=big[32:32 + M])
        assert (big[:32] == SENTINEL).all() and (big[32 + M:] == SENTINEL).all()


# ------------------------------------------------------------------------------------------- gate/up
def run_silu(c, out, t):
    I = c["N"] // 2
    H = torch.full((c["rows"], I), SENTINEL, dtype=out, device=DEV)
    L.w4a8_moe_gemm_silu_mx(t["Xq"], t["sx"], c["fmt"], t["gather"], c["k"], t["offsets"], len(c["w"]), t["W"], t["W"].shape[1], c["K"], H)
    return H


@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("counts", ["few", "edges", "tiles", "large"])
@pytest.mark.parametrize("K,I", [(128, 16), (320, 48), (1408, 144)])
def test_silu(counts, K, I, fmt):
    c = moe_inputs(K + I, COUNTS[counts], K, 2 * I, fmt, spread=2)
    c["sx"][c["sx"] > 0] -= 6                                       # gates of a few units
    y, mag = moe_reference(c)
    owned = int(c["offsets"][-1])
    h, b = silu_bound(K, y[:owned], mag[:owned], fmt)
    t = moe_device(c)
    for out in (torch.bfloat16, torch.float16):
        H = run_silu(c, out, t)
        if out == torch.float16 and np.abs(h).max() > 60000:
            continue
        assert_within(H[:owned], h, b + half_step(out, np.abs(h) + b), (out, K, I))
    for h_fmt in (FP4, FP8):
        Hq, sh = L.mx_empty(h_fmt, c["rows"] + 3, I, DEV)
        Hq.fill_(0xa5), sh.fill_(0xa5)
        L.w4a8_moe_gemm_silu_mx_quant(t["Xq"], t["sx"], fmt, t["gather"], c["k"], t["offsets"], len(c["w"]), t["W"], t["W"].shape[1], K, I,
                                      h_fmt, Hq[:owned], sh[:owned])
        assert (Hq[owned:] == 0xa5).all() and (sh[owned:] == 0xa5).all()
        q, s = unstored(Hq[:owned].cpu().numpy(), h_fmt), sh[:owned].cpu().numpy()
        assert (q[:, I:] == 0).all() and (s[:, up(I, 32) // 32:] == 0).all()
        assert_within(values(q, s, h_fmt, I), h, quant_bound(h, b, h_fmt), (h_fmt, K, I))
        # the same values quantized apart: nearly all codes equal.  A value within its error of a tie may differ: steps are 2^-4 of a
        # value and more, errors some 1e-5 of it with MXFP8 activations (whose codes here spread over all exponents), 1e-6 with MXFP4
        code, sc = encode(h.astype(np.float32), h_fmt)
        assert np.mean(code != q) < (1e-2 if fmt == FP8 else 1e-3) and np.mean(sc != s) < (1e-2 if fmt == FP8 else 1e-3)


@pytest.mark.parametrize("M,K,N", [(8, 2048, 256), (200, 1408, 300), (700, 1024, 512)])
def test_fp8_error_on_normal_values(M, K, N):
    """What the products of MXFP8 lose in 16-bit outputs is far below their rounding: normwise, a float16 rounding is at most
    2^-11 / sqrt(3) = 2.9e-4 (uniform within half a step of at most 2^-10 of the value), and the sums add 1e-5."""
    g = np.random.default_rng(K)
    x, w = encode(g.standard_normal((M, K)), FP8), encode(g.standard_normal((N, K)) * 0.1, FP4)
    c = dict(x=x[0], sx=x[1], w=[w], gather=None, k=1, offsets=np.array([0, M], np.int32), rows=M, K=K, N=N, fmt=FP8)
    y, _ = moe_reference(c)
    t = moe_device(c)
    for out, most in ((torch.float16, 3.0e-4), (torch.float32, 1e-6)):
        got = run_moe(c, out, t).double().cpu().numpy()
        assert np.linalg.norm(got - y) / np.linalg.norm(y) < most


@pytest.mark.parametrize("T", [1, 40, 700])
def test_silu_gather_and_rows_of_nobody(T):
    g = np.random.default_rng(T)
    counts = np.bincount(g.integers(0, 6, size=T * 2), minlength=6)
    c = moe_inputs(T, counts, 256, 64, FP8, src_rows=T, k=2, extra_rows=4)
    c["sx"][c["sx"] > 0] -= 6
    c["gather"][0] = -1
    y, mag = moe_reference(c)
    owned = int(c["offsets"][-1])
    h, b = silu_bound(256, y[:owned], mag[:owned], FP8)
    t = moe_device(c)
    H = run_silu(c, torch.bfloat16, t)
    assert (H[owned:] == SENTINEL).all()
    assert_within(H[:owned], h, b + half_step(torch.bfloat16, np.abs(h) + b), T)
    Hq, sh = L.mx_empty(FP8, c["rows"], 32, DEV)
    Hq.fill_(0xa5), sh.fill_(0xa5)
    L.w4a8_moe_gemm_silu_mx_quant(t["Xq"], t["sx"], FP8, t["gather"], 2, t["offsets"], 6, t["W"], t["W"].shape[1], 256, 32, FP8, Hq, sh)
    assert (Hq[owned:] == 0xa5).all() and (sh[owned:] == 0xa5).all() and (Hq[0] == 0).all() and (sh[0] == 0).all()


# ------------------------------------------------------------------------------------------- the layer
def layer_reference(x, ids, w, gu, dn, H, I, fmt):
    """Float64 steps of the layer, with the two quantizations; gu, dn: (codes, scales) of each expert."""
    x = values(*encode(x, fmt), fmt, H)
    out, mag = np.zeros((len(x), H)), np.zeros((len(x), H))
    for t in range(len(x)):
        for j in range(ids.shape[1]):
            e = ids[t, j]
            if not 0 <= e < len(gu):
                continue
            y = values(*gu[e], FP4, H) @ x[t]
            with np.errstate(all="ignore"):
                h = y[:I] / (1 + np.exp(-y[:I])) * y[I:]
            h = values(*encode(h[None].astype(np.float32), fmt), fmt, I)[0]
            d = values(*dn[e], FP4, I) @ h
            out[t] += w[t, j] * d
            mag[t] += np.abs(w[t, j] * d)
    return out, mag


@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("T,k,E,H,I", [(1, 2, 4, 256, 64), (9, 3, 5, 300, 48), (70, 2, 3, 129, 96), (300, 2, 2, 64, 32)])
def test_layer(T, k, E, H, I, fmt):
    g = np.random.default_rng(T)
    from mx_cases import pack, random_codes

    gu = [random_codes(g, 2 * I, H, FP4, 1) for _ in range(E)]
    dn = [random_codes(g, H, I, FP4, 1) for _ in range(E)]
    for q, s in gu:
        s[s > 0] -= 5
    x = torch.from_numpy(g.standard_normal((T, H), dtype=np.float32)).to(torch.bfloat16)
    ids = np.stack([g.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    if T > 5:
        ids[3] = -1                                                 # a padded token
        ids[4, 0] = E
    w = g.random((T, k), dtype=np.float32)
    want, mag = layer_reference(x, ids, w, gu, dn, H, I, fmt)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    GU, DN = dev(np.stack([pack(*q, 2 * I, H) for q in gu])), dev(np.stack([pack(*q, H, I) for q in dn]))
    ws = torch.empty(L.w4a8_moe_mx_workspace_size(T, k, H, I, E, fmt), dtype=torch.uint8, device=DEV)
    ws.fill_(0xff)
    out = torch.full((T, H), SENTINEL, dtype=torch.bfloat16, device=DEV)

    def call(o):
        L.w4a8_moe_forward_mx(x.to(DEV), dev(ids), dev(w), E, fmt, GU, GU.shape[1], DN, DN.shape[1], I, ws, o)
    call(out)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    # an element of h within its float32 error of a tie may be quantized to its other neighbour, which moves an output by a share of its
    # magnitude: the bulk is held to one bfloat16 rounding, each output to the widest step (1/3 of a value of E2M1, 1/8 of E4M3)
    err = np.abs(got - want)
    assert np.quantile(err - half_step(torch.bfloat16, want) - 2.0 ** -14 * mag, 0.97) <= 0
    assert (err <= half_step(torch.bfloat16, want) + mag / (3 if fmt == FP4 else 8)).all()
    if T > 5:
        assert (got[3] == 0).all()
    assert torch.equal(out, _again(call, out))
