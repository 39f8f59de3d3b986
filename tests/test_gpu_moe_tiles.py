"""Grouped products at sizes whose experts are worth MFMA tiles, of 128 x 128 (about 2050 columns) and of 256 x 256 (4100), beside experts of every smaller row class, and at
the limits of the launches: many experts, more tiles than a workgroup lists at once, weights past the Infinity Cache,
activations that 32-bit offsets do not reach."""
import numpy as np
import pytest
import torch

import moe_token_int8_amd as L
from moe_formats_cases import DEV, assert_within, half_step, offsets_of, w16_bound, w16_inputs, w16_reference, w8_inputs
from test_gpu_moe_formats import SENTINEL, check_silu, check_w16, check_w8, run_w16, run_w8, w8_device

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.lib()


# full tiles, half tiles (up to 128 rows behind the last full one) and ends inside a 16-row slice; then also every small class
LARGE = [129, 255, 300, 700, 1031]
MIXED = [1, 2, 16, 17, 32, 33, 64, 65, 129, 255, 257, 0, 511, 300, 5, 0]


@pytest.mark.parametrize("K,N", [(1152, 2306), (1280, 2049), (1152, 4102), (1280, 4097)])     # an odd and an even number of steps
def test_w8_tiles(K, N):
    print("w8 tiles", K, N, flush=True)
    check_w8(w8_inputs(21, LARGE, K, N))
    check_w8(w8_inputs(22, LARGE, K, N, src_rows=333, k=3, extra_rows=70), (torch.bfloat16,))


@pytest.mark.parametrize("K,N", [(1096, 2050), (1152, 2051), (1096, 4100), (1152, 4099)])     # K ends inside a step; whole steps
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_w16_tiles(K, N, dtype):
    print("w16 tiles", K, N, dtype, flush=True)
    check_w16(w16_inputs(23, dtype, LARGE, K, N), (dtype, torch.float32))
    check_w16(w16_inputs(24, dtype, LARGE, K, N, src_rows=333, k=3, extra_rows=70), (dtype,), pad=8)


@pytest.mark.parametrize("K,I", [(1096, 1100), (1280, 1153), (1096, 2060), (1280, 2051)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_silu_tiles(K, I, dtype):
    print("silu tiles", K, I, dtype, flush=True)
    check_silu(w16_inputs(25, dtype, LARGE, K, 2 * I, std=K ** -0.5))
    check_silu(w16_inputs(26, dtype, LARGE, K, 2 * I, src_rows=333, k=3, extra_rows=70, std=K ** -0.5), pad=8)


def test_every_row_class_in_one_call():
    print("classes w16", flush=True)
    check_w16(w16_inputs(48, torch.bfloat16, MIXED, 2200, 4100, src_rows=500, k=4, extra_rows=3), (torch.bfloat16,))
    check_w16(w16_inputs(27, torch.bfloat16, MIXED, 2200, 2050, src_rows=500, k=4, extra_rows=3), (torch.bfloat16,))
    print("classes silu", flush=True)
    check_silu(w16_inputs(28, torch.bfloat16, MIXED, 2200, 2 * 1030, std=0.02))
    print("classes w8", flush=True)
    check_w8(w8_inputs(29, MIXED, 2304, 4100, src_rows=500, k=4, extra_rows=3), (torch.bfloat16,))


@pytest.mark.parametrize("N", [2050, 4100])
def test_tiles_gather_entries_that_name_no_row(N):
    """Invalid entries give zero rows in tiles, and no row reads the one they would clamp to."""
    c = w16_inputs(30, torch.bfloat16, LARGE, 1096, N, src_rows=50, k=2)
    c["gather"][::5] = -1
    c["gather"][1::7] = 100
    c["gather"][2::9] = 2 ** 31 - 1
    c["X"][0] = float("nan")
    src = torch.div(c["gather"].long(), 2, rounding_mode="floor")
    zero = (src < 0) | (src >= 50)
    Y = run_w16(c).cpu()
    assert (Y[zero] == 0).all()
    assert torch.isnan(Y[src == 0]).all() and torch.isfinite(Y[~zero & (src != 0)]).all()


@pytest.mark.parametrize("N", [2050, 4100])
def test_tiles_infinity_in_the_last_values_of_k(N):
    """K = 1096 ends inside a 128-byte step; behind it the rows hold NaN, which must not reach any sum."""
    c = w16_inputs(31, torch.bfloat16, LARGE, 1096, N)
    c["X"][140, 1095] = float("inf")
    c["W"][3, 7, 1094] = float("-inf")
    Y = run_w16(c, torch.float32, pad=8).cpu()
    off = c["offsets"].tolist()
    bad = torch.zeros(c["rows"], N, dtype=torch.bool)
    bad[140] = True
    bad[off[3]:off[4], 7] = True
    assert not torch.isfinite(Y[bad]).any() and torch.isfinite(Y[~bad]).all()


@pytest.mark.parametrize("N", [2047, 4095])
def test_tiles_output_views_and_repeats(N):
    c = w16_inputs(32, torch.bfloat16, LARGE, 1096, N)
    want = run_w16(c)
    buf = torch.full((c["rows"] + 2, N + 6), SENTINEL, dtype=torch.bfloat16, device=DEV)
    got = run_w16(c, Y=buf[1:-1, 3:N + 3])
    assert torch.equal(got, want)
    buf[1:-1, 3:N + 3] = SENTINEL
    assert (buf == SENTINEL).all()
    c8 = w8_inputs(33, LARGE, 1152, N)
    dw = w8_device(c8)
    assert torch.equal(run_w8(c8, dw=dw), run_w8(c8, dw=dw))


def test_a_thousand_experts():
    g = np.random.default_rng(34)
    print("1000 experts", flush=True)
    check_w16(w16_inputs(34, torch.bfloat16, g.integers(0, 141, 1000).tolist(), 256, 512), (torch.bfloat16,))
    print("1024 experts, narrow", flush=True)
    check_w16(w16_inputs(35, torch.float16, g.integers(0, 9, 1024).tolist(), 64, 40), (torch.float16,))


def test_the_most_rows():
    """2^24 rows of one expert: a workgroup has more tiles than it lists at once.  Small integers, so every sum is exact."""
    rows, K, N = 1 << 24, 8, 513
    g = torch.Generator(device=DEV).manual_seed(36)
    X = torch.randint(-4, 5, (rows, K), generator=g, device=DEV).to(torch.bfloat16)
    W = torch.randint(-4, 5, (1, N, K), generator=g, device=DEV).to(torch.bfloat16)
    Y = torch.full((rows, N), SENTINEL, dtype=torch.bfloat16, device=DEV)
    print("most rows", flush=True)
    L.w4a8_moe_gemm_w16a16(X, None, 1, torch.tensor([0, rows], dtype=torch.int32, device=DEV), W, Y)
    torch.cuda.synchronize()
    wt = W[0].float().t().contiguous()
    for a in range(0, rows, 1 << 21):
        assert torch.equal(Y[a:a + (1 << 21)].float(), X[a:a + (1 << 21)].float() @ wt), a


def test_the_most_rows_of_small_tiles():
    """2^24 rows of two experts and 100 columns: 131073 tiles of 128 rows, one more than 512 workgroups list at once."""
    rows, K, N, cut = 1 << 24, 8, 100, (1 << 23) + 1
    g = torch.Generator(device=DEV).manual_seed(42)
    X = torch.randint(-4, 5, (rows, K), generator=g, device=DEV).to(torch.bfloat16)
    W = torch.randint(-4, 5, (2, N, K), generator=g, device=DEV).to(torch.bfloat16)
    Y = torch.full((rows, N), SENTINEL, dtype=torch.bfloat16, device=DEV)
    print("most rows, small tiles", flush=True)
    L.w4a8_moe_gemm_w16a16(X, None, 1, torch.tensor([0, cut, rows], dtype=torch.int32, device=DEV), W, Y)
    torch.cuda.synchronize()
    for e, (a, b) in enumerate(((0, cut), (cut, rows))):
        assert torch.equal(Y[a:b].float(), X[a:b].float() @ W[e].float().t().contiguous()), e


def test_weights_past_the_infinity_cache():
    """One row for each of 16 experts and more than 256 MiB of weights."""
    print("large weights w16", flush=True)
    check_w16(w16_inputs(37, torch.bfloat16, [1] * 16, 2056, 4096), (torch.bfloat16,))
    print("large weights silu", flush=True)
    check_silu(w16_inputs(38, torch.bfloat16, [1] * 16, 2056, 4096, std=0.02))
    print("large weights w8", flush=True)
    check_w8(w8_inputs(39, [1] * 16, 4224, 4096), (torch.bfloat16,))


@pytest.mark.parametrize("counts", [[20, 30], [129, 700]])
def test_gathered_activations_past_4_gib(counts):
    c = w16_inputs(40, torch.bfloat16, counts, 128, 48, src_rows=100, k=2)
    ldx = ((1 << 31) // 60 + 7) // 8 * 8                        # row 60 starts past 2^32 bytes
    X = torch.empty(100 * ldx, dtype=torch.bfloat16, device=DEV).as_strided((100, 128), (ldx, 1))
    X.copy_(c["X"])
    Y = torch.empty(c["rows"], 48, dtype=torch.bfloat16, device=DEV)
    L.w4a8_moe_gemm_w16a16(X, c["gather"].to(DEV), 2, c["offsets"].to(DEV), c["W"].to(DEV), Y)
    torch.cuda.synchronize()
    y, mag = w16_reference(c)
    assert_within(Y, y, w16_bound(torch.bfloat16, 128, y, mag), "far gathered rows")


def test_most_columns_of_many_experts():
    """2^20 columns: 128 experts with a row or more need more workgroups of 16 rows than a launch may have work-items for."""
    counts = [1] * 127 + [2]
    g = torch.Generator(device=DEV).manual_seed(41)
    X = torch.randint(-4, 5, (129, 8), generator=g, device=DEV).to(torch.bfloat16)
    W = torch.randint(-4, 5, (128, 1 << 20, 8), generator=g, device=DEV, dtype=torch.int8).to(torch.bfloat16)
    Y = torch.full((129, 1 << 20), SENTINEL, dtype=torch.bfloat16, device=DEV)
    print("most columns", flush=True)
    L.w4a8_moe_gemm_w16a16(X, None, 1, torch.from_numpy(offsets_of(counts)).to(DEV), W, Y)
    torch.cuda.synchronize()
    for e in range(128):
        r = slice(e, e + counts[e])
        assert torch.equal(Y[r].float(), X[r].float() @ W[e].float().t().contiguous()), e


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows", [1, 40, 300])
def test_silu_at_the_ends_of_the_range(rows, dtype):
    """h = g / (1 + exp(-g)) u for every pair of edge values, each made by one product with 1.  For g < 0 that is
    g exp(g) / (1 + exp(g)) u, and exp(g) may count as 0 below float32's least normal 2^-126: up to 2^-126 |g u|.  With an infinite u
    that is either side of 0 times infinity: g < -87.3 = ln 2^-126 gives a NaN there as float32's own silu(g) does (-250
    exp(-250) = -7e-107 is 0 in float32) where float64 still holds an infinity; both are taken."""
    inf, nan, big = float("inf"), float("nan"), torch.finfo(dtype).max
    v = torch.tensor([0.0, -0.0, 1.0, -1.0, 5.5, -5.5, 88.0, -88.0, 104.0, -104.0, 250.0, -250.0, big, -big, inf, -inf, nan]).to(dtype)
    g, u = (t.reshape(-1) for t in torch.meshgrid(v, v, indexing="ij"))
    W = torch.zeros(1, 2 * len(g), 8, dtype=dtype)
    W[0, :, 0] = torch.cat([g, u])
    X = torch.zeros(rows, 8, dtype=dtype)
    X[:, 0] = 1
    H = torch.empty(rows, len(g), dtype=dtype, device=DEV)
    L.w4a8_moe_gemm_silu_w16a16(X.to(DEV), None, 1, torch.tensor([0, rows], dtype=torch.int32, device=DEV), W.to(DEV), H)
    H = H.cpu()
    want = (g.double() / (1 + torch.exp(-g.double())) * u.double()).expand(rows, -1)
    under = (torch.isinf(u) & (g < -87.3)).expand(rows, -1)
    assert torch.equal(torch.isnan(H)[~under], torch.isnan(want)[~under])
    assert not torch.isfinite(H[under]).any()
    want = torch.where(under & torch.isnan(H), float("nan"), want)
    fit = want.abs() < torch.finfo(dtype).max                   # the rest are infinities or round to the largest values
    top = ~torch.isnan(want) & ~fit
    assert (H[top].double().abs() >= torch.finfo(dtype).max).all() and torch.equal(torch.sign(H[top]).double(), torch.sign(want[top]))
    e = 8 * 2.0 ** -23 * want[fit].abs() + 2.0 ** -126 * (g.double() * u.double()).abs().expand(rows, -1)[fit].nan_to_num(posinf=0)
    assert_within(H[fit], want[fit], e + half_step(dtype, want[fit].abs() + e) + 1e-38, "silu edges")


@pytest.mark.parametrize("N", [1026, 4100])
def test_tiles_in_a_graph(N):
    """Every product captured at tile sizes, replayed on other splits of the rows with eager calls between."""
    rows, E = 2400, 5
    c8 = w8_inputs(49, [rows, 0, 0, 0, 0], 1152, N, src_rows=200, k=3)
    c16 = w16_inputs(50, torch.bfloat16, [rows, 0, 0, 0, 0], 1096, N)
    d, w, t = w8_device(c8)
    X, W, off = c16["X"].to(DEV), c16["W"].to(DEV), t["offsets"]
    Y = [torch.zeros(rows, n, dtype=torch.bfloat16, device=DEV) for n in (N, N, N // 2)]

    def step():
        L.w4a8_moe_gemm_w8a8(t["Xq"], t["sx"], t["gather"], 3, off, E, rows, w.blob, w.stride, d, Y[0])
        L.w4a8_moe_gemm_w16a16(X, None, 1, off, W, Y[1])
        L.w4a8_moe_gemm_silu_w16a16(X, None, 1, off, W, Y[2])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for counts in ([rows, 0, 0, 0, 0], [300, 129, 70, 1800, 101], [0, 16, 33, 64, 2000], [480] * 5):
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


@pytest.mark.parametrize("E,counts", [(8, [100]), (64, [300, 0, 16, 5, 17, 0, 33]), (512, [70, 1, 2])])
def test_experts_named_more_than_once_by_a_token(E, counts):
    """With k = 8 no expert of an ordinary call has more than rows / 8 rows; these have, as if tokens named one repeatedly."""
    print("repeated", E, counts, flush=True)
    counts = counts + [0] * (E - len(counts))
    N = 2000 if E < 100 else 260
    check_w8(w8_inputs(51, counts, 2048, N, src_rows=30, k=8, extra_rows=2), (torch.bfloat16,))
    check_w16(w16_inputs(52, torch.bfloat16, counts, 2048, N, src_rows=30, k=8), (torch.bfloat16,))
    check_silu(w16_inputs(53, torch.float16, counts, 2048, N, src_rows=30, k=8, std=0.02))
