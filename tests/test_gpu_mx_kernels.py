"""Every kernel of the microscaled (MX) products at sizes that choose it, against float64 products of the same codes on the device,
and its behaviour under calls that repeat, are captured, share a device or reach far into memory."""
import numpy as np
import pytest
import torch

import moe_token_int8_amd as L
from mx_cases import DEV, FP4, FP8, half_step, quant_bound, silu_bound, sum_bound

SENTINEL = 7.0
FEW, SOME, MANY = [9, 0, 1, 16, 0, 5, 9], [300, 0, 1, 17, 254, 0, 128], [0, 900, 31, 513, 1, 0, 55]
LARGE = [2100, 0, 129, 1800, 2, 0, 78]
# (rows of each expert, K, N): one size for each kernel at least, ragged in all three
SIZES = {
    "dense": [([5], 300, 523), ([200], 1099, 4109), ([400], 1099, 4109), ([2053], 1099, 2573), ([2053], 399, 4109), ([4109], 4199, 2571)],
    "moe": [(FEW, 300, 523), (SOME, 1099, 1037), (SOME, 400, 2575), (MANY, 1100, 4109), (MANY, 399, 8205), (LARGE, 4199, 2571)],
    "silu": [(FEW, 300, 528), (SOME, 1100, 528), (SOME, 400, 2576), (SOME, 1100, 4112), (MANY, 1099, 4112), (LARGE, 4199, 4112)],
}
SIZES["quantized"] = SIZES["silu"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.lib()


def random(seed, *shape):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(*shape, device=DEV, generator=g) * torch.exp2(torch.randint(-3, 4, (shape[-2], 1), device=DEV, generator=g))


def quantized(x, fmt):
    """Codes, scales and their values in float64."""
    q, s = L.mx_empty(fmt, *x.shape, DEV)
    L.w4a8_mx_quant(x, fmt, q, s)
    v = torch.empty_like(x)
    L.w4a8_mx_dequant(q, s, fmt, v)
    return q, s, v.double()


class Problem:
    def __init__(self, counts, K, width, fmt, seed=0, gathered=False):
        self.E, self.rows, self.K, self.fmt = len(counts), sum(counts), K, fmt
        self.src = max(1, self.rows // 3) if gathered else self.rows
        self.k = 3 if gathered else 1
        self.q, self.s, x = quantized(random(seed, self.src, K), fmt)
        off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        self.off = torch.from_numpy(off).to(DEV)
        g = np.random.default_rng(seed)
        entries = g.integers(0, self.src * self.k, size=self.rows).astype(np.int32)
        self.gather = torch.from_numpy(entries).to(DEV) if gathered else None
        self.blobs = torch.empty(self.E, L.w4a8_mx_packed_size(K, width), dtype=torch.uint8, device=DEV)
        y, mag = [], []
        for e in range(self.E):
            w = random(seed + 1 + e, width, K)
            L.w4a8_mx_pack(w, self.blobs[e])
            r = entries[off[e]:off[e + 1]] // self.k if gathered else np.arange(off[e], off[e + 1])
            xe, we = x[torch.from_numpy(r.astype(np.int64)).to(DEV)], quantized(w, FP4)[2].t().contiguous()
            y.append((xe @ we).cpu().numpy())
            mag.append((xe.abs() @ we.abs()).cpu().numpy())
        self.y, self.mag = np.concatenate(y), np.concatenate(mag)

    def moe(self):
        return (self.q, self.s, self.fmt, self.gather, self.k, self.off, self.E, self.blobs, self.blobs.shape[1], self.K)


def worst(got, want, bound):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    return float((np.abs(got - want) - bound).max())


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("counts,K,N", SIZES["dense"])
def test_dense(counts, K, N, fmt):
    p = Problem(counts, K, N, fmt)
    for dtype in (torch.bfloat16, torch.float32):
        Y = torch.full((p.rows, N + 5), SENTINEL, dtype=dtype, device=DEV)
        L.w4a8_mx_gemm(p.q, p.s, fmt, p.blobs[0], K, N, Y[:, :N])
        e = sum_bound(K, p.mag, fmt, dtype == torch.float32)
        assert worst(Y[:, :N], p.y, e + half_step(dtype, np.abs(p.y) + e) + 1e-37) <= 0
        assert (Y[:, N:] == SENTINEL).all()


@pytest.mark.gpu
@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("counts,K,N", SIZES["moe"])
def test_moe(counts, K, N, fmt, gathered):
    p = Problem(counts, K, N, fmt, 10, gathered)
    for dtype in (torch.float16, torch.float32):
        Y = torch.full((p.rows, N), SENTINEL, dtype=dtype, device=DEV)
        L.w4a8_moe_gemm_mx(*p.moe(), Y)
        e = sum_bound(K, p.mag, fmt, dtype == torch.float32)
        assert np.abs(p.y).max() < 60000
        assert worst(Y, p.y, e + half_step(dtype, np.abs(p.y) + e) + 1e-37) <= 0


@pytest.mark.gpu
@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("counts,K,I", SIZES["silu"])
def test_silu(counts, K, I, fmt, gathered):
    p = Problem(counts, K, 2 * I, fmt, 20, gathered)
    h, b = silu_bound(K, p.y, p.mag, fmt)
    H = torch.full((p.rows, I), SENTINEL, dtype=torch.bfloat16, device=DEV)
    L.w4a8_moe_gemm_silu_mx(*p.moe(), H)
    assert worst(H, h, b + half_step(torch.bfloat16, np.abs(h) + b)) <= 0
    for h_fmt in (FP4, FP8):
        q, s = L.mx_empty(h_fmt, p.rows, I, DEV)
        q.fill_(0xa5), s.fill_(0xa5)
        L.w4a8_moe_gemm_silu_mx_quant(*p.moe(), I, h_fmt, q, s)
        got = torch.empty(p.rows, I, device=DEV)
        L.w4a8_mx_dequant(q, s, h_fmt, got)
        assert worst(got, h, quant_bound(h, b, h_fmt)) <= 0
        Ip = -(-I // 128) * 128
        assert (q.view(p.rows, Ip // 32, -1)[:, -(-I // 32):] == 0).all() and (s[:, -(-I // 32):] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("rows,I", [(5, 16), (300, 2064), (700, 528)])
def test_small_parts_of_products_reach_quantized_h(rows, I):
    """x = 448, -448, 2^-6: gate 448 (silu is itself), up 448 - 448 + 2^-6, 14 bits below the largest product: h = 7."""
    x = torch.zeros(rows, 32, device=DEV)
    x[:, 0], x[:, 1], x[:, 2] = 448.0, -448.0, 2.0 ** -6
    q, s = L.mx_empty(FP8, rows, 32, DEV)
    L.w4a8_mx_quant(x, FP8, q, s)
    w = torch.zeros(2 * I, 32, device=DEV)
    w[:I, 0], w[I:, :3] = 1.0, 1.0
    W = torch.empty(L.w4a8_mx_packed_size(32, 2 * I), dtype=torch.uint8, device=DEV)
    # E2M1 blocks scale their largest value, 1, to 4: the products are the same
    L.w4a8_mx_pack(w, W)
    off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    hq, hs = L.mx_empty(FP8, rows, I, DEV)
    L.w4a8_moe_gemm_silu_mx_quant(q, s, FP8, None, 1, off, 1, W, W.numel(), 32, I, FP8, hq, hs)
    h = torch.empty(rows, I, device=DEV)
    L.w4a8_mx_dequant(hq, hs, FP8, h)
    assert (h == 7).all()


# ------------------------------------------------------------------------------------------- calls that repeat or meet others
def launches(p, N):
    """The products of p as closures over their outputs."""
    I = N // 2
    Y, H = torch.empty(p.rows, N, device=DEV), torch.empty(p.rows, I, dtype=torch.bfloat16, device=DEV)
    q, s = L.mx_empty(FP8, p.rows, I, DEV)
    return [(lambda: L.w4a8_moe_gemm_mx(*p.moe(), Y), (Y,)), (lambda: L.w4a8_moe_gemm_silu_mx(*p.moe(), H), (H,)),
            (lambda: L.w4a8_moe_gemm_silu_mx_quant(*p.moe(), I, FP8, q, s), (q, s))]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("counts,K,N", [(FEW, 300, 1024), (SOME, 400, 2080), (MANY, 1099, 4128)])
def test_repeat_and_replay(counts, K, N, fmt):
    """A call repeats bit for bit, also as a captured graph replayed several times with other work in between, on changed inputs."""
    p = Problem(counts, K, N, fmt, 30, True)
    ops = launches(p, N)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            for f, _ in ops:
                f()
    torch.cuda.synchronize()
    x = random(77, p.src, K)
    for i in range(4):
        x *= -1.25 if i % 2 else 0.7                                # eager work and new inputs between the replays
        L.w4a8_mx_quant(x, fmt, p.q, p.s)
        torch.cuda.synchronize()
        for f, outs in ops:
            for o in outs:
                o.fill_(1)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [o.clone() for _, outs in ops for o in outs]
        for f, _ in ops:
            f()
        for a, b in zip(replayed, [o for _, outs in ops for o in outs]):
            assert torch.equal(a, b)


@pytest.mark.gpu
def test_two_streams():
    """Calls on two streams at once, neither the current one, share nothing but their inputs."""
    ps = [(Problem(MANY, 1099, 4128, FP8, 40), 4128), (Problem(FEW, 300, 1024, FP4, 41, True), 1024)]
    alone, ops = [launches(*p) for p in ps], [launches(*p) for p in ps]
    for o in alone:
        for f, _ in o:
            f()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(21):
        for st, o in zip(streams, ops):
            with torch.cuda.stream(st):
                o[i % 3][0]()
    p = ps[1][0]
    Y = torch.empty(p.rows, 1024, device=DEV)
    L.w4a8_moe_gemm_mx(*p.moe(), Y, stream=streams[0].cuda_stream)  # by the argument
    torch.cuda.synchronize()
    for a, b in zip(alone, ops):
        for (_, x), (_, y) in zip(a, b):
            assert all(torch.equal(s, t) for s, t in zip(x, y))
    assert torch.equal(Y, alone[1][0][1][0])


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [FP4, FP8])
def test_many_experts(fmt):
    """1024 experts, a third of them without rows, more of them than rows or fewer."""
    g = np.random.default_rng(3)
    for top in (2, 40):
        counts = [int(c) if g.random() > 0.33 else 0 for c in g.integers(0, top, size=1024)]
        p = Problem(counts, 130, 272, fmt, 50, True)
        Y = torch.full((p.rows, 272), SENTINEL, device=DEV)
        L.w4a8_moe_gemm_mx(*p.moe(), Y)
        assert worst(Y, p.y, sum_bound(130, p.mag, fmt, True) + 1e-37) <= 0


# ------------------------------------------------------------------------------------------- far offsets
@pytest.mark.gpu
@pytest.mark.parametrize("rows", [3, 300])
def test_rows_of_the_output_far_apart(rows):
    """Row strides whose product with the rows passes 2^32 bytes."""
    N, ld = 528, 1 << 23
    p = Problem([rows], 399, N, FP8, 60)
    whole = torch.empty(rows * ld, device=DEV)
    for o in (torch.float32, torch.bfloat16):
        Y = whole.view(o)[:rows * ld].view(rows, ld)[:, 64:64 + N]
        Z = torch.empty(rows, N, dtype=o, device=DEV)
        Y.fill_(SENTINEL)
        L.w4a8_mx_gemm(p.q, p.s, FP8, p.blobs[0], 399, N, Y)
        L.w4a8_mx_gemm(p.q, p.s, FP8, p.blobs[0], 399, N, Z)
        assert torch.equal(Y, Z)


@pytest.mark.gpu
def test_rows_of_the_input_far_apart():
    """Activations past 4 GiB, dense and gathered from both ends (past the reach of 32-bit offsets the gathered call streams)."""
    K, N, M = 8192, 272, 540000
    p = Problem([200], K, N, FP8, 70)
    q, s = L.mx_empty(FP8, M, K, DEV)
    assert q.numel() > 1 << 32
    q.zero_(), s.zero_()
    q[:200], q[M - 200:], s[:200], s[M - 200:] = p.q, p.q, p.s, p.s
    Y = torch.empty(M, N, device=DEV)
    L.w4a8_mx_gemm(q, s, FP8, p.blobs[0], K, N, Y)
    assert worst(Y[:200], p.y, sum_bound(K, p.mag, FP8, True)) <= 0 and torch.equal(Y[:200], Y[M - 200:])
    assert (Y[200:M - 200] == 0).all()
    r = torch.arange(200, dtype=torch.int32, device=DEV)
    gather = torch.stack([r, r + (M - 200)], 1).reshape(-1).contiguous()
    Y = torch.empty(400, N, device=DEV)
    off = torch.tensor([0, 400], dtype=torch.int32, device=DEV)
    L.w4a8_moe_gemm_mx(q, s, FP8, gather, 1, off, 1, p.blobs, p.blobs.shape[1], K, Y)
    assert worst(Y[0::2], p.y, sum_bound(K, p.mag, FP8, True)) <= 0 and torch.equal(Y[0::2], Y[1::2])
    Y = torch.empty(200, K, dtype=torch.bfloat16, device=DEV)
    L.w4a8_mx_dequant(q[M - 200:], s[M - 200:], FP8, Y)
    x = torch.empty(M, K, dtype=torch.bfloat16, device=DEV)         # 8.8 GB
    L.w4a8_mx_dequant(q, s, FP8, x)
    assert torch.equal(x[M - 200:], Y) and torch.equal(x[:200], Y)
    q2, s2 = L.mx_empty(FP8, M, K, DEV)
    L.w4a8_mx_quant(x, FP8, q2, s2)
    q3, s3 = L.mx_empty(FP8, 200, K, DEV)
    L.w4a8_mx_quant(Y, FP8, q3, s3)
    assert torch.equal(q2[M - 200:], q3) and torch.equal(s2[M - 200:], s3) and torch.equal(q2[:200], q3)


# ------------------------------------------------------------------------------------------- together
def layer_inputs(T, k, E, H, I, fmt, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    GU = torch.empty(E, L.w4a8_mx_packed_size(H, 2 * I), dtype=torch.uint8, device=DEV)
    DN = torch.empty(E, L.w4a8_mx_packed_size(I, H), dtype=torch.uint8, device=DEV)
    L.w4a8_mx_pack(torch.randn(E, 2 * I, H, device=DEV, generator=g) / H ** 0.5, GU)
    down = torch.randn(E, H, I, device=DEV, generator=g) / I ** 0.5
    L.w4a8_mx_pack(down, DN)
    x = torch.randn(T, H, device=DEV, generator=g).to(torch.bfloat16)
    return GU, DN, down, x, torch.randn(T, E, device=DEV, generator=g)


def steps(x, ids, w, fmt, E, GU, DN, down, H, I):
    """The layer from the single calls, its last sum in float64; and the bound of a layer's distance from it.  Only the down product
    may differ (sum_bound of either call), and the weighted sum: k products and additions in float32, one rounding to bfloat16."""
    T, k = ids.shape
    q, s = L.mx_empty(fmt, T, H, DEV)
    L.w4a8_mx_quant(x, fmt, q, s)
    rows, inv = torch.zeros(T * k, dtype=torch.int32, device=DEV), torch.empty(T, k, dtype=torch.int32, device=DEV)
    off = torch.empty(E + 1, dtype=torch.int32, device=DEV)
    L.w4a8_moe_align(ids, E, rows, off, inv)
    hq, hs = L.mx_empty(fmt, T * k, I, DEV)
    hq.zero_(), hs.zero_()
    L.w4a8_moe_gemm_silu_mx_quant(q, s, fmt, rows, k, off, E, GU, GU.shape[1], H, I, fmt, hq, hs)
    y, h = torch.zeros(T * k, H, device=DEV), torch.empty(T * k, I, device=DEV)
    L.w4a8_moe_gemm_mx(hq, hs, fmt, None, 1, off, E, DN, DN.shape[1], I, y)
    L.w4a8_mx_dequant(hq, hs, fmt, h)
    mag, o = torch.zeros(T * k, H, dtype=torch.float64, device=DEV), off.tolist()
    for e in range(E):
        if o[e + 1] > o[e]:
            mag[o[e]:o[e + 1]] = h[o[e]:o[e + 1]].double().abs() @ quantized(down[e], FP4)[2].abs().t().contiguous()
    at, f = inv.long(), w.double()[..., None]
    there = (at >= 0)[..., None]
    term = torch.where(there, y[at.clamp(min=0)].double() * f, 0.0).cpu().numpy()
    m = torch.where(there, mag[at.clamp(min=0)] * f, 0.0).cpu().numpy()
    err = (sum_bound(I, m, fmt, False) + sum_bound(I, m, fmt, True)).sum(1)
    want = term.sum(1)
    err += (k + 1) * 2.0 ** -23 * (np.abs(term).sum(1) + err)
    return want, err + half_step(torch.bfloat16, np.abs(want) + err) + 1e-37


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("T,k,E", [(1, 6, 64), (5, 6, 64), (341, 6, 9), (342, 6, 64), (1400, 2, 7), (3, 3, 1), (40, 3, 1024)])
def test_layer_is_its_steps(T, k, E, fmt):
    """Small layers order the rows and quantize the tokens in one launch, larger ones (more than 2048 routed rows) in two: either
    agrees with the single calls.  Ids outside the experts add nothing, a token's id may be there twice."""
    H, I = 256, 96
    GU, DN, down, x, logits = layer_inputs(T, k, E, H, I, fmt, T)
    ids = logits.topk(min(k, E), 1).indices.to(torch.int32).repeat(1, k)[:, :k].contiguous()
    w = torch.rand(T, k, device=DEV)
    if T > 4:
        ids[1] = -1
        ids[2, 0], ids[3, :2] = E, ids[3, 0].item()
    ws = torch.empty(L.w4a8_moe_mx_workspace_size(T, k, H, I, E, fmt), dtype=torch.uint8, device=DEV)
    ws.fill_(0xff)
    out = torch.full((T, H), SENTINEL, dtype=torch.bfloat16, device=DEV)
    L.w4a8_moe_forward_mx(x, ids, w, E, fmt, GU, GU.shape[1], DN, DN.shape[1], I, ws, out)
    want, bound = steps(x, ids, w, fmt, E, GU, DN, down, H, I)
    assert worst(out, want, bound) <= 0
    if T > 4:
        assert (out[1] == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("T", [1, 37, 500])
def test_a_block_of_a_decoder(T, fmt):
    """As a decoder runs them: norm with quantized output -> dense product -> norm -> router -> expert layer -> norm with the block's
    gate, captured into one graph and replayed, against the same calls made one by one on another stream."""
    H, I, E, k = 512, 128, 16, 4
    GU, DN, _, x, _ = layer_inputs(T, k, E, H, I, fmt, 9)
    g = torch.Generator(device=DEV).manual_seed(T)
    B = torch.empty(L.w4a8_mx_packed_size(H, H), dtype=torch.uint8, device=DEV)
    L.w4a8_mx_pack(torch.randn(H, H, device=DEV, generator=g) / H ** 0.5, B)
    R = torch.randn(H, E, device=DEV, generator=g).to(torch.bfloat16)
    w1, w2, w3, gate = (torch.rand(H, device=DEV, generator=g) + 0.5 for _ in range(4))
    gate = gate.to(torch.bfloat16)[None]
    d, route = L.norm_desc(alpha=0.5), L.route_desc(E, k, renormalize=True)
    res0 = torch.randn(T, H, device=DEV, generator=g)

    def block(b):
        L.w4a8_norm_residual_quant(x, b["res"], L.norm_desc(), w1, b["res"], fmt, b["q"], b["s"])
        L.w4a8_mx_gemm(b["q"], b["s"], fmt, B, H, H, b["y"])
        L.w4a8_norm_residual(b["y"], b["res"], d, w2, b["res"], b["h"], post_w=w1)
        torch.mm(b["h"], R, out=b["logits"])
        L.w4a8_moe_route(b["logits"], route, b["ids"], b["w"])
        L.w4a8_moe_forward_mx(b["h"], b["ids"], b["w"], E, fmt, GU, GU.shape[1], DN, DN.shape[1], I, b["ws"], b["m"])
        L.w4a8_norm_residual(b["m"], b["res"], d, w3, b["res"], b["out"], post_w=w2, gate=gate)

    def buffers():
        b = {n: torch.empty(T, H, dtype=torch.bfloat16, device=DEV) for n in ("y", "h", "m", "out")}
        b["q"], b["s"] = L.mx_empty(fmt, T, H, DEV)
        b["logits"] = torch.empty(T, E, dtype=torch.bfloat16, device=DEV)
        b["ids"], b["w"] = torch.empty(T, k, dtype=torch.int32, device=DEV), torch.empty(T, k, device=DEV)
        b["ws"] = torch.empty(L.w4a8_moe_mx_workspace_size(T, k, H, I, E, fmt), dtype=torch.uint8, device=DEV)
        b["res"] = res0.clone()
        return b

    eager, captured = buffers(), buffers()
    torch.mm(eager["h"], R, out=eager["logits"])                    # the library's own set-up, outside the capture
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(captured)
    captured["res"].copy_(res0)
    for _ in range(3):
        graph.replay()
        with torch.cuda.stream(side):
            block(eager)
        torch.cuda.synchronize()
        for n in ("res", "q", "s", "y", "h", "ids", "m", "out"):
            assert torch.equal(captured[n], eager[n]), n
        assert torch.isfinite(eager["out"].float()).all()
