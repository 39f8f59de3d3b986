"""Whole layers as they are used: router, dispatch, both products and combine, on 8-bit per-channel and on bfloat16 experts."""
import numpy as np
import pytest
import torch

import moe_token_int8_amd as L
import oracle as O
import workloads as W
from gpu_cases import check_moe
from moe_formats_cases import DEV, assert_within, half_step, silu_reference, w16_bound, w16_reference

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.lib()


def routed(seed, T, E, k, H, padded=0, hot=None):
    """X on the device, and the router's choice from random logits; `padded` tokens have no expert at all."""
    g = torch.Generator().manual_seed(seed)
    X = torch.randn(T, H, generator=g).to(BF16).to(DEV)
    logits = torch.randn(T, E, generator=g)
    if hot is not None:
        logits[:, hot] += 3.0
    if padded:
        logits[-padded:] = float("-inf")
    ids = torch.empty(T, k, dtype=torch.int32, device=DEV)
    w = torch.empty(T, k, dtype=torch.float32, device=DEV)
    L.w4a8_moe_route(logits.to(DEV), L.route_desc(E, k, renormalize=True), ids, w)
    return X, ids, w


def weights16(seed, E, H, I):
    g = torch.Generator().manual_seed(seed)
    return ((torch.randn(E, 2 * I, H, generator=g) * H ** -0.5).to(BF16), (torch.randn(E, H, I, generator=g) * I ** -0.5).to(BF16))


def run16(X, ids, w, Wgu, Wd, ws=None, out=None):
    T, k = ids.shape
    E, I2, H = Wgu.shape
    ws = torch.empty(L.w4a8_moe_w16a16_workspace_size(T, k, H, I2 // 2, E), dtype=torch.uint8, device=DEV) if ws is None else ws
    out = torch.empty_like(X) if out is None else out
    L.w4a8_moe_forward_w16a16(X, ids, w, Wgu, Wd, ws, out)
    return out


def reference16(X, ids, w, Wgu, Wd):
    """(out, bound) in float64 from the definition, choice by choice.  h carries the bound of its own product and rounding;
    the down product adds sum|w| times that and its own; combine sums k terms in float32 and rounds once."""
    X, ids, w = X.cpu(), ids.cpu(), w.cpu().double()
    T, k = ids.shape
    E, H, I = Wd.shape
    out, bound, mag = (torch.zeros(T, H, dtype=torch.float64) for _ in range(3))
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if not len(t):
            continue
        n = len(t)
        one = torch.tensor([0, n], dtype=torch.int32)
        h, hb = silu_reference(dict(X=X[t], W=Wgu[e:e + 1], gather=None, k=1, offsets=one, rows=n))
        d = Wd[e].double()
        y, ymag = h @ d.t(), (h.abs() + hb) @ d.abs().t()
        yb = hb @ d.abs().t() + I * 2.0 ** -23 * ymag
        yb = yb + half_step(BF16, y.abs() + yb)
        c = w[t, j][:, None]
        out.index_add_(0, t, c * y)
        bound.index_add_(0, t, c.abs() * yb)
        mag.index_add_(0, t, c.abs() * (y.abs() + yb))
    bound = bound + 2 * k * 2.0 ** -24 * mag
    return out, bound + half_step(BF16, out.abs() + bound) + 1e-38


@pytest.mark.parametrize("T,E,k,H,I,padded,hot", [
    (1, 8, 2, 64, 40, 0, None), (3, 64, 6, 264, 72, 1, None), (33, 16, 4, 512, 256, 5, 3), (200, 5, 2, 136, 328, 0, 0),
    (700, 4, 2, 1024, 1096, 30, 1), (1, 1, 1, 8, 8, 0, None), (9, 300, 8, 128, 64, 9, None),
])
def test_w16_layer(T, E, k, H, I, padded, hot):
    print("w16 layer", T, E, k, H, I, flush=True)
    X, ids, w = routed(51, T, E, k, H, padded, hot)
    Wgu, Wd = weights16(52, E, H, I)
    out = run16(X, ids, w, Wgu.to(DEV), Wd.to(DEV))
    want, bound = reference16(X, ids, w, Wgu, Wd)
    assert_within(out, want, bound, (T, E, k, H, I))
    if padded:
        assert (ids[-padded:] == -1).all() and (out[-padded:] == 0).all()


def weights8(seed, E, H, I):
    """(descs, device blobs, codes of every expert) with per-channel scales that keep the outputs near the inputs' size."""
    g = np.random.default_rng(seed)
    dgu, dd = L.desc(H, 2 * I, H, False, bits=8), L.desc(I, H, I, False, bits=8)
    qw, gu, dn = {}, [], []
    for e in range(E):
        cgu, cd = g.integers(-127, 128, (H, 2 * I), dtype=np.int8), g.integers(-127, 128, (I, H), dtype=np.int8)
        sgu = ((g.random((1, 2 * I)) + 0.5) * H ** -0.5 / 73).astype(np.float32)
        sd = ((g.random((1, H)) + 0.5) * I ** -0.5 / 73).astype(np.float32)
        gu.append(L.w4a8_pack_codes(dgu, cgu, sgu, None))
        dn.append(L.w4a8_pack_codes(dd, cd, sd, None))
        qw[e] = (cgu, sgu, None, cd, sd, None)
    return dgu, dd, L.to_device(dgu, gu, DEV), L.to_device(dd, dn, DEV), qw


def run8(X, ids, w, E, wts, ws=None, out=None):
    dgu, dd, gu, dn = wts[:4]
    T, k = ids.shape
    ws = torch.empty(L.w4a8_moe_workspace_size(T, k, dgu.K, dd.K, E), dtype=torch.uint8, device=DEV) if ws is None else ws
    out = torch.empty_like(X) if out is None else out
    L.w4a8_moe_forward_w8a8(X, ids, w, E, gu.blob, gu.stride, dgu, dn.blob, dn.stride, dd, ws, out)
    return out


def chain8(X, ids, w, E, wts):
    """The same layer call by call."""
    dgu, dd, gu, dn = wts[:4]
    T, k = ids.shape
    H, I, R = dgu.K, dd.K, T * k
    e = lambda *s, dt=torch.int32: torch.zeros(*s, dtype=dt, device=DEV)
    xq, sx, rows, offs, inv = e(T, H, dt=torch.int8), e(T, dt=torch.float32), e(R), e(E + 1), e(T, k)
    g, hq, sh, yd, out = e(R, 2 * I, dt=BF16), e(R, I, dt=torch.int8), e(R, dt=torch.float32), e(R, H, dt=BF16), e(T, H, dt=BF16)
    L.w4a8_quant_act(X, xq, sx)
    L.w4a8_moe_align(ids, E, rows, offs, inv)
    L.w4a8_moe_gemm_w8a8(xq, sx, rows, k, offs, E, R, gu.blob, gu.stride, dgu, g)
    L.w4a8_silu_mul_quant(g, hq, sh)
    L.w4a8_moe_gemm_w8a8(hq, sh, None, k, offs, E, R, dn.blob, dn.stride, dd, yd)
    L.w4a8_moe_combine(yd, inv, w, out)
    return out


@pytest.mark.parametrize("T,E,k,H,I,padded,hot", [
    (1, 8, 2, 128, 128, 0, None), (5, 32, 4, 384, 256, 2, None), (64, 16, 4, 512, 128, 0, 2), (700, 4, 2, 1152, 1280, 30, 1),
])
def test_w8_layer_is_its_steps(T, E, k, H, I, padded, hot):
    print("w8 layer", T, E, k, H, I, flush=True)
    X, ids, w = routed(53, T, E, k, H, padded, hot)
    wts = weights8(54, E, H, I)
    out = run8(X, ids, w, E, wts)
    assert torch.equal(out, chain8(X, ids, w, E, wts)) and torch.isfinite(out).all()
    if padded:
        assert (out[-padded:] == 0).all()


@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (40, 8, 3)])
def test_w8_layer_against_the_oracle(T, E, k):
    """K = H = I, so that the oracle's layer has one group size: the whole depth of both products."""
    K = 256
    X, ids, w = routed(55, T, E, k, K)
    wts = weights8(56, E, K, K)
    ref = O.moe_layer(X.float().cpu().numpy(), ids.cpu().numpy(), w.cpu().numpy(), lambda e: wts[4][e], E, K, K)
    check_moe(run8(X, ids, w, E, wts), ref, {e: wts[4][e] for e in np.unique(ids.cpu().numpy())}, K)


def guarded(n):
    buf = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=DEV)
    return buf, buf[256:-256]


def test_layers_write_their_output_and_workspace_only():
    T, E, k, H, I = 21, 6, 3, 256, 128
    X, ids, w = routed(57, T, E, k, H, 2)
    Wgu, Wd = (t.to(DEV) for t in weights16(58, E, H, I))
    wts = weights8(59, E, H, I)
    for run, size in ((lambda ws, out: run16(X, ids, w, Wgu, Wd, ws, out), L.w4a8_moe_w16a16_workspace_size(T, k, H, I, E)),
                      (lambda ws, out: run8(X, ids, w, E, wts, ws, out), L.w4a8_moe_workspace_size(T, k, H, I, E))):
        wbuf, ws = guarded(size)
        obuf, ob = guarded(T * H * 2)
        run(ws, ob.view(BF16).view(T, H))
        torch.cuda.synchronize()
        for buf in (wbuf, obuf):
            assert (buf[:256] == 0xA5).all() and (buf[-256:] == 0xA5).all()


def test_layers_in_graphs_on_two_streams():
    """A layer of each format captured with the router before it, replayed on other tokens while the other one runs on a
    second stream; every replay equals the eager result."""
    T, E, k, H, I = 48, 8, 2, 256, 384
    Wgu, Wd = (t.to(DEV) for t in weights16(60, E, H, I))
    wts = weights8(61, E, H, I)
    d = L.route_desc(E, k, renormalize=True)
    st = []
    for fmt in (16, 8):
        s = dict(X=torch.zeros(T, H, dtype=BF16, device=DEV), logits=torch.zeros(T, E, device=DEV), out=torch.zeros(T, H, dtype=BF16, device=DEV),
                 ids=torch.zeros(T, k, dtype=torch.int32, device=DEV), w=torch.zeros(T, k, device=DEV))
        size = L.w4a8_moe_w16a16_workspace_size if fmt == 16 else L.w4a8_moe_workspace_size
        s["ws"] = torch.empty(size(T, k, H, I, E), dtype=torch.uint8, device=DEV)

        def step(s=s, fmt=fmt):
            L.w4a8_moe_route(s["logits"], d, s["ids"], s["w"])
            if fmt == 16:
                run16(s["X"], s["ids"], s["w"], Wgu, Wd, s["ws"], s["out"])
            else:
                run8(s["X"], s["ids"], s["w"], E, wts, s["ws"], s["out"])

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        st.append((s, step, graph, side))
    g = torch.Generator(device=DEV).manual_seed(62)
    for i in range(4):
        want = []
        for s, step, _, _ in st:
            s["X"].copy_(torch.randn(T, H, generator=g, device=DEV))
            s["logits"].copy_(torch.randn(T, E, generator=g, device=DEV) * (i + 1))
            step()
            torch.cuda.synchronize()
            want.append(s["out"].clone())
            s["out"].zero_()
        torch.cuda.synchronize()
        for s, _, graph, side in st:
            with torch.cuda.stream(side):
                graph.replay()
        torch.cuda.synchronize()
        for (s, _, _, _), y in zip(st, want):
            assert torch.equal(s["out"], y), i
