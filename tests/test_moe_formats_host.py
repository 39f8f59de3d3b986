"""Argument checks of the router and of the 8-bit and 16-bit grouped products: every refusal happens on the host before a
launch, so these run without a GPU (the pointers are never used)."""
import ctypes

import pytest

import moe_token_int8_amd as L

EI, EU, OK = L.W4A8_EINVAL, L.W4A8_EUNSUPPORTED, L.W4A8_OK
P = ctypes.c_void_p(1 << 20)                                    # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 2)


def route(desc=None, logits=P, dtype=L.W4A8_F32, T=4, ldl=None, bias=None, ids=P, w=P, **over):
    f = dict(E=64, k=4, score=0, renormalize=0, n_group=1, topk_group=1, scale=1.0)
    f.update(over)
    d = L.RouteDesc(**f)
    return L.lib().w4a8_moe_route(logits, dtype, T, f["E"] if ldl is None else ldl, bias, ctypes.byref(d), ids, w, None)


@pytest.mark.parametrize("over,want", [
    (dict(E=0), EI), (dict(E=-1), EI), (dict(k=0), EI), (dict(k=65), EI), (dict(E=128, k=65), EU), (dict(E=1025), EU),
    (dict(score=2), EI), (dict(score=-1), EI), (dict(renormalize=2), EI), (dict(n_group=-1), EI),
    (dict(n_group=5, topk_group=2), EI), (dict(n_group=8, topk_group=0), EI), (dict(n_group=8, topk_group=9), EI),
    (dict(n_group=32, topk_group=1), EI), (dict(scale=float("nan")), EI), (dict(scale=float("inf")), EI),
    (dict(T=-1), EI), (dict(T=(1 << 24) + 1), EU), (dict(ldl=63), EI), (dict(dtype=3), EI), (dict(dtype=-1), EI),
    (dict(logits=None), EI), (dict(ids=None), EI), (dict(w=None), EI), (dict(logits=ODD), EI), (dict(ids=ODD), EI),
    (dict(w=ODD), EI), (dict(bias=ODD), EI), (dict(logits=ctypes.c_void_p((1 << 20) + 1), dtype=L.W4A8_BF16), EI),
    (dict(T=0), OK), (dict(T=0, logits=None, ids=None, w=None), OK),
])
def test_route_refusals(over, want):
    assert route(**over) == want


def test_route_null_desc():
    assert L.lib().w4a8_moe_route(P, 1, 1, 64, None, None, P, P, None) == EI


def w8(d=None, Xq=P, sx=P, gather=None, k=2, off=P, E=4, rows=8, src=8, blobs=P, stride=None, Y=P, out=0, K=256, N=64):
    d = d or L.desc(K, N, K, False, bits=8)
    stride = L.w4a8_packed_size(d) if stride is None else stride
    return L.lib().w4a8_moe_gemm_w8a8(Xq, sx, gather, k, off, E, rows, src, blobs, stride, ctypes.byref(d), Y, out, None)


@pytest.mark.parametrize("over,want", [
    (dict(d=L.desc(256, 64, 128, False)), EU), (dict(d=L.desc(256, 64, 128, False, bits=8)), EU),
    (dict(d=L.desc(512, 64, 512, False)), EU), (dict(d=L.desc(256, 64, 256, True, bits=8)), EI),
    (dict(d=L.desc(192, 64, 192, False, bits=8)), EU), (dict(d=L.desc(256, 64, 256, False, bits=8, scale_bits=16)), EU),
    (dict(d=L.desc(133248, 16, 133248, False, bits=8)), EU), (dict(N=(1 << 20) + 1, K=128), EU),
    (dict(d=L.desc(128, 1 << 24, 128, False, bits=8)), EU),
    (dict(rows=-1), EI), (dict(src=-1), EI), (dict(E=0), EI), (dict(out=2), EI), (dict(out=-1), EI),
    (dict(rows=(1 << 24) + 1, src=1 << 25), EU), (dict(Xq=None), EI), (dict(sx=None), EI), (dict(off=None), EI),
    (dict(blobs=None), EI), (dict(Y=None), EI), (dict(src=7), EI), (dict(gather=P, k=0), EI), (dict(gather=P, src=0), EI),
    (dict(stride=1024), EI), (dict(Xq=ODD), EI), (dict(blobs=ODD), EI), (dict(Y=ODD, out=1), EI),
    (dict(Y=ctypes.c_void_p((1 << 20) + 1)), EI), (dict(rows=0), OK), (dict(rows=0, Xq=None, Y=None), OK),
])
def test_w8_refusals(over, want):
    assert w8(**over) == want


def w16(silu=False, X=P, dtype=0, ldx=None, gather=None, k=2, off=P, E=4, rows=8, src=8, W=P, stride=None, ldw=None, K=64,
        N=48, Y=P, ldy=None, out=None):
    ldw = K if ldw is None else ldw
    stride = (2 if silu else 1) * N * ldw if stride is None else stride
    a = (X, dtype, K if ldx is None else ldx, gather, k, off, E, rows, src, W, stride, ldw, K, N, Y, N if ldy is None else ldy)
    if silu:
        return L.lib().w4a8_moe_gemm_silu_w16a16(*a, None)
    return L.lib().w4a8_moe_gemm_w16a16(*a, dtype if out is None else out, None)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("over,want", [
    (dict(dtype=1), EI), (dict(dtype=3), EI), (dict(rows=-1), EI), (dict(src=-1), EI), (dict(E=0), EI), (dict(K=0), EI),
    (dict(N=0), EI), (dict(K=60), EI), (dict(ldx=68), EI), (dict(ldx=56), EI), (dict(ldw=68), EI), (dict(ldw=56), EI),
    (dict(ldy=47), EI), (dict(stride=64), EI), (dict(stride=8 * 64 * 48 + 4), EI), (dict(N=(1 << 20) + 1), EU),
    (dict(ldw=(1 << 23) + 8), EU), (dict(rows=(1 << 24) + 1, src=1 << 25), EU), (dict(X=None), EI), (dict(off=None), EI),
    (dict(W=None), EI), (dict(Y=None), EI), (dict(src=7), EI), (dict(gather=P, k=0), EI), (dict(gather=P, src=0), EI),
    (dict(X=ODD), EI), (dict(W=ODD), EI), (dict(Y=ctypes.c_void_p((1 << 20) + 1)), EI), (dict(rows=0), OK),
    (dict(rows=0, X=None, W=None, Y=None, off=None), OK),
])
def test_w16_refusals(silu, over, want):
    assert w16(silu, **over) == want


def test_w16_output_types():
    assert w16(dtype=0, out=2) == EI and w16(dtype=2, out=0) == EI and w16(out=3) == EI
    assert w16(dtype=0, out=1, rows=0) == OK and w16(dtype=2, out=1, rows=0) == OK
    assert w16(out=1, Y=ODD) == EI


def test_w16_silu_needs_both_halves():
    """A stride that holds I rows but not 2 I is refused."""
    assert w16(True, stride=48 * 64, rows=8) == EI
    assert w16(True, stride=(2 * 48 - 1) * 64 + 64, rows=0) == OK


def test_python_checks():
    import torch
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        L.w4a8_moe_route(x, L.route_desc(64, 4), torch.zeros(4, 4, dtype=torch.int32), torch.zeros(4, 4))   # not on a GPU


def test_experts_up_to_1024():
    assert w8(E=1024, rows=0) == OK and w8(E=1025) == EI
    assert w16(E=1024, rows=0) == OK and w16(E=1025) == EI
    assert w16(True, E=1024, rows=0) == OK and w16(True, E=1025) == EI


WS = ctypes.c_void_p(1 << 20)


def layer8(gu=None, dn=None, X=P, ids=P, w=P, T=4, k=2, E=8, gub=P, gus=None, db=P, ds=None, ws=WS, nws=None, out=P, H=256, I=128):
    gu = gu or L.desc(H, 2 * I, H, False, bits=8)
    dn = dn or L.desc(I, H, I, False, bits=8)
    gus = L.w4a8_packed_size(gu) if gus is None else gus
    ds = L.w4a8_packed_size(dn) if ds is None else ds
    nws = L.w4a8_moe_workspace_size(max(T, 0), max(k, 1), H, I, max(E, 1)) if nws is None else nws
    return L.lib().w4a8_moe_forward_w8a8(X, ids, w, T, k, E, gub, gus, ctypes.byref(gu), db, ds, ctypes.byref(dn), ws, nws, out, None)


@pytest.mark.parametrize("over,want", [
    (dict(T=-1), EI), (dict(k=0), EI), (dict(E=0), EI), (dict(E=1025), EI), (dict(X=None), EI), (dict(ids=None), EI),
    (dict(w=None), EI), (dict(ws=None), EI), (dict(out=None), EI), (dict(gub=None), EI), (dict(db=None), EI),
    (dict(X=ODD), EI), (dict(out=ODD), EI), (dict(gub=ODD), EI), (dict(ws=ctypes.c_void_p((1 << 20) + 16)), EI),
    (dict(nws=1024), L.W4A8_ESIZE), (dict(gus=64), EI), (dict(ds=64), EI), (dict(T=1 << 23, k=4), EU),
    (dict(gu=L.desc(256, 257, 256, False, bits=8)), EI), (dict(dn=L.desc(128, 128, 128, False, bits=8)), EI),
    (dict(dn=L.desc(256, 256, 256, False, bits=8)), EI), (dict(gu=L.desc(256, 256, 128, False)), EU),
    (dict(dn=L.desc(128, 256, 128, False)), EU), (dict(H=128, I=16512), EU), (dict(H=65664, I=128), EU),
    (dict(T=0), OK), (dict(T=0, X=None, ids=None, w=None, ws=None, out=None), OK),
])
def test_w8_layer_refusals(over, want):
    assert layer8(**over) == want


def layer16(X=P, ids=P, w=P, T=4, k=2, E=8, gu=P, gus=None, dn=P, ds=None, H=256, I=72, ws=WS, nws=None, out=P):
    nws = L.w4a8_moe_w16a16_workspace_size(max(T, 0), max(k, 1), H, I, max(E, 1)) if nws is None else nws
    return L.lib().w4a8_moe_forward_w16a16(X, ids, w, T, k, E, gu, 2 * I * H if gus is None else gus, dn, H * I if ds is None else ds,
                                           H, I, ws, nws, out, None)


@pytest.mark.parametrize("over,want", [
    (dict(T=-1), EI), (dict(k=0), EI), (dict(E=0), EI), (dict(E=1025), EI), (dict(H=0), EI), (dict(I=0), EI), (dict(H=252), EI),
    (dict(I=68), EI), (dict(X=None), EI), (dict(ids=None), EI), (dict(w=None), EI), (dict(ws=None), EI), (dict(out=None), EI),
    (dict(gu=None), EI), (dict(dn=None), EI), (dict(X=ODD), EI), (dict(out=ODD), EI), (dict(gu=ODD), EI), (dict(dn=ODD), EI),
    (dict(ws=ctypes.c_void_p((1 << 20) + 16)), EI), (dict(nws=1024), L.W4A8_ESIZE), (dict(gus=72 * 256), EI), (dict(ds=64), EI),
    (dict(gus=2 * 72 * 256 + 4), EI), (dict(T=1 << 23, k=4), EU), (dict(T=0), OK),
    (dict(T=0, X=None, ids=None, w=None, ws=None, out=None), OK),
])
def test_w16_layer_refusals(over, want):
    assert layer16(**over) == want


def test_w16_workspace_size():
    """Routing (three integer arrays), h and the expert outputs, each piece 256-byte aligned."""
    up = lambda n: (n + 255) // 256 * 256
    assert L.w4a8_moe_w16a16_workspace_size(5, 3, 64, 24, 7) == 2 * up(60) + up(32) + up(15 * 24 * 2) + up(15 * 64 * 2)
    for bad in ((-1, 1, 8, 8, 1), (1, 0, 8, 8, 1), (1, 1, 0, 8, 1), (1, 1, 8, 0, 1), (1, 1, 8, 8, 0)):
        assert L.w4a8_moe_w16a16_workspace_size(*bad) == 0
