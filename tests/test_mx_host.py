"""Argument checks of the microscaled (MX) calls and of the norm around a block, and the numbers that the host computes for them.
Every refusal happens on the host before a launch, so these run without a GPU (the pointers are never used)."""
import ctypes

import pytest

import moe_token_int8_amd as L

EI, EU, ES, OK = L.W4A8_EINVAL, L.W4A8_EUNSUPPORTED, L.W4A8_ESIZE, L.W4A8_OK
FP4, FP8, I8 = L.W4A8_MX_FP4, L.W4A8_MX_FP8, L.W4A8_QUANT_INT8
BASE = 1 << 20
P = ctypes.c_void_p(BASE)                                       # aligned, never dereferenced


def odd(n):
    return ctypes.c_void_p(BASE + n)


SIZES = [(dict(K=0), EI), (dict(K=-1), EI), (dict(K=(1 << 20) + 1), EU)]


def rows_call(name, X=P, dtype=L.W4A8_BF16, M=4, K=64, ld=None, fmt=FP8, Xq=P, sx=P):
    ld = K if ld is None else ld
    if name == "quant":
        return L.lib().w4a8_mx_quant(X, dtype, M, K, ld, fmt, Xq, sx, None)
    return L.lib().w4a8_mx_dequant(Xq, sx, fmt, M, K, X, dtype, ld, None)


@pytest.mark.parametrize("name", ["quant", "dequant"])
@pytest.mark.parametrize("over,want", SIZES + [
    (dict(M=-1), EI), (dict(fmt=2), EI), (dict(fmt=-1), EI), (dict(dtype=3), EI), (dict(dtype=-1), EI), (dict(ld=63), EI),
    (dict(X=None), EI), (dict(Xq=None), EI), (dict(sx=None), EI), (dict(X=odd(1)), EI), (dict(X=odd(2), dtype=L.W4A8_F32), EI),
    (dict(Xq=odd(8)), EI), (dict(sx=odd(2)), EI), (dict(M=1 << 30, K=1 << 20), EU), (dict(M=0), OK),
    (dict(M=0, X=None, Xq=None, sx=None), OK),
])
def test_rows_refusals(name, over, want):
    assert rows_call(name, **over) == want


@pytest.mark.parametrize("K,N,size", [
    (1, 1, 1024 + 256), (128, 16, 1024 + 256), (129, 17, 4 * 1024 + 2 * 256), (2048, 2816, 176 * 16 * 1024 + 44 * 16 * 256),
    (0, 8, 0), (8, 0, 0), (-1, 8, 0), ((1 << 20) + 1, 16, 0), (128, (1 << 20) + 1, 0), (1 << 20, 1 << 12, 0),
])
def test_packed_size(K, N, size):
    assert L.lib().w4a8_mx_packed_size(K, N) == size


def pack(W=P, dtype=L.W4A8_BF16, E=2, N=32, K=64, ldw=None, es=None, blobs=P, bs=None):
    ldw = K if ldw is None else ldw
    return L.lib().w4a8_mx_pack(W, dtype, E, N, K, ldw, N * ldw if es is None else es, blobs,
                                L.w4a8_mx_packed_size(K, N) if bs is None else bs, None)


@pytest.mark.parametrize("over,want", [
    (dict(N=0, bs=2560), EI), (dict(K=0, bs=2560), EI), (dict(E=-1), EI), (dict(E=1025), EI), (dict(dtype=3), EI), (dict(ldw=63), EI),
    (dict(W=None), EI), (dict(blobs=None), EI), (dict(W=odd(1)), EI), (dict(blobs=odd(8)), EI), (dict(bs=1024), EI),
    (dict(bs=2568), EI), (dict(es=31 * 64 + 63), EI), (dict(es=1 << 61), EI), (dict(N=1 << 20, K=1 << 12, bs=1 << 40), EU),
    (dict(E=0), OK), (dict(E=0, W=None, blobs=None), OK), (dict(E=1024, N=1 << 20, K=2048, bs=1 << 31, es=1 << 40), EU),
])
def test_pack_refusals(over, want):
    assert pack(**over) == want


@pytest.mark.parametrize("over,want", [
    (dict(K=48), EI), (dict(ldc=16), EI), (dict(ldc=40), EI), (dict(lds=1), EI), (dict(codes=None), EI), (dict(scales=None), EI),
    (dict(blob=None), EI), (dict(codes=odd(8)), EI), (dict(blob=odd(8)), EI), (dict(N=0), EI), (dict(K=1 << 20, N=1 << 12), EU),
])
def test_pack_codes_refusals(over, want):
    f = dict(codes=P, scales=P, N=32, K=64, ldc=None, lds=None, blob=P)
    f.update(over)
    ldc, lds = f["K"] // 2 if f["ldc"] is None else f["ldc"], f["K"] // 32 if f["lds"] is None else f["lds"]
    assert L.lib().w4a8_mx_pack_codes(f["codes"], f["scales"], f["N"], f["K"], ldc, lds, f["blob"], None) == want


@pytest.mark.parametrize("blob,N,K,codes,scales,want", [
    (None, 32, 64, P, P, EI), (P, 32, 64, None, P, EI), (P, 32, 64, P, None, EI), (odd(8), 32, 64, P, P, EI),
    (P, 32, 64, odd(8), P, EI), (P, 0, 64, P, P, EI), (P, 1 << 12, 1 << 20, P, P, EU),
])
def test_unpack_codes_refusals(blob, N, K, codes, scales, want):
    assert L.lib().w4a8_mx_unpack_codes(blob, N, K, codes, scales, None) == want


@pytest.mark.parametrize("over,want", SIZES + [
    (dict(fmt=2), EI), (dict(M=-1), EI), (dict(M=(1 << 24) + 1), EU), (dict(N=0), EI), (dict(N=(1 << 20) + 1), EU),
    (dict(K=1 << 20, N=1 << 12), EU), (dict(ldy=47), EI), (dict(out=3), EI), (dict(Xq=None), EI), (dict(sx=None), EI),
    (dict(blob=None), EI), (dict(Y=None), EI), (dict(Xq=odd(8)), EI), (dict(sx=odd(2)), EI), (dict(blob=odd(8)), EI),
    (dict(Y=odd(1)), EI), (dict(Y=odd(2), out=L.W4A8_F32), EI), (dict(M=0), OK), (dict(M=0, Xq=None, sx=None, blob=None, Y=None), OK),
])
def test_gemm_refusals(over, want):
    f = dict(Xq=P, sx=P, fmt=FP4, M=4, blob=P, K=64, N=48, Y=P, ldy=None, out=L.W4A8_BF16)
    f.update(over)
    assert L.lib().w4a8_mx_gemm(f["Xq"], f["sx"], f["fmt"], f["M"], f["blob"], f["K"], f["N"], f["Y"],
                                f["N"] if f["ldy"] is None else f["ldy"], f["out"], None) == want


def moe(form, Xq=P, sx=P, fmt=FP8, gather=None, k=2, off=P, E=4, rows=8, src=8, blobs=P, stride=None, K=64, N=48, Y=P, ldy=None,
        out=L.W4A8_BF16, sh=P, h_fmt=FP4):
    width = N if form == "product" else 2 * N
    stride = L.lib().w4a8_mx_packed_size(K, width) if stride is None else stride
    a = (Xq, sx, fmt, gather, k, off, E, rows, src, blobs, stride, K, N)
    ldy = N if ldy is None else ldy
    if form == "product":
        return L.lib().w4a8_moe_gemm_mx(*a, Y, ldy, out, None)
    if form == "silu":
        return L.lib().w4a8_moe_gemm_silu_mx(*a, Y, ldy, out, None)
    return L.lib().w4a8_moe_gemm_silu_mx_quant(*a, h_fmt, Y, sh, None)


FORMS = ["product", "silu", "quantized"]


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("over,want", SIZES + [
    (dict(fmt=2), EI), (dict(fmt=-1), EI), (dict(rows=-1), EI), (dict(src=-1), EI), (dict(E=0), EI), (dict(E=1025), EI), (dict(N=0), EI),
    (dict(N=1 << 20 | 16), EU), (dict(rows=(1 << 24) + 1, src=1 << 25), EU), (dict(src=(1 << 24) + 1), EU), (dict(Xq=None), EI),
    (dict(sx=None), EI), (dict(off=None), EI), (dict(off=None, E=1), EI), (dict(blobs=None), EI), (dict(Y=None), EI), (dict(src=7), EI),
    (dict(gather=P, k=0), EI), (dict(gather=P, src=0), EI), (dict(gather=odd(2)), EI), (dict(off=odd(2)), EI), (dict(stride=1024), EI),
    (dict(stride=(1 << 20) + 8), EI), (dict(Xq=odd(8)), EI), (dict(sx=odd(2)), EI), (dict(blobs=odd(8)), EI), (dict(Y=odd(1)), EI),
    (dict(rows=0), OK), (dict(rows=0, Xq=None, sx=None, blobs=None, Y=None, off=None, sh=None), OK),
])
def test_moe_refusals(form, over, want):
    assert moe(form, **over) == want


@pytest.mark.parametrize("form,over", [
    ("product", dict(ldy=47)), ("product", dict(out=3)), ("product", dict(out=L.W4A8_F32, Y=odd(2))),
    ("silu", dict(ldy=47)), ("silu", dict(out=L.W4A8_F32)), ("silu", dict(N=40)), ("quantized", dict(N=40)),
    ("quantized", dict(h_fmt=I8)), ("quantized", dict(h_fmt=-1)), ("quantized", dict(sh=None)), ("quantized", dict(sh=odd(2))),
    ("quantized", dict(Y=odd(8))),
])
def test_moe_refusals_of_one_form(form, over):
    assert moe(form, **over) == EI


def layer(X=P, ids=P, w=P, T=4, k=2, E=8, fmt=FP8, gu=P, gus=None, dn=P, ds=None, H=256, I=48, ws=P, nws=None, out=P):
    gus = L.lib().w4a8_mx_packed_size(H, 2 * I) if gus is None else gus
    ds = L.lib().w4a8_mx_packed_size(I, H) if ds is None else ds
    nws = L.lib().w4a8_moe_mx_workspace_size(T, k, H, I, E, fmt) if nws is None else nws
    return L.lib().w4a8_moe_forward_mx(X, ids, w, T, k, E, fmt, gu, gus, dn, ds, H, I, ws, nws, out, None)


@pytest.mark.parametrize("over,want", [
    (dict(T=-1), EI), (dict(k=0), EI), (dict(E=0), EI), (dict(E=1025), EI), (dict(fmt=2), EI), (dict(H=0), EI), (dict(I=0), EI),
    (dict(I=40), EI), (dict(H=(1 << 20) + 1), EU), (dict(I=(1 << 19) + 16), EU), (dict(T=1 << 23, k=4), EU),
    (dict(H=1 << 19, I=1 << 13), EU), (dict(T=1 << 20, H=1 << 15, nws=1 << 62), EU), (dict(X=None), EI), (dict(ids=None), EI),
    (dict(w=None), EI), (dict(ws=None), EI), (dict(out=None), EI), (dict(gu=None), EI), (dict(dn=None), EI), (dict(X=odd(1)), EI),
    (dict(out=odd(1)), EI), (dict(ids=odd(2)), EI), (dict(w=odd(2)), EI), (dict(gu=odd(8)), EI), (dict(dn=odd(8)), EI),
    (dict(ws=odd(16)), EI), (dict(nws=1024), ES), (dict(gus=64), EI), (dict(ds=64), EI), (dict(T=0), OK),
    (dict(T=0, X=None, ids=None, w=None, ws=None, out=None, gu=None, dn=None), OK),
])
def test_layer_refusals(over, want):
    assert layer(**over) == want


@pytest.mark.parametrize("a", [(-1, 2, 64, 32, 4, FP8), (4, 0, 64, 32, 4, FP8), (4, 2, 0, 32, 4, FP8), (4, 2, 64, 0, 4, FP8),
                               (4, 2, 64, 32, 0, FP8), (4, 2, 64, 32, 4, I8), (1 << 23, 4, 64, 32, 4, FP8),
                               ((1 << 31) - 1, (1 << 31) - 1, 64, 32, 4, FP8)])
def test_workspace_of_no_layer(a):
    assert L.lib().w4a8_moe_mx_workspace_size(*a) == 0


def test_workspace_grows_with_its_pieces():
    size = L.lib().w4a8_moe_mx_workspace_size
    for fmt, codes in ((FP4, 64 + 4), (FP8, 128 + 4)):
        # codes and scales of 5 tokens of 200 and 10 rows of 48, float32 [10, 200], 10 rows and places, 5 offsets; pieces end at 256
        need = 5 * 2 * codes + 10 * codes + 10 * 200 * 4 + 2 * 40 + 20
        assert need <= size(5, 2, 200, 48, 4, fmt) <= need + 8 * 256
    assert size(0, 2, 200, 48, 4, FP8) >= 0


# ------------------------------------------------------------------------------------------- norm
def norm(quant=False, X=P, dtype=L.W4A8_BF16, ldx=None, res=P, rt=L.W4A8_BF16, ldr=None, gate=None, ldg=0, pw=None, w=P, M=4, H=64,
         ro=P, ldo=None, Y=P, ldy=None, fmt=FP8, sx=P, desc=True, eps=1e-6, eps_post=1e-6, alpha=1.0):
    d = L.norm_desc(eps, eps_post, alpha)
    ld = lambda v: H if v is None else v  # noqa: E731
    a = (X, dtype, ld(ldx), res, rt, ld(ldr), gate, ldg, pw, w, ctypes.byref(d) if desc else None, M, H, ro, ld(ldo))
    if quant:
        return L.lib().w4a8_norm_residual_quant(*a, fmt, Y, sx, None)
    return L.lib().w4a8_norm_residual(*a, Y, ld(ldy), None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("over,want", [
    (dict(M=-1), EI), (dict(H=0), EI), (dict(H=65537), EU), (dict(M=(1 << 22) + 1), EU), (dict(dtype=3), EI), (dict(rt=3), EI),
    (dict(ldx=63), EI), (dict(ldr=63), EI), (dict(ldo=63), EI), (dict(gate=P, ldg=63), EI), (dict(desc=False), EI), (dict(eps=-1), EI),
    (dict(eps=NAN), EI), (dict(eps=INF), EI), (dict(pw=P, eps_post=-1), EI), (dict(pw=P, eps_post=NAN), EI), (dict(alpha=NAN), EI),
    (dict(alpha=INF), EI), (dict(X=None), EI), (dict(w=None), EI), (dict(X=odd(1)), EI), (dict(res=odd(1)), EI), (dict(ro=odd(1)), EI),
    (dict(gate=odd(1)), EI), (dict(w=odd(2)), EI), (dict(pw=odd(2)), EI), (dict(X=odd(2), dtype=L.W4A8_F32), EI),
    (dict(res=odd(2), rt=L.W4A8_F32), EI), (dict(M=0), OK), (dict(M=0, X=None, res=None, ro=None, Y=None, w=None, sx=None), OK),
])
def test_norm_refusals(quant, over, want):
    assert norm(quant, **over) == want


@pytest.mark.parametrize("quant,over", [
    (False, dict(Y=None, ro=None)), (False, dict(ldy=63)), (False, dict(Y=odd(1))), (True, dict(Y=None)), (True, dict(sx=None)),
    (True, dict(fmt=3)), (True, dict(fmt=-1)), (True, dict(Y=odd(8))), (True, dict(sx=odd(2))), (True, dict(fmt=I8, H=40)),
])
def test_norm_refusals_of_one_form(quant, over):
    assert norm(quant, **over) == EI


# ------------------------------------------------------------------------------------------- the host's numbers
def test_division_by_the_number_of_experts_of_a_token():
    """Gather entries r < 2^31 are divided by k as (mulhi(r, m) + r) >> s with s = ceil(log2 k), m = 2^32 (2^s - k) / k + 1."""
    for k in list(range(1, 130)) + [1 << 10, (1 << 10) + 1, 4095, 65535, 65536, 65537, 1 << 20, (1 << 24) - 1, 1 << 24, (1 << 31) - 1]:
        s = (k - 1).bit_length()
        m = (2 ** 32 * (2 ** s - k)) // k + 1
        assert m < 2 ** 32
        for q in {0, 1, 2, 3, 1000, (2 ** 31 - 1) // k - 1, (2 ** 31 - 1) // k}:
            for r in (q * k - 1, q * k, q * k + 1, q * k + k - 1):
                if 0 <= r < 2 ** 31:
                    t = (r * m >> 32) + r
                    assert t < 2 ** 32 and t >> s == r // k, (k, r)
