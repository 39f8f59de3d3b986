"""Argument checks of the Python calls of the microscaled (MX) formats and of the norm around a block.  Every refusal comes before
the library is called, so these run without a GPU: the calls see meta tensors (shapes, strides and types without storage) as tensors
of the current device, and the library is replaced by one that records its arguments."""
import pytest
import torch

import moe_token_int8_amd as L

META = torch.empty(0, device="meta").get_device()
FP4, FP8, I8 = L.W4A8_MX_FP4, L.W4A8_MX_FP8, L.W4A8_QUANT_INT8
BF16, F16, F32, U8, I32 = torch.bfloat16, torch.float16, torch.float32, torch.uint8, torch.int32


class Recorder:
    """Stands for the library: every entry point returns OK and notes its arguments; sizes are the real ones."""

    def __init__(self, real):
        self.calls, self.real = [], real

    def __getattr__(self, name):
        if name.endswith("_size") or name == "w4a8_status_string":
            return getattr(self.real, name)

        def entry(*args):
            self.calls.append((name, args))
            return L.W4A8_OK
        return entry


def require_current(tensors, int32=(), float32=(), int8=()):
    """The library's check of types (a meta tensor's device is no other than the host's, whose tensors the last test sees refused)."""
    if any(t.dtype is not d for d, of in ((torch.int32, int32), (F32, float32), (torch.int8, int8)) for t in of if t is not None):
        raise ValueError("another type is expected")


@pytest.fixture
def calls(monkeypatch):
    t = L._Torch()
    t.device, t.current, t.initialized, t.raw_stream = lambda: META, lambda: META, lambda: True, lambda dev: 0
    rec = Recorder(L.lib())
    monkeypatch.setattr(L, "_torch_of_calls", t)
    monkeypatch.setattr(L, "_torch", lambda: t)
    monkeypatch.setattr(L, "_require_current", require_current)
    monkeypatch.setattr(L, "lib", lambda: rec)
    return rec.calls


def meta(*shape, dtype=F32, ld=None):
    if ld is not None:
        return torch.empty_strided(shape, (ld, 1), dtype=dtype, device="meta")
    return torch.empty(*shape, dtype=dtype, device="meta")


def codes(fmt, M, K):
    return L.mx_empty(fmt, M, K, "meta")


def refused(calls, f, match=None, error=ValueError):
    with pytest.raises(error, match=match):
        f()
    assert not calls


# ------------------------------------------------------------------------------------------- quantization
@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("call", ["w4a8_mx_quant", "w4a8_mx_dequant"])
def test_rows(calls, call, fmt):
    def f(X=meta(5, 200, dtype=BF16), q=None, s=None, fmt=fmt):
        q, s = q if q is not None else codes(fmt if fmt in (FP4, FP8) else FP8, 5, 200)[0], s if s is not None else codes(FP8, 5, 200)[1]
        return L.w4a8_mx_quant(X, fmt, q, s) if call == "w4a8_mx_quant" else L.w4a8_mx_dequant(q, s, fmt, X)

    other = FP8 if fmt == FP4 else FP4
    refused(calls, lambda: f(q=codes(other, 5, 200)[0]), "codes and scales")
    refused(calls, lambda: f(q=codes(fmt, 4, 200)[0]), "codes and scales")
    refused(calls, lambda: f(s=codes(fmt, 4, 200)[1]), "codes and scales")
    refused(calls, lambda: f(q=codes(fmt, 5, 200)[0].view(torch.int8)), "codes and scales")
    refused(calls, lambda: f(q=codes(fmt, 10, 200)[0][::2]), "codes and scales")
    refused(calls, lambda: f(fmt=2), "fmt")
    refused(calls, lambda: f(X=meta(5, 200, dtype=torch.float64)))
    refused(calls, lambda: f(X=meta(200, 5, dtype=BF16).t()), "contiguous rows")
    refused(calls, lambda: f(X=meta(5, 200, dtype=BF16, ld=199)), "overlap")
    f()
    f(X=meta(5, 200, dtype=F32, ld=300))
    f(X=meta(5, 300, dtype=F16)[:, 50:250])
    at = (2, 3, 4) if call == "w4a8_mx_quant" else (3, 4, 7)
    assert [tuple(a[i] for i in at) for _, a in calls] == [(5, 200, 200), (5, 200, 300), (5, 200, 300)]


def test_packing(calls):
    size = L.w4a8_mx_packed_size(200, 48)
    W, B = meta(48, 200, dtype=BF16), meta(size, dtype=U8)
    W3, B3 = meta(3, 48, 200, dtype=BF16), meta(3, size, dtype=U8)
    refused(calls, lambda: L.w4a8_mx_pack(W, meta(size - 1, dtype=U8)), "packed weights")
    refused(calls, lambda: L.w4a8_mx_pack(W, meta(size, dtype=torch.int8)), "packed weights")
    refused(calls, lambda: L.w4a8_mx_pack(W3, B3[:2]), "same experts")
    refused(calls, lambda: L.w4a8_mx_pack(W3, meta(3, size - 16, dtype=U8)), "packed weights")
    refused(calls, lambda: L.w4a8_mx_pack(W3, B), "must be")
    refused(calls, lambda: L.w4a8_mx_pack(W3.transpose(1, 2), B3), "contiguous rows")
    refused(calls, lambda: L.w4a8_mx_pack(meta(48, 200, dtype=torch.int32), B))
    L.w4a8_mx_pack(W, B), L.w4a8_mx_pack(W3, B3), L.w4a8_mx_pack(W3[:0], B3[:0]), L.w4a8_mx_pack(W3[::2], B3[::2].contiguous())
    assert [(a[2], a[6], a[8]) for _, a in calls] == [(1, 0, 0), (3, 9600, size), (2, 19200, size)]
    calls.clear()
    c, s = meta(48, 96, dtype=U8), meta(48, 6, dtype=U8)
    B = meta(L.w4a8_mx_packed_size(192, 48), dtype=U8)
    refused(calls, lambda: L.w4a8_mx_pack_codes(c, meta(48, 5, dtype=U8), B), "codes and scales")
    refused(calls, lambda: L.w4a8_mx_pack_codes(meta(48, 88, dtype=U8), s, B), "codes and scales")
    refused(calls, lambda: L.w4a8_mx_pack_codes(c, s, B[16:]), "packed weights")
    refused(calls, lambda: L.w4a8_mx_unpack_codes(B, 48, 192, *codes(FP8, 48, 192)), "codes and scales")
    refused(calls, lambda: L.w4a8_mx_unpack_codes(B[16:], 48, 192, *codes(FP4, 48, 192)), "packed weights")
    L.w4a8_mx_pack_codes(c, s, B), L.w4a8_mx_unpack_codes(B, 48, 192, *codes(FP4, 48, 192))
    assert [n for n, _ in calls] == ["w4a8_mx_pack_codes", "w4a8_mx_unpack_codes"]


# ------------------------------------------------------------------------------------------- products
def test_gemm(calls):
    def f(fmt=FP8, M=5, K=200, N=48, x=None, blob=None, Y=None):
        q, s = codes(fmt, M, K) if x is None else x
        L.w4a8_mx_gemm(q, s, fmt, meta(L.w4a8_mx_packed_size(K, N), dtype=U8) if blob is None else blob, K, N,
                       meta(M, N, dtype=BF16) if Y is None else Y)

    refused(calls, lambda: f(x=codes(FP4, 5, 200)), "codes and scales")
    refused(calls, lambda: f(x=codes(FP8, 6, 200)), "codes and scales")
    refused(calls, lambda: f(blob=meta(L.w4a8_mx_packed_size(200, 48) - 1, dtype=U8)), "packed weights")
    refused(calls, lambda: f(Y=meta(5, 47, dtype=BF16)), "Y must be")
    refused(calls, lambda: f(Y=meta(5, 48, dtype=torch.float64)))
    refused(calls, lambda: f(Y=meta(48, 5, dtype=BF16).t()), "contiguous rows")
    refused(calls, lambda: f(Y=meta(1, 48, dtype=BF16).expand(5, 48)), "overlap")
    f(), f(Y=meta(5, 48, ld=64)), f(M=0), f(FP4)
    assert [(a[2], a[3], a[8], a[9]) for _, a in calls] == [(FP8, 5, 48, L.W4A8_BF16), (FP8, 5, 64, L.W4A8_F32), (FP8, 0, 48, L.W4A8_BF16),
                                                            (FP4, 5, 48, L.W4A8_BF16)]
    refused([], lambda: f(K=1 << 20, N=1 << 12, blob=meta(16, dtype=U8)), error=L.W4A8Error)


FORMS = ["product", "silu", "quantized"]


def moe(form, rows=6, K=200, N=48, E=3, k=2, src=4, fmt=FP8, x=None, gather=True, off=None, blobs=None, stride=None, out=None, h_fmt=FP4):
    size = L.w4a8_mx_packed_size(K, N if form == "product" else 2 * N)
    q, s = codes(fmt, src, K) if x is None else x
    a = (q, s, fmt, meta(rows, dtype=I32) if gather is True else gather, k, meta(E + 1, dtype=I32) if off is None else off, E,
         meta(E, size, dtype=U8) if blobs is None else blobs, size if stride is None else stride, K)
    if form == "quantized":
        return L.w4a8_moe_gemm_silu_mx_quant(*a, N, h_fmt, *(codes(h_fmt, rows, N) if out is None else out))
    return (L.w4a8_moe_gemm_mx if form == "product" else L.w4a8_moe_gemm_silu_mx)(*a, meta(rows, N, dtype=BF16) if out is None else out)


@pytest.mark.parametrize("form", FORMS)
def test_moe(calls, form):
    size = L.w4a8_mx_packed_size(200, 48 if form == "product" else 96)
    for over, match in [
        (dict(x=codes(FP4, 4, 200)), "codes and scales"), (dict(x=(codes(FP8, 4, 200)[0], codes(FP8, 5, 200)[1])), "codes and scales"),
        (dict(gather=meta(5, dtype=I32)), None), (dict(gather=meta(6, dtype=torch.int64)), None), (dict(gather=meta(12, dtype=I32)[::2]), None),
        (dict(off=meta(3, dtype=I32)), None), (dict(off=meta(5, dtype=I32)), None), (dict(off=meta(4, dtype=torch.int64)), None),
        (dict(off=meta(8, dtype=I32)[::2]), None), (dict(blobs=meta(3, size - 16, dtype=U8)), "packed weights"),
        (dict(blobs=meta(3, size, dtype=torch.int8)), "packed weights"), (dict(stride=size + 16), "packed weights"),
        (dict(stride=-16), "packed weights"), (dict(k=1 << 31), None),
    ]:
        refused(calls, lambda: moe(form, **over), match)
    moe(form), moe(form, gather=None, src=6), moe(form, rows=0), moe(form, fmt=FP4), moe(form, gather=meta(9, dtype=I32))
    assert [(a[2], a[4], a[6], a[7], a[8], a[11], a[12]) for _, a in calls] == [
        (FP8, 2, 3, 6, 4, 200, 48), (FP8, 2, 3, 6, 6, 200, 48), (FP8, 2, 3, 0, 4, 200, 48), (FP4, 2, 3, 6, 4, 200, 48), (FP8, 2, 3, 6, 4, 200, 48)]


def test_moe_outputs(calls):
    for form in ("product", "silu"):
        refused(calls, lambda: moe(form, out=meta(48, 6, dtype=BF16).t()), "contiguous rows")
        refused(calls, lambda: moe(form, out=meta(6, 48, dtype=torch.float64)))
    refused(calls, lambda: moe("quantized", out=codes(FP8, 6, 48)), "codes and scales")
    refused(calls, lambda: moe("quantized", out=(codes(FP4, 6, 48)[0], codes(FP4, 5, 48)[1])), "codes and scales")
    refused(calls, lambda: moe("quantized", h_fmt=I8, out=codes(FP8, 6, 48)), "fmt")


def test_layer(calls):
    def f(T=5, k=2, E=3, H=200, I=48, fmt=FP8, **over):
        sg, sd = L.w4a8_mx_packed_size(H, 2 * I), L.w4a8_mx_packed_size(I, H)
        a = dict(X=meta(T, H, dtype=BF16), ids=meta(T, k, dtype=I32), w=meta(T, k), gu=meta(E, sg, dtype=U8), gus=sg,
                 dn=meta(E, sd, dtype=U8), ds=sd, ws=meta(4096, dtype=U8), out=meta(T, H, dtype=BF16))
        a.update(over)
        L.w4a8_moe_forward_mx(a["X"], a["ids"], a["w"], E, fmt, a["gu"], a["gus"], a["dn"], a["ds"], I, a["ws"], a["out"])

    size = L.w4a8_mx_packed_size(200, 96)
    for over in [
        dict(X=meta(5, 200, dtype=F16)), dict(out=meta(5, 200, dtype=F16)), dict(out=meta(4, 200, dtype=BF16)), dict(ids=meta(4, 2, dtype=I32)),
        dict(ids=meta(5, 2, dtype=torch.int64)), dict(ids=meta(5, 3, dtype=I32)), dict(w=meta(5, 2, dtype=BF16)), dict(w=meta(5, 3)),
        dict(ids=meta(4, 2, dtype=I32), w=meta(4, 2)), dict(X=meta(5, 400, dtype=BF16)[:, ::2]), dict(X=meta(10, 200, dtype=BF16)[::2]),
        dict(out=meta(10, 200, dtype=BF16)[::2]), dict(ids=meta(2, 5, dtype=I32).t()), dict(w=meta(2, 5).t()),
        dict(ws=meta(8192, dtype=U8)[::2]),
        dict(gu=meta(3, size - 16, dtype=U8)), dict(dn=meta(3, size, dtype=torch.int8)), dict(gus=size + 16), dict(gu=meta(2, size, dtype=U8)),
        dict(gu=meta(3, size, dtype=U8)[:, ::2]),
    ]:
        refused(calls, lambda: f(**over))
    f(), f(T=0), f(ws=meta(1024))
    assert [(a[3], a[4], a[5], a[6], a[11], a[12], a[14]) for _, a in calls] == [(5, 2, 3, FP8, 200, 48, 4096), (0, 2, 3, FP8, 200, 48, 4096),
                                                                              (5, 2, 3, FP8, 200, 48, 4096)]


# ------------------------------------------------------------------------------------------- norm
D = L.norm_desc()


@pytest.mark.parametrize("quant", [False, True])
def test_norm(calls, quant):
    def f(M=5, H=64, **over):
        a = dict(X=meta(M, H, dtype=BF16), res=meta(M, H), w=meta(H), ro=meta(M, H), Y=meta(M, H, dtype=BF16), pw=None, gate=None)
        a.update(over)
        if quant:
            L.w4a8_norm_residual_quant(a["X"], a["res"], D, a["w"], a["ro"], FP8, *codes(FP8, M, H), post_w=a["pw"], gate=a["gate"])
        else:
            L.w4a8_norm_residual(a["X"], a["res"], D, a["w"], a["ro"], a["Y"], post_w=a["pw"], gate=a["gate"])

    for over in [
        dict(w=meta(63)), dict(w=meta(64, dtype=BF16)), dict(w=meta(128)[::2]), dict(pw=meta(65)), dict(pw=meta(64, dtype=F16)),
        dict(res=meta(4, 64)), dict(res=meta(5, 64, dtype=torch.int32)), dict(ro=meta(5, 64, dtype=BF16)), dict(ro=meta(5, 65)),
        dict(gate=meta(5, 64)), dict(gate=meta(4, 64, dtype=BF16)), dict(gate=meta(5, 63, dtype=BF16)), dict(gate=meta(64, dtype=BF16)),
        dict(X=meta(64, 5, dtype=BF16).t()), dict(X=meta(5, 64, dtype=BF16, ld=63)), dict(res=meta(1, 64).expand(5, 64)),
        dict(ro=meta(1, 64).expand(5, 64)),
    ] + ([] if quant else [dict(Y=meta(5, 64)), dict(Y=meta(4, 64, dtype=BF16)), dict(Y=meta(1, 64, dtype=BF16).expand(5, 64))]):
        refused(calls, lambda: f(**over))
    f(), f(X=meta(5, 64, dtype=BF16, ld=80)), f(gate=meta(1, 64, dtype=BF16)), f(gate=meta(5, 64, dtype=BF16, ld=72)), f(M=0)
    f(gate=meta(1, 64, dtype=BF16).expand(1, 64), M=1), f(res=None, ro=None), f(res=None)
    assert [(a[2], a[7], a[11]) for _, a in calls] == [(64, 0, 5), (80, 0, 5), (64, 0, 5), (64, 72, 5), (64, 0, 0), (64, 0, 1), (64, 0, 5), (64, 0, 5)]
    res = meta(5, 64)
    calls.clear()
    f(res=res, ro=res)
    assert calls[0][1][14] == 64


@pytest.mark.parametrize("q,s", [
    (meta(5, 64, dtype=U8), meta(5)), (meta(5, 64, dtype=torch.int8), meta(4)), (meta(5, 63, dtype=torch.int8), meta(5)),
    (meta(5, 64, dtype=torch.int8), meta(5, dtype=BF16)), (meta(10, 64, dtype=torch.int8)[::2], meta(5)), codes(FP8, 5, 64),
])
def test_norm_int8_outputs(calls, q, s):
    refused(calls, lambda: L.w4a8_norm_residual_quant(meta(5, 64, dtype=BF16), None, D, meta(64), None, I8, q, s), "int8")


def test_norm_quantized_formats(calls):
    X, w = meta(5, 64, dtype=BF16), meta(64)
    refused(calls, lambda: L.w4a8_norm_residual_quant(X, None, D, w, None, FP4, *codes(FP8, 5, 64)), "codes and scales")
    refused(calls, lambda: L.w4a8_norm_residual_quant(X, None, D, w, None, 3, *codes(FP8, 5, 64)), "fmt")
    L.w4a8_norm_residual_quant(X, None, D, w, None, I8, meta(5, 64, dtype=torch.int8), meta(5))
    L.w4a8_norm_residual_quant(X, None, D, w, None, FP4, *codes(FP4, 5, 64))
    assert [a[15] for _, a in calls] == [I8, FP4]


# ------------------------------------------------------------------------------------------- tensors of the host
def host_calls():
    q, s = L.mx_empty(FP8, 5, 64, "cpu")
    X, w, off, B = torch.zeros(5, 64, dtype=BF16), torch.ones(64), torch.zeros(3, dtype=I32), torch.zeros(2, 4096, dtype=U8)
    moe = (q, s, FP8, None, 1, off, 2, B, 4096, 64)
    return [lambda: L.w4a8_mx_quant(X, FP8, q, s), lambda: L.w4a8_mx_dequant(q, s, FP8, X), lambda: L.w4a8_mx_pack(X, B[0]),
            lambda: L.w4a8_mx_pack_codes(q[:, :32].contiguous(), s[:, :2].contiguous(), B[0]),
            lambda: L.w4a8_mx_unpack_codes(B[0], 5, 64, *L.mx_empty(FP4, 5, 64, "cpu")),
            lambda: L.w4a8_mx_gemm(q, s, FP8, B[0], 64, 64, X), lambda: L.w4a8_moe_gemm_mx(*moe, X),
            lambda: L.w4a8_moe_gemm_silu_mx(*moe, X[:, :16].contiguous()),
            lambda: L.w4a8_moe_gemm_silu_mx_quant(*moe, 16, FP8, *L.mx_empty(FP8, 5, 16, "cpu")),
            lambda: L.w4a8_moe_forward_mx(X, torch.zeros(5, 1, dtype=I32), torch.ones(5, 1), 2, FP8, B, 4096, B, 4096, 16,
                                          torch.zeros(1 << 16, dtype=U8), X.clone()),
            lambda: L.w4a8_norm_residual(X, X.clone(), D, w, None, X.clone()),
            lambda: L.w4a8_norm_residual_quant(X, None, D, w, None, FP8, q, s)]


@pytest.mark.parametrize("i", range(12))
def test_tensors_of_the_host(i):
    with pytest.raises(ValueError, match="device"):
        host_calls()[i]()
