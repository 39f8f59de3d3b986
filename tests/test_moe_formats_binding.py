"""Argument checks of the Python calls of the router and of the 8-bit and 16-bit grouped products.  Every refusal comes before
the library is called, so these run without a GPU: the calls see meta tensors (shapes, strides and types without storage) as
tensors of the current device, and the library is replaced by one that records its arguments."""
import pytest
import torch

import moe_token_int8_amd as L

META = torch.empty(0, device="meta").get_device()


class Recorder:
    """Stands for the library: every entry point returns OK and notes its arguments."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def entry(*args):
            self.calls.append((name, args))
            return L.W4A8_OK
        return entry


@pytest.fixture
def calls(monkeypatch):
    t = L._Torch()
    t.device, t.initialized, t.raw_stream = lambda: META, lambda: True, lambda dev: 0
    rec = Recorder()
    L.lib()                                                     # the real one stays loaded for the sizes of blobs
    monkeypatch.setattr(L, "_torch_of_calls", t)
    monkeypatch.setattr(L, "_require_current", lambda *a, **k: None)
    monkeypatch.setattr(L, "_stream", lambda s: 0)
    monkeypatch.setattr(L, "_packed_size", lambda d, real=L.lib(): int(real.w4a8_packed_size(d)))
    monkeypatch.setattr(L, "lib", lambda: rec)
    return rec.calls


def meta(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype, device="meta")


def route(x, k=4, bias=None):
    T, E = x.shape
    L.w4a8_moe_route(x, L.route_desc(E, k), meta(T, k, dtype=torch.int32), meta(T, k), bias=bias)


# ------------------------------------------------------------------------------------------- router
@pytest.mark.parametrize("stride", [0, 1, 63])
def test_route_rows_that_overlap(calls, stride):
    """A row stride below E would have the kernel read E elements of every row from storage that ends before them."""
    with pytest.raises(ValueError, match="overlap"):
        route(torch.empty_strided((5, 64), (stride, 1), device="meta"))
    assert not calls


def test_route_expanded_rows(calls):
    with pytest.raises(ValueError, match="overlap"):
        route(meta(64).expand(5, 64))
    assert not calls


@pytest.mark.parametrize("T,stride,ldl", [(1, 0, 64), (1, 7, 64), (1, 640, 64), (0, 0, 64), (5, 64, 64), (5, 101, 101)])
def test_route_row_stride(calls, T, stride, ldl):
    """The stride of a single row says nothing; any other is handed on."""
    route(torch.empty_strided((T, 64), (stride, 1), device="meta"))
    (name, args), = calls
    assert name == "w4a8_moe_route" and args[2:4] == (T, ldl)


# ------------------------------------------------------------------------------------------- W8A8 product
I32, BF16, F16 = torch.int32, torch.bfloat16, torch.float16


def w8(rows=6, K=256, N=48, E=3, k=2, gather=True, off=None, blob=None, stride=None, Y=None, out=L.W4A8_OUT_BF16):
    d = L.desc(K, N, K, False, bits=8)
    size = L._packed_size(d)
    src = 4 if gather is not None else rows
    g = meta(rows, dtype=I32) if gather is True else gather
    L.w4a8_moe_gemm_w8a8(meta(src, K, dtype=torch.int8), meta(src), g, k, meta(E + 1, dtype=I32) if off is None else off, E, rows,
                         meta(E, size, dtype=torch.uint8) if blob is None else blob, size if stride is None else stride, d,
                         meta(rows, N, dtype=BF16) if Y is None else Y, out)


@pytest.mark.parametrize("dtype,out", [
    (F16, L.W4A8_OUT_BF16),                                     # would be filled with bfloat16 bits
    (torch.int16, L.W4A8_OUT_BF16), (torch.int32, L.W4A8_OUT_F32),
    (torch.uint8, L.W4A8_OUT_BF16), (torch.int8, L.W4A8_OUT_BF16),      # would be written to twice their length
    (torch.float64, L.W4A8_OUT_BF16), (torch.float32, L.W4A8_OUT_BF16), (BF16, L.W4A8_OUT_F32), (F16, L.W4A8_F16),
])
def test_w8_output_type(calls, dtype, out):
    with pytest.raises(ValueError, match="out_dtype"):
        w8(Y=meta(6, 48, dtype=dtype), out=out)
    assert not calls


def test_w8_output_types_that_fit(calls):
    w8()
    w8(Y=meta(6, 48), out=L.W4A8_OUT_F32)
    w8(Y=meta(7, 48, dtype=BF16))                               # longer than the rows of the call
    assert [c[0] for c in calls] == ["w4a8_moe_gemm_w8a8"] * 3


# ------------------------------------------------------------------------------------------- 16-bit products
def w16(X=None, W=None, Y=None, rows=6, K=64, N=48, E=3, k=2, gather=True, off=None, silu=False):
    src = 4 if gather is not None else rows
    f = L.w4a8_moe_gemm_silu_w16a16 if silu else L.w4a8_moe_gemm_w16a16
    f(meta(src, K, dtype=BF16) if X is None else X, meta(rows, dtype=I32) if gather is True else gather, k,
      meta(E + 1, dtype=I32) if off is None else off, meta(E, (2 if silu else 1) * N, K, dtype=BF16) if W is None else W,
      meta(rows, N, dtype=BF16) if Y is None else Y)


PRODUCTS = [pytest.param(w8, id="w8a8"), pytest.param(w16, id="w16a16"),
            pytest.param(lambda **a: w16(silu=True, **a), id="silu_w16a16")]


@pytest.mark.parametrize("call", PRODUCTS)
@pytest.mark.parametrize("bad", [dict(gather=meta(6, 2, dtype=I32)[:, 0]), dict(gather=meta(12, dtype=I32)[::2]),
                                 dict(gather=meta(1, dtype=I32).expand(6)), dict(gather=meta(5, dtype=I32)),
                                 dict(off=meta(4, 2, dtype=I32)[:, 1]), dict(off=meta(8, dtype=I32)[::2]),
                                 dict(off=meta(1, dtype=I32).expand(4)), dict(off=meta(5, dtype=I32)),
                                 dict(off=meta(3, dtype=I32))])
def test_index_arrays_are_dense(calls, call, bad):
    """The kernels read them one entry after another: a column, every other entry or an expanded one would be read as if its
    storage were dense, and past its end."""
    with pytest.raises(ValueError, match="contiguous"):
        call(**bad)
    assert not calls


@pytest.mark.parametrize("call", PRODUCTS)
def test_index_arrays_that_fit(calls, call):
    call()
    call(gather=None)
    call(gather=meta(9, dtype=I32))                             # longer than the rows of the call
    call(gather=meta(9, dtype=I32)[2:8], off=meta(9, dtype=I32)[5:])
    assert len(calls) == 4


# ------------------------------------------------------------------------------------------- packed weights
BLOB = L.w4a8_packed_size(L.desc(256, 48, 256, False, bits=8))


def layer8(blob=None, stride=None, down=False, E=3, H=256, I=128, T=4, k=2):
    """A layer whose gate/up (or down) weights are the given ones."""
    gu, dn = L.desc(H, 2 * I, H, False, bits=8), L.desc(I, H, I, False, bits=8)
    w = [[meta(E, L._packed_size(d), dtype=torch.uint8), L._packed_size(d)] for d in (gu, dn)]
    if blob is not None:
        w[down][0] = blob(w[down][1])
    if stride is not None:
        w[down][1] = stride(w[down][1])
    L.w4a8_moe_forward_w8a8(meta(T, H, dtype=BF16), meta(T, k, dtype=I32), meta(T, k), E, w[0][0], w[0][1], gu, w[1][0], w[1][1], dn,
                            meta(1 << 20, dtype=torch.uint8), meta(T, H, dtype=BF16))


def product8(blob=None, stride=None):
    w8(blob=None if blob is None else blob(BLOB), stride=None if stride is None else stride(BLOB))


PACKED = [pytest.param(product8, id="product"), pytest.param(layer8, id="layer_gate_up"),
          pytest.param(lambda **a: layer8(down=True, **a), id="layer_down")]


@pytest.mark.parametrize("call", PACKED)
@pytest.mark.parametrize("bad", [
    dict(blob=lambda n: meta(1, n, dtype=torch.uint8).expand(3, n)),            # one blob seen as three
    dict(blob=lambda n: meta(3, 2 * n, dtype=torch.uint8)[:, :n]), dict(blob=lambda n: meta(n, 3, dtype=torch.uint8).t()),
    dict(blob=lambda n: meta(3 * n - 1, dtype=torch.uint8)), dict(stride=lambda n: n + 16),
    dict(stride=lambda n: -16), dict(stride=lambda n: -n),                      # a size_t past every check of the library
])
def test_packed_weights_that_do_not_lie_as_said(calls, call, bad):
    with pytest.raises(ValueError, match="packed weights"):
        call(**bad)
    assert not calls


@pytest.mark.parametrize("call", PACKED)
def test_packed_weights_that_fit(calls, call):
    call()
    call(blob=lambda n: meta(3, n + 256, dtype=torch.uint8), stride=lambda n: n + 256)
    call(blob=lambda n: meta(3 * n + 5, dtype=torch.uint8))
    assert len(calls) == 3


# ------------------------------------------------------------------------------------------- sizes past 32 bits
BIG = 1 << 32                                                   # each of these would arrive as a small number


def strided(rows, width, stride, dtype=BF16):
    return torch.empty_strided((rows, width), (stride, 1), dtype=dtype, device="meta")


def layer16(T=4, k=2, E=3, H=64, I=24):
    L.w4a8_moe_forward_w16a16(meta(T, H, dtype=BF16), meta(T, k, dtype=I32), meta(T, k), meta(E, 2 * I, H, dtype=BF16),
                              meta(E, H, I, dtype=BF16), meta(1 << 20, dtype=torch.uint8), meta(T, H, dtype=BF16))


@pytest.mark.parametrize("call", [
    lambda: route(strided(5, 64, BIG + 64, torch.float32)), lambda: route(meta(BIG + 1, 4), k=1),
    lambda: w8(k=BIG + 2), lambda: w8(rows=BIG + 6), lambda: w8(E=BIG + 3, blob=meta(1 << 45, dtype=torch.uint8)),
    lambda: w16(X=strided(4, 64, BIG + 64)), lambda: w16(Y=strided(6, 48, BIG + 48)), lambda: w16(k=BIG + 2),
    lambda: w16(W=torch.empty_strided((3, 48, 64), (48 * (BIG + 64), BIG + 64, 1), dtype=BF16, device="meta")),
    lambda: w16(X=meta(BIG + 4, 64, dtype=BF16)), lambda: w16(rows=BIG + 6),
    lambda: w16(silu=True, Y=strided(6, 48, BIG + 48)), lambda: layer8(T=BIG + 4), lambda: layer8(E=BIG + 3),
    lambda: layer16(T=BIG + 4), lambda: layer16(E=BIG + 3), lambda: layer16(I=BIG + 24),
    lambda: L.w4a8_moe_w16a16_workspace_size(BIG + 4, 2, 64, 24, 3),
])
def test_sizes_past_32_bits(calls, call):
    with pytest.raises(ValueError, match="32 bits"):
        call()
    assert not calls


def test_largest_strides(calls):
    route(strided(5, 64, (1 << 31) - 1, torch.float32))
    w16(X=strided(4, 64, (1 << 31) - 8), Y=strided(6, 48, (1 << 31) - 1))
    layer16()
    layer8()
    assert len(calls) == 4


# ------------------------------------------------------------------------------------------- single columns
def test_single_columns_with_any_stride(calls):
    """One expert, one output column: the step to a next one says nothing, as in torch's own idea of contiguous."""
    route(meta(1, 5).t(), k=1)
    assert calls[-1][1][2:4] == (5, 1)
    w16(N=1, Y=meta(1, 6, dtype=BF16).t())
    assert calls[-1][1][14:16] == (0, 1)
    w16(N=1, silu=True, Y=torch.empty_strided((6, 1), (9, 7), dtype=BF16, device="meta"))
    assert calls[-1][1][14:16] == (0, 9)


@pytest.mark.parametrize("call", [lambda: route(meta(64, 5).t()), lambda: w16(Y=meta(48, 6, dtype=BF16).t()),
                                  lambda: w16(X=meta(64, 4, dtype=BF16).t())])
def test_columns_that_are_not_next_to_each_other(calls, call):
    with pytest.raises(ValueError, match="contiguous"):
        call()
    assert not calls


# ------------------------------------------------------------------------------------------- shapes of a layer
def shaped16(X=(4, 64), ids=(4, 2), w=(4, 2), out=None, E=3, H=64, I=24):
    L.w4a8_moe_forward_w16a16(meta(*X, dtype=BF16), meta(*ids, dtype=I32), meta(*w), meta(E, 2 * I, H, dtype=BF16),
                              meta(E, H, I, dtype=BF16), meta(1 << 20, dtype=torch.uint8), meta(*(out or X), dtype=BF16))


def shaped8(X=(4, 256), ids=(4, 2), w=(4, 2), out=None, E=3, H=256, I=128):
    gu, dn = L.desc(H, 2 * I, H, False, bits=8), L.desc(I, H, I, False, bits=8)
    L.w4a8_moe_forward_w8a8(meta(*X, dtype=BF16), meta(*ids, dtype=I32), meta(*w), E, meta(E, L._packed_size(gu), dtype=torch.uint8),
                            L._packed_size(gu), gu, meta(E, L._packed_size(dn), dtype=torch.uint8), L._packed_size(dn), dn,
                            meta(1 << 20, dtype=torch.uint8), meta(*(out or X), dtype=BF16))


@pytest.mark.parametrize("call,H", [(shaped16, 64), (shaped8, 256)])
def test_layers_take_matrices(calls, call, H):
    """A third dimension behind [T, H] or [T, k] would be read as more rows of them."""
    call()
    for bad in (dict(X=(4, H, 3)), dict(X=(4, H, 1)), dict(ids=(4, 2, 2), w=(4, 2, 2)), dict(ids=(4,), w=(4,)), dict(X=(4,)),
                dict(out=(5, H)), dict(ids=(4, 3)), dict(ids=(5, 2), w=(5, 2)), dict(X=(4, H + 8))):
        with pytest.raises(ValueError):
            call(**bad)
    assert len(calls) == 1
