"""Sizes past 32 bits in the Python calls of the norm around a block: refused before the library is called, whatever the tensors' strides."""
import pytest

import moe_token_int8_amd as L
from test_mx_binding import BF16, calls, meta, refused  # noqa: F401

FAR = [(1 << 32) + 1, 1 << 31]


@pytest.mark.parametrize("M", FAR)
def test_many_rows(calls, M):  # noqa: F811
    X, w, d = meta(M, 1, dtype=BF16), meta(1), L.norm_desc()
    refused(calls, lambda: L.w4a8_norm_residual(X, None, d, w, None, meta(M, 1, dtype=BF16)))
    refused(calls, lambda: L.w4a8_norm_residual(X, meta(M, 1), d, None, meta(M, 1), None))
    refused(calls, lambda: L.w4a8_norm_residual(X, meta(M, 1), d, w, None, meta(M, 1, dtype=BF16), gate=meta(1, 1, dtype=BF16)))
    refused(calls, lambda: L.w4a8_norm_residual_quant(X, None, d, w, None, L.W4A8_MX_FP8, *L.mx_empty(L.W4A8_MX_FP8, M, 1, "meta")))
    refused(calls, lambda: L.w4a8_norm_residual(meta(M, 2, dtype=BF16)[:, :1], None, d, w, None, meta(M, 1, dtype=BF16)))


@pytest.mark.parametrize("H", FAR)
def test_wide_rows(calls, H):  # noqa: F811
    X, d = meta(1, H, dtype=BF16), L.norm_desc()
    refused(calls, lambda: L.w4a8_norm_residual(X, None, d, meta(H), None, meta(1, H, dtype=BF16)))
    refused(calls, lambda: L.w4a8_norm_residual(X, meta(1, H), d, None, meta(1, H), None))
    X = meta(0, H, dtype=BF16)
    refused(calls, lambda: L.w4a8_norm_residual(X, None, d, meta(H), None, X))
