"""MXFP8 products drop nothing, whatever the output, the kernel and the call: the matrix unit by itself would lose what lies 14 bits
below the largest of 8 neighbouring products.  Sizes run every kernel of every product (tests/test_mx_dispatch.py)."""
import numpy as np
import pytest
import torch

import moe_token_int8_amd as L
from mx_cases import DEV, FP4, FP8, half_step, quant_bound, silu_bound
from test_gpu_mx_kernels import SENTINEL, SIZES, Problem, layer_inputs, worst

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.lib()


class Small:
    """Rows of 448, -448 and 2^-6 in one group of 8 (a different one for each row) and zeros, weights of 1: sums are 2^-6.  Gate weights are 1
    at even places of each group and 0 at odd ones: with 448 at an even place and the others at odd ones a gate is 448 (silu is itself), and h = 7."""

    def __init__(self, counts, K, width, pair):
        self.E, self.rows = len(counts), sum(counts)
        x = torch.zeros(self.rows, K, device=DEV)
        r = torch.arange(self.rows, device=DEV)
        first = r % (K // 8) * 8
        x[r, first + 2 * (r % 4)], x[r, first + 2 * (r // 4 % 4) + 1], x[r, first + 2 * ((r // 4 + 1) % 4) + 1] = 448.0, -448.0, 2.0 ** -6
        self.q, self.s = L.mx_empty(FP8, self.rows, K, DEV)
        L.w4a8_mx_quant(x, FP8, self.q, self.s)
        w = torch.ones(width, K, device=DEV)
        if pair:
            w[:width // 2, 1::2] = 0
        self.blobs = torch.empty(self.E, L.w4a8_mx_packed_size(K, width), dtype=torch.uint8, device=DEV)
        for b in self.blobs:
            L.w4a8_mx_pack(w, b)
        self.off = torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).to(DEV)
        self.args = (self.q, self.s, FP8, None, 1, self.off, self.E, self.blobs, self.blobs.shape[1], K)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("counts,K,N", SIZES["dense"])
def test_small_parts_dense(counts, K, N, out):
    p = Small(counts, K, N, False)
    Y = torch.empty(p.rows, N, dtype=out, device=DEV)
    L.w4a8_mx_gemm(p.q, p.s, FP8, p.blobs[0], K, N, Y)
    assert (Y == 2.0 ** -6).all()


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("counts,K,N", SIZES["moe"])
def test_small_parts_by_expert(counts, K, N, out):
    p = Small(counts, K, N, False)
    Y = torch.empty(p.rows, N, dtype=out, device=DEV)
    L.w4a8_moe_gemm_mx(*p.args, Y)
    assert (Y == 2.0 ** -6).all()


@pytest.mark.parametrize("counts,K,I", SIZES["silu"])
def test_small_parts_of_gate_up(counts, K, I):
    p = Small(counts, K, 2 * I, True)
    for out in (torch.bfloat16, torch.float16):
        H = torch.empty(p.rows, I, dtype=out, device=DEV)
        L.w4a8_moe_gemm_silu_mx(*p.args, H)
        assert (H == 7).all()
    for fmt in (FP4, FP8):
        q, s = L.mx_empty(fmt, p.rows, I, DEV)
        L.w4a8_moe_gemm_silu_mx_quant(*p.args, I, fmt, q, s)
        h = torch.empty(p.rows, I, device=DEV)
        L.w4a8_mx_dequant(q, s, fmt, h)
        assert (h == (6 if fmt == FP4 else 7)).all()            # E2M1 blocks of 7 have the scale 1 and saturate


@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("counts,K,N", SIZES["moe"])
def test_16_bits_are_the_rounded_float32(counts, K, N, fmt):
    p = Problem(counts, K, N, fmt, 5)
    Y = torch.full((p.rows, N), SENTINEL, device=DEV)
    L.w4a8_moe_gemm_mx(*p.moe(), Y)
    for out in (torch.bfloat16, torch.float16):
        Z = torch.full((p.rows, N), SENTINEL, dtype=out, device=DEV)
        L.w4a8_moe_gemm_mx(*p.moe(), Z)
        assert torch.equal(Z, Y.to(out))


@pytest.mark.parametrize("gathered", [False, True])
@pytest.mark.parametrize("counts,K,I", SIZES["silu"])
def test_gate_up_to_the_bound_of_exact_products(counts, K, I, gathered):
    """The sums' bound is that of MXFP4 activations: no part of a product is lost."""
    p = Problem(counts, K, 2 * I, FP8, 25, gathered)
    h, b = silu_bound(K, p.y, p.mag, FP4)
    H = torch.full((p.rows, I), SENTINEL, dtype=torch.bfloat16, device=DEV)
    L.w4a8_moe_gemm_silu_mx(*p.moe(), H)
    assert worst(H, h, b + half_step(torch.bfloat16, np.abs(h) + b)) <= 0
    for fmt in (FP4, FP8):
        q, s = L.mx_empty(fmt, p.rows, I, DEV)
        L.w4a8_moe_gemm_silu_mx_quant(*p.moe(), I, fmt, q, s)
        got = torch.empty(p.rows, I, device=DEV)
        L.w4a8_mx_dequant(q, s, fmt, got)
        assert worst(got, h, quant_bound(h, b, fmt)) <= 0


@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("T,E", [(1, 8), (37, 64), (300, 8), (3000, 16)])
def test_layer_has_the_bits_of_its_steps(T, E, fmt):
    """With one expert a token the weighted sum is one product: the layer is w4a8_moe_gemm_mx in float32, times the weight."""
    H, I = 520, 240
    GU, DN, _, x, logits = layer_inputs(T, 1, E, H, I, fmt, T)
    ids, w = logits.argmax(1).to(torch.int32)[:, None].contiguous(), torch.rand(T, 1, device=DEV)
    q, s = L.mx_empty(fmt, T, H, DEV)
    L.w4a8_mx_quant(x, fmt, q, s)
    rows, inv, off = (torch.empty(n, dtype=torch.int32, device=DEV) for n in (T, (T, 1), E + 1))
    L.w4a8_moe_align(ids, E, rows, off, inv)
    hq, hs = L.mx_empty(fmt, T, I, DEV)
    L.w4a8_moe_gemm_silu_mx_quant(q, s, fmt, rows, 1, off, E, GU, GU.shape[1], H, I, fmt, hq, hs)
    y = torch.empty(T, H, device=DEV)
    L.w4a8_moe_gemm_mx(hq, hs, fmt, None, 1, off, E, DN, DN.shape[1], I, y)
    want = (w * y[inv[:, 0].long()]).to(torch.bfloat16)
    for ws in (L.w4a8_moe_mx_workspace_size(T, 1, H, I, E, fmt), L.w4a8_moe_mx_workspace_size(T, 1, H // 2, I, E, fmt) + T * H):
        out = torch.full((T, H), SENTINEL, dtype=torch.bfloat16, device=DEV)
        L.w4a8_moe_forward_mx(x, ids, w, E, fmt, GU, GU.shape[1], DN, DN.shape[1], I, torch.empty(ws, dtype=torch.uint8, device=DEV), out)
        assert torch.equal(out, want)
