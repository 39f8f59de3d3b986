"""The norm around a block with per-token INT8 output, from every type of X, against the oracle's quantization of the h that the call without
quantization stores."""
import numpy as np
import pytest
import torch

import moe_token_int8_amd as L
import oracle as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.lib()


@pytest.mark.parametrize("x", list(TYPES))
@pytest.mark.parametrize("res", list(TYPES))
@pytest.mark.parametrize("M,H", [(1, 16), (5, 464), (9, 512), (7, 2048), (4, 4096), (3, 7168), (600, 4112), (2, 16400), (3, 40000)])
def test_codes_and_scales(M, H, x, res):
    g = torch.Generator(device=DEV).manual_seed(M + H)
    X = torch.randn(M, H, device=DEV, generator=g)
    X[:, H // 3] *= 30
    r = torch.randn(M, H, device=DEV, generator=g) * 2
    if M > 2:                                                    # a row of zeros, one with a NaN, one with an infinity
        X[0], r[0] = 0, 0
        X[1, H - 1] = float("nan")
        r[2, 0] = float("inf")
    X, r = X.to(TYPES[x]), r.to(TYPES[res])
    w, gate = 1 + 0.2 * torch.randn(H, device=DEV, generator=g), torch.randn(1, H, device=DEV, generator=g).to(TYPES[x])
    d = L.norm_desc(1e-6, 1e-5, 0.5)
    h, out, out2 = torch.empty_like(X), torch.empty_like(r), torch.empty_like(r)
    L.w4a8_norm_residual(X, r, d, w, out, h, gate=gate)
    q, s = torch.full((M, H), 99, dtype=torch.int8, device=DEV), torch.full((M,), 9.0, device=DEV)
    L.w4a8_norm_residual_quant(X, r, d, w, out2, L.W4A8_QUANT_INT8, q, s, gate=gate)
    want_q, want_s = O.quant_act(h.float().cpu().numpy())
    assert np.array_equal(q.cpu().numpy(), want_q)
    assert np.array_equal(s.cpu().numpy(), want_s, equal_nan=True)
    assert torch.equal(out.nan_to_num(7.0), out2.nan_to_num(7.0))
