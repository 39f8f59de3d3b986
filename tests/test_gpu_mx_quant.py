"""Quantization to the microscaled formats, its inverse and the packing of weights: bit for bit against the definition."""
import numpy as np
import pytest
import torch

import moe_token_int8_amd as L
from mx_cases import DEV, FP4, FP8, encode, pack, random_codes, same_codes, stored, unstored, up, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.lib()


def rows(seed, M, K, dtype):
    """Values over the whole range of exponents, blocks of zeros, ties of both formats, negative zeros."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g)
    x *= torch.exp2(torch.randint(-10, 11, (M, 1), generator=g).float())
    x[torch.rand(M, K, generator=g) < 0.05] = -0.0
    if M > 2 and K >= 64:
        x[0, :32] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0] * 4)      # ties of E2M1 at scale 1
        x[0, 32:64] = 0
        x[1, :32] = torch.tensor([17 / 16, 19 / 16, 448.0, 464.0, 480.0, 511.0, 2 ** -9, 3 * 2 ** -10] * 4)
        x[2, :32] *= 2.0 ** -12
    return x.to(dtype)


def quant(x, fmt):
    Xq, sx = L.mx_empty(fmt, x.shape[0], x.shape[1], DEV)
    Xq.fill_(0xa5), sx.fill_(0xa5)
    L.w4a8_mx_quant(x.to(DEV) if x.device.type == "cpu" else x, fmt, Xq, sx)
    return Xq, sx


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 32), (3, 31), (5, 129), (2, 512), (7, 1000), (33, 4096), (3, 7168)])
def test_quant_is_the_definition(M, K, fmt, dtype):
    x = rows(M * K + fmt, M, K, dtype)
    Xq, sx = quant(x, fmt)
    code, s = encode(x, fmt)
    assert np.array_equal(sx.cpu().numpy(), s)
    assert same_codes(Xq.cpu().numpy(), code, fmt)
    for out in (torch.bfloat16, torch.float32, torch.float16):
        Y = torch.full((M, K + 3), 7.0, dtype=out, device=DEV)
        L.w4a8_mx_dequant(Xq, sx, fmt, Y[:, :K])
        want = torch.from_numpy(values(code, s, fmt, K)).to(out)
        assert torch.equal(Y[:, :K].cpu(), want) and (Y[:, K:] == 7.0).all()


@pytest.mark.parametrize("fmt", [FP4, FP8])
def test_every_exponent(fmt):
    """Blocks whose largest value has each exponent of float32, subnormals included: the scale and the codes of the definition."""
    e = torch.arange(-149, 128).double()
    x = (torch.linspace(-1.999, 1.999, 32).double()[None, :] * torch.exp2(e)[:, None]).clamp(-3.4e38, 3.4e38).float()
    Xq, sx = quant(x, fmt)
    code, s = encode(x, fmt)
    assert np.array_equal(sx.cpu().numpy(), s)
    assert same_codes(Xq.cpu().numpy(), code, fmt)
    Y = torch.empty(len(x), 32, device=DEV)
    L.w4a8_mx_dequant(Xq, sx, fmt, Y)
    assert torch.equal(Y.cpu().double(), torch.from_numpy(values(code, s, fmt, 32)))


@pytest.mark.parametrize("fmt", [FP4, FP8])
def test_all_bfloat16_values(fmt):
    """Every finite bfloat16 as the second largest of a block whose largest is 1."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    v = bits[torch.isfinite(bits) & (bits.abs() <= 1)]
    x = torch.zeros(len(v), 32, dtype=torch.bfloat16)
    x[:, 5], x[:, 17] = 1.0, v
    Xq, sx = quant(x, fmt)
    code, s = encode(x, fmt)
    assert np.array_equal(sx.cpu().numpy(), s) and same_codes(Xq.cpu().numpy(), code, fmt)


@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_blocks_with_nan_or_inf(fmt, bad, dtype):
    x = rows(3, 4, 160, dtype)
    x[1, 37], x[3, 159] = bad, bad
    Xq, sx = quant(x, fmt)
    code, s = encode(x, fmt)
    assert s[1, 1] == 255 and s[3, 4] == 255 and (s == 255).sum() == 2
    assert np.array_equal(sx.cpu().numpy(), s) and same_codes(Xq.cpu().numpy(), code, fmt)
    Y = torch.zeros(4, 160, device=DEV)
    L.w4a8_mx_dequant(Xq, sx, fmt, Y)
    assert int(torch.isnan(Y).sum()) == 64 and torch.isnan(Y[1, 32:64]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_and_unaligned_rows(dtype):
    base = rows(9, 6, 301, dtype).to(DEV)
    x = base[1:, 3:290]                                             # rows that start at any element
    Xq, sx = quant(x, FP8)
    code, s = encode(x.cpu(), FP8)
    assert np.array_equal(sx.cpu().numpy(), s) and same_codes(Xq.cpu().numpy(), code, FP8)
    out = torch.full((6, 301), 7.0, dtype=dtype, device=DEV)
    L.w4a8_mx_dequant(Xq, sx, FP8, out[1:, 3:290])
    assert torch.equal(out[1:, 3:290].cpu().double(), torch.from_numpy(values(code, s, FP8, 287)).to(dtype).double())
    out[1:, 3:290] = 7.0
    assert (out == 7.0).all()


def test_no_rows():
    for fmt in (FP4, FP8):
        Xq, sx = L.mx_empty(fmt, 0, 64, DEV)
        L.w4a8_mx_quant(torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), fmt, Xq, sx)
        L.w4a8_mx_dequant(Xq, sx, fmt, torch.empty(0, 64, device=DEV))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("N,K", [(1, 1), (15, 33), (64, 128), (65, 200), (130, 512), (2, 1408)])
def test_pack(N, K, dtype):
    W = rows(N + K, N, K, dtype)
    blob = torch.full((L.w4a8_mx_packed_size(K, N),), 0xa5, dtype=torch.uint8, device=DEV)
    L.w4a8_mx_pack(W.to(DEV), blob)
    code, s = encode(W, FP4)
    want, got = pack(code, s, N, K), blob.cpu().numpy()
    end, base = up(N, 16) * up(K, 128) // 2, up(up(N, 16) * up(K, 128) // 2, 256)
    assert np.array_equal(got[:end], want[:end]) and np.array_equal(got[base:], want[base:])
    q, sq = L.mx_empty(FP4, N, K, DEV)
    L.w4a8_mx_unpack_codes(blob, N, K, q, sq)
    assert np.array_equal(unstored(q.cpu().numpy(), FP4), code) and np.array_equal(sq.cpu().numpy(), s)


def test_pack_experts_and_strided_weights():
    base = rows(4, 3 * 70, 300, torch.bfloat16).view(3, 70, 300).to(DEV)
    W = base[:, 1:60, 2:262]
    size = L.w4a8_mx_packed_size(260, 59)
    blobs = torch.full((3, size + 256), 0xa5, dtype=torch.uint8, device=DEV)
    L.w4a8_mx_pack(W, blobs)
    for e in range(3):
        one = torch.empty(size, dtype=torch.uint8, device=DEV)
        L.w4a8_mx_pack(W[e].contiguous(), one)
        q, s = L.mx_empty(FP4, 59, 260, DEV)
        q2, s2 = L.mx_empty(FP4, 59, 260, DEV)
        L.w4a8_mx_unpack_codes(one, 59, 260, q, s)
        L.w4a8_mx_unpack_codes(blobs[e], 59, 260, q2, s2)
        assert torch.equal(q, q2) and torch.equal(s, s2)
        assert (blobs[e, size:] == 0xa5).all()


@pytest.mark.parametrize("N,K", [(1, 32), (17, 96), (100, 1408)])
def test_pack_codes(N, K):
    """Existing codes, in rows of their own stride (a multiple of 16 bytes)."""
    code, s = random_codes(np.random.default_rng(N), N, K, FP4)
    q = torch.full((N, K // 2 + 48), 0xff, dtype=torch.uint8)
    q[:, : K // 2] = torch.from_numpy(np.ascontiguousarray(stored(code, FP4)[:, : K // 2]))
    sc = torch.full((N, K // 32 + 3), 0xff, dtype=torch.uint8)
    sc[:, : K // 32] = torch.from_numpy(np.ascontiguousarray(s[:, : K // 32]))
    blob = torch.zeros(L.w4a8_mx_packed_size(K, N), dtype=torch.uint8, device=DEV)
    # rows up to a multiple of 16 bytes
    stride = (K // 2 + 48) // 16 * 16
    q = q[:, :stride].contiguous().to(DEV)
    L.w4a8_mx_pack_codes(q[:, : K // 2], sc.to(DEV)[:, : K // 32], blob)
    assert np.array_equal(blob.cpu().numpy(), pack(code, s, N, K))


def test_quant_of_weights_then_pack_is_pack():
    W = rows(8, 50, 320, torch.bfloat16).to(DEV)
    q, s = quant(W, FP4)
    a = torch.zeros(L.w4a8_mx_packed_size(320, 50), dtype=torch.uint8, device=DEV)
    b = torch.zeros_like(a)
    L.w4a8_mx_pack(W, a)
    L.w4a8_mx_pack_codes(q[:, :160], s[:, :10], b)
    assert torch.equal(a, b)
