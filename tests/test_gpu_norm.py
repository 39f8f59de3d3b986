"""The norm around a block against float64, and its quantized forms against the separate calls, bit for bit."""
import numpy as np
import pytest
import torch

import moe_token_int8_amd as L

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.lib()


TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def inputs(seed, M, H, x, res, post, gate):
    g = torch.Generator().manual_seed(seed)
    return dict(X=torch.randn(M, H, generator=g).to(TYPES[x]), r=(torch.randn(M, H, generator=g) * 2).to(TYPES[res]),
                w=1 + 0.2 * torch.randn(H, generator=g), p=1 + 0.2 * torch.randn(H, generator=g) if post else None,
                gate=None if not gate else torch.randn(M if gate == "token" else 1, H, generator=g).to(TYPES[x]))


def step(dtype, y):
    e = 2.0 ** -25 if dtype == torch.float16 else 0.0
    return y.abs() * (torch.finfo(dtype).eps / 2) + e


def check(c, alpha=0.5, eps=1e-6, eps_post=1e-5, got_r=None, got_h=None):
    """Bounds.  A float32 sum of H squares of one sign is within (H / 512 + 16) 2^-23 of its value, relatively (each lane adds at most
    H / 512 * 8 / 8 ... <= H / 64 terms one after another, then 6 + 16 partial sums): with the division, the square root and the
    reciprocal the factor is within q = (H / 64 + 32) 2^-24.  u = X rs p: 2 more roundings, gate 1: (q + 3 2^-24) |u|.  r' = one
    fma and the rounding to its type.  h: from r' as stored, (q + 2 2^-24) |h| and the rounding to its type."""
    H = c["X"].shape[1]
    q = (H / 64 + 32) * 2.0 ** -24
    u = c["X"].double()
    eu = torch.zeros_like(u)
    if c["p"] is not None:
        u = u / torch.sqrt(u.square().mean(1, keepdim=True) + eps_post) * c["p"].double()
        eu = (q + 2 * 2.0 ** -24) * u.abs()
    if c["gate"] is not None:
        u = u * c["gate"].double()
        eu = eu * c["gate"].double().abs() + 2.0 ** -24 * u.abs() * 1.01
    r = (c["r"].double() if c["r"] is not None else 0.0) + alpha * u
    er = alpha * eu * 1.01 + 2.0 ** -24 * r.abs() * 1.01
    rt = got_r.dtype
    assert ((got_r.cpu().double() - r).abs() <= er + step(rt, r.abs() + er) + 1e-37).all()
    if got_h is not None:
        k = got_r.cpu().double()
        h = k / torch.sqrt(k.square().mean(1, keepdim=True) + eps) * c["w"].double()
        eh = (q + 2 * 2.0 ** -24) * h.abs()
        assert ((got_h.cpu().double() - h).abs() <= eh + step(got_h.dtype, h.abs() + eh) + 1e-37).all()


def run(c, alpha=0.5, with_y=True):
    t = {n: None if v is None else v.to(DEV) for n, v in c.items()}
    like = t["r"] if t["r"] is not None else t["X"]
    out = torch.full_like(like, 7.0)
    Y = torch.full_like(t["X"], 7.0) if with_y else None
    L.w4a8_norm_residual(t["X"], t["r"], L.norm_desc(1e-6, 1e-5, alpha), t["w"] if with_y else None, out, Y, post_w=t["p"], gate=t["gate"])
    return out, Y


@pytest.mark.parametrize("H", [1, 7, 32, 129, 512, 513, 1000, 2048, 4096, 7168, 8200, 16392, 40000])
@pytest.mark.parametrize("M", [1, 5])
def test_sizes(M, H):
    c = inputs(H, M, H, "bf16", "f32", True, "token")
    check(c, got_r=run(c)[0], got_h=run(c)[1])


@pytest.mark.parametrize("x", list(TYPES))
@pytest.mark.parametrize("res", list(TYPES))
@pytest.mark.parametrize("post,gate", [(False, ""), (True, "channel"), (False, "token"), (True, "token")])
def test_types_and_parts(x, res, post, gate):
    for M, H in ((3, 300), (130, 1024), (6, 4104)):
        c = inputs(M, M, H, x, res, post, gate)
        r, h = run(c)
        check(c, got_r=r, got_h=h)
        assert torch.equal(run(c, with_y=False)[0], r)


@pytest.mark.parametrize("H", [64, 640, 5000])
def test_norm_alone(H):
    """No residual: h is the RMS norm of X, which is stored unchanged."""
    c = inputs(1, 9, H, "bf16", "bf16", False, "")
    c["r"] = None
    r, h = run(c, alpha=1.0)
    assert torch.equal(r.cpu(), c["X"])
    check(c, alpha=1.0, got_r=r, got_h=h)
    X, w = c["X"].to(DEV), c["w"].to(DEV)
    Y = torch.empty_like(X)
    L.w4a8_norm_residual(X, None, L.norm_desc(1e-6), w, None, Y)
    assert torch.equal(Y, h)


def test_strides_and_in_place():
    c = inputs(5, 12, 515, "bf16", "bf16", True, "token")
    want_r, want_h = run(c)
    wide = {n: torch.full((12, 700), 7.0, dtype=torch.bfloat16, device=DEV) for n in ("X", "r", "gate", "Y")}
    view = {n: wide[n][:, 5:520] for n in wide}
    for n in ("X", "r", "gate"):
        view[n].copy_(c[n])
    L.w4a8_norm_residual(view["X"], view["r"], L.norm_desc(1e-6, 1e-5, 0.5), c["w"].to(DEV), view["r"], view["Y"], post_w=c["p"].to(DEV),
                         gate=view["gate"])
    assert torch.equal(view["r"], want_r) and torch.equal(view["Y"], want_h)
    for n in ("r", "Y"):
        assert (wide[n][:, :5] == 7.0).all() and (wide[n][:, 520:] == 7.0).all()


@pytest.mark.parametrize("fmt", [L.W4A8_MX_FP4, L.W4A8_MX_FP8, L.W4A8_QUANT_INT8])
@pytest.mark.parametrize("x", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,H", [(1, 32), (5, 464), (9, 512), (4, 4096), (3, 7168), (2, 16400)])
def test_quantized_is_the_separate_call(M, H, x, fmt):
    if fmt == L.W4A8_QUANT_INT8 and x != "bf16":
        pytest.skip("w4a8_quant_act takes bfloat16")
    c = inputs(M + H, M, H, x, "f32", True, "channel")
    r, h = run(c)
    t = {n: None if v is None else v.to(DEV) for n, v in c.items()}
    out = torch.zeros_like(r)
    if fmt == L.W4A8_QUANT_INT8:
        q, s = torch.full((M, H), 99, dtype=torch.int8, device=DEV), torch.full((M,), 9.0, device=DEV)
        q2, s2 = torch.zeros_like(q), torch.zeros_like(s)
        L.w4a8_quant_act(h, q2, s2)
    else:
        q, s = L.mx_empty(fmt, M, H, DEV)
        q.fill_(0xa5), s.fill_(0xa5)
        q2, s2 = L.mx_empty(fmt, M, H, DEV)
        L.w4a8_mx_quant(h, fmt, q2, s2)
    L.w4a8_norm_residual_quant(t["X"], t["r"], L.norm_desc(1e-6, 1e-5, 0.5), t["w"], out, fmt, q, s, post_w=t["p"], gate=t["gate"])
    assert torch.equal(out, r) and torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("H", [60, 600, 5000])
def test_zeros_and_nan_rows(H):
    c = inputs(2, 6, H, "bf16", "bf16", True, "")
    c["X"][1], c["r"][1] = 0, 0
    c["X"][2, H // 2] = float("nan")
    c["r"][3, 1] = float("inf")
    r, h = run(c)
    assert (r[1] == 0).all() and (h[1] == 0).all()
    assert torch.isnan(r[2]).all() and torch.isnan(h[2]).all()      # the norm of a row with a NaN
    assert torch.isinf(r[3, 1]) and torch.isnan(h[3, 1])
    good = [0, 4, 5]
    sub = {n: v[good] if n in ("X", "r") else v for n, v in c.items()}
    check(sub, got_r=r[good], got_h=h[good])
    for fmt in (L.W4A8_MX_FP4, L.W4A8_MX_FP8):
        q, s = L.mx_empty(fmt, 6, H, DEV)
        q2, s2 = L.mx_empty(fmt, 6, H, DEV)
        L.w4a8_mx_quant(h, fmt, q2, s2)
        L.w4a8_norm_residual_quant(c["X"].to(DEV), c["r"].to(DEV), L.norm_desc(1e-6, 1e-5, 0.5), c["w"].to(DEV), None, fmt, q, s,
                                   post_w=c["p"].to(DEV))
        assert torch.equal(q, q2) and torch.equal(s, s2)


def test_no_rows():
    X = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    L.w4a8_norm_residual(X, X, L.norm_desc(), torch.ones(64, device=DEV), X, X)


def test_rows_far_apart():
    """Row strides whose product with the rows passes 2^32 bytes, and rows as wide as the calls take."""
    for M, H, ld in ((300, 700, 1 << 23), (2, 65536, 1 << 30)):
        c = inputs(8, M, H, "bf16", "bf16", True, "token")
        want_r, want_h = run(c)
        d = {n: torch.empty(M * ld, dtype=torch.bfloat16, device=DEV).view(M, ld)[:, 3:3 + H] for n in ("X", "r", "gate", "Y")}
        for n in ("X", "r", "gate"):
            d[n].copy_(c[n])
        L.w4a8_norm_residual(d["X"], d["r"], L.norm_desc(1e-6, 1e-5, 0.5), c["w"].to(DEV), d["r"], d["Y"], post_w=c["p"].to(DEV),
                             gate=d["gate"])
        assert torch.equal(d["r"], want_r) and torch.equal(d["Y"], want_h)
        check(c, got_r=want_r, got_h=want_h)


@pytest.mark.parametrize("M", [4097, 70001])
def test_many_rows(M):
    """More rows than workgroups at a time: every row is the one that a call of it alone gives."""
    c = inputs(M, M, 96, "bf16", "f32", True, "channel")
    r, h = run(c)
    pick = [0, 1, 255, 256, 4095, M - 2, M - 1]
    part = dict(c, X=c["X"][pick], r=c["r"][pick])
    r2, h2 = run(part)
    assert torch.equal(r[pick], r2) and torch.equal(h[pick], h2)
    check(c, got_r=r, got_h=h)
