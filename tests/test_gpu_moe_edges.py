"""Inputs of the router and of the grouped products on which forms of the same operator once disagreed, or left their
definition: each is checked in every form that takes it."""
import numpy as np
import pytest
import torch

import moe_token_int8_amd as L
import oracle as O
from gpu_cases import check_moe
from moe_formats_cases import DEV, assert_within, half_step, offsets_of, route_reference, w8_device, w8_inputs, w8_reference
from test_gpu_moe_formats import COUNTS, run_w8
from test_gpu_moe_layers import routed, run8, weights8
from test_gpu_moe_route import call, check
from test_gpu_moe_tiles import LARGE

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.lib()


# ------------------------------------------------------------------------------------------- router
# experts, groups, groups kept: 16 lanes a token, 64 lanes, and more groups than lanes
FORMS = [(64, 1, 1), (64, 4, 2), (1000, 1, 1), (1024, 2, 1), (200, 100, 30)]


@pytest.mark.parametrize("E,groups,keep", FORMS)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nan_bias_of_a_masked_expert(E, groups, keep, score):
    """An expert with a -Inf logit is never chosen, whatever its bias; a NaN bias of one that could be leaves no order."""
    print("nan bias", E, groups, keep, score, flush=True)
    x = torch.randn(5, E, generator=torch.Generator().manual_seed(E))
    x[0, 5] = -INF
    x[1] = -INF                                                 # a padded token
    x[2, E // 2:] = -INF
    x[2, 5] = -INF
    bias = torch.zeros(E)
    bias[5] = NAN
    check(x.to(DEV), bias.to(DEV), 6, score, groups=groups, keep=keep)
    check(x.to(DEV), bias.to(DEV), 6, score, renorm=True, groups=groups, keep=keep)
    ids, w = call(x.to(DEV), bias.to(DEV), 6, score, groups=groups, keep=keep)
    assert (ids[1] == -1).all() and (w[1] == 0).all() and torch.isfinite(w[[0, 1, 2]]).all() and torch.isnan(w[3:]).all()


@pytest.mark.parametrize("E,groups,keep", [(64, 4, 1), (64, 4, 2), (1024, 2, 1), (200, 100, 1), (200, 100, 30)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_infinite_biases_of_groups(E, groups, keep, score):
    """A group with one +Inf bias and a later one with two both have the score +Inf: equal, so the lower index goes first."""
    print("infinite bias", E, groups, keep, score, flush=True)
    size = E // groups
    x = torch.randn(4, E, generator=torch.Generator().manual_seed(E + keep))
    bias = torch.zeros(E)
    last = (groups - 1) * size
    bias[last - size + 1], bias[last], bias[last + 1] = INF, INF, INF
    x[2, last - size + 1] = -INF                                # masked: the bias does not bring it back
    k = min(6, keep * size)
    check(x.to(DEV), bias.to(DEV), k, score, groups=groups, keep=keep)
    ids, _ = call(x.to(DEV), bias.to(DEV), k, score, groups=groups, keep=keep)
    assert ids[:, 0].tolist() == [last - size + 1] * 2 + [last] + [last - size + 1]


@pytest.mark.parametrize("E,groups", [(64, 4), (256, 8), (512, 4), (200, 100), (1020, 3)])
def test_group_scores_count_42_bits(E, groups):
    """Ranks 1000 + p of two groups, all truncated to a multiple of 2^-33 (1000 has 10 bits before the point): p(-40) = 4e-18
    counts as nothing and p(-22.5) = 1.69e-10 as 2^-33.  The sums 2000 and 2000 + 2^-33 are equal once 42 bits of them count
    (a step of 2^-32), so the lower group goes first; one step more, p(-21) = 7.6e-10 = 6 2^-33, tells them apart."""
    size, low, high = E // groups, 1, groups - 1
    x = torch.zeros(2, E)
    bias = torch.zeros(E)
    for g in (low, high):
        x[:, g * size:(g + 1) * size] = -40.0
        bias[g * size:g * size + 2] = 1000.0
    x[0, high * size], x[1, high * size] = -22.5, -21.0
    ids, _ = call(x.to(DEV), bias.to(DEV), 2, "sigmoid", groups=groups, keep=1)
    assert ids[0].tolist() == [low * size, low * size + 1]
    assert ids[1].tolist() == [high * size, high * size + 1]


def weight_error(E, groups, k, score, with_bias, renorm, dtype, seed):
    """Largest |got - want| / |want| of a call's weights, in units of 2^-24 (half a unit of float32, the last rounding's share)."""
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(64, E, generator=g) * 2).to(dtype)
    bias = torch.randn(E, generator=g) * 0.2 if with_bias else None
    ids, w = call(x.to(DEV), None if bias is None else bias.to(DEV), k, score, renorm=renorm, scale=2.5, groups=groups, keep=groups)
    ri, rw = route_reference(x.float().numpy(), None if bias is None else bias.numpy(), E, k, score, renorm, 2.5, groups, groups)
    assert np.array_equal(ids.cpu().numpy(), ri)
    return float((np.abs(w.cpu().numpy().astype(np.float64) - rw) / rw).max() * 2.0 ** 24)


@pytest.mark.parametrize("E,groups,k", [(60, 1, 6), (64, 4, 8), (256, 1, 8), (256, 8, 8), (1000, 1, 10), (200, 100, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_weights_are_float64_but_for_one_denominator(E, groups, k, dtype):
    """Everything but the softmax denominator without a bias is formed in float64 (2^-45 at worst), so that a weight errs by its one
    rounding to float32, 2^-24, and renormalized weights, in which that denominator cancels, do too.

    That denominator is a float32 sum of exp(-d), d = max - x.  With p = exp(-d) / sum, each d rounded by 2^-24 d moves the sum by
    sum p d 2^-24 <= ln(E) 2^-24 (the entropy of p, less ln sum >= 0); the exponential is good to 2 units, 4 2^-24; at most
    15 + 6 additions on the way of a term round by 2^-24 each; and the weight once: under (ln E + 4 + 21 + 1) 2^-24."""
    for score in ("softmax", "sigmoid"):
        for with_bias in (False, True):
            for renorm in (False, True):
                float32_sum = score == "softmax" and not with_bias and not renorm and groups < 100
                bound = np.log(E) + 26 if float32_sum else 1 + 2.0 ** -16
                err = weight_error(E, groups, k, score, with_bias, renorm, dtype, E + k)
                print(E, groups, score, with_bias, renorm, dtype, "%.2f of %.2f" % (err, bound), flush=True)
                assert err <= bound, (score, with_bias, renorm, err, bound)


# ------------------------------------------------------------------------------------------- grouped products
def test_as_many_workgroups_as_a_launch_may_not_have():
    """1024 experts of 131071 columns in the paired form (2^32 work-items in tiles of 16 columns).  Small integers: both sums are
    exact, and h adds the 8 2^-23 of its float32 evaluation and half a bfloat16 step, 2^-8.  Gates reach -8 * 16 = -128, and for
    g < -87.3 exp(g) may count as 0: g exp(g) u / (1 + exp(g)) is then 0 in place of up to |g u| 2^-126 <= 2^-112, far above
    bfloat16's least value, so that much is allowed for."""
    E, I, K = 1024, 131071, 8
    counts = [2] * 16 + [1] * (E - 16)
    rows = sum(counts)
    g = torch.Generator(device=DEV).manual_seed(70)
    X = torch.randint(-4, 5, (rows, K), generator=g, device=DEV).to(torch.bfloat16)
    W = torch.randint(-4, 5, (E, 2 * I, K), generator=g, device=DEV, dtype=torch.int8).to(torch.bfloat16)
    H = torch.full((rows, I), 7.0, dtype=torch.bfloat16, device=DEV)
    off = offsets_of(counts)
    print("2^32 work-items", flush=True)
    L.w4a8_moe_gemm_silu_w16a16(X, None, 1, torch.from_numpy(off).to(DEV), W, H)
    torch.cuda.synchronize()
    for e in range(0, E, 31):
        r = slice(int(off[e]), int(off[e + 1]))
        y = X[r].float() @ W[e].float().t().contiguous()
        a, u = y[:, :I].double(), y[:, I:].double()
        h = a * torch.sigmoid(a) * u
        e8 = 8 * 2.0 ** -23 * h.abs() + 2.0 ** -126 * (a * u).abs() * (a < 0)
        over = (H[r].double() - h).abs() - (e8 + (h.abs() + e8) * 2.0 ** -8 + 1e-38)
        i = int(over.argmax())
        assert float(over.reshape(-1)[i]) <= 0, (e, float(a.reshape(-1)[i]), float(u.reshape(-1)[i]), float(H[r].reshape(-1)[i]))


# W8A8 calls (counts of the experts, K, N; with a gather of k = 2) and the kernel that each is there for
W8_FORMS = {
    "16-row tiles": ([5, 0, 2], 256, 70),
    "32-row tiles": (COUNTS["edges"], 256, 70),
    "128 x 128": (LARGE, 1152, 2306),
    "128 x 128, whole stores": (LARGE, 1152, 2304),
    "256 x 256": (LARGE, 1152, 4102),
    "256 x 256, whole stores": (LARGE, 1152, 4096),
}


@pytest.mark.parametrize("form", list(W8_FORMS))
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
def test_w8_rows_of_nothing_under_any_scale(form, out):
    """A gather entry that names no row gives zeros also where the channel's scale is infinite, NaN or so large that its product
    with another row's sum overflows; the other rows are as ever."""
    counts, K, N = W8_FORMS[form]
    print("rows of nothing", form, out, flush=True)
    c = w8_inputs(71, counts, K, N, src_rows=50, k=2)
    c["gather"][::5] = -1
    c["gather"][1::7] = 100                                     # token 50 of 50
    c["gather"][2::9] = 2 ** 31 - 1
    odd = [3, 4, 5, 6, N - 1]
    c["sw"][:, odd] = np.array([np.inf, np.nan, -np.inf, 3e38, np.nan], np.float32)
    c["codes"][:, :, 6] = 127
    c["Xq"][0] = 127
    Y = run_w8(c, out).cpu()
    none = torch.from_numpy((c["gather"] < 0) | (c["gather"] >= 100))
    assert none.any() and (Y[none] == 0).all()
    keep = [n for n in range(N) if n not in odd]
    with np.errstate(all="ignore"):
        want = torch.from_numpy(w8_reference(c))[:, keep]
    e = 4 * 2.0 ** -24 * want.abs()
    assert_within(Y[:, keep], want, e + half_step(out, want.abs() + e) + 1e-38, form)
    assert torch.isnan(Y[~none][:, [4, N - 1]]).all() and not torch.isfinite(Y[~none][:, [3, 5]]).any()


def test_w8_rows_do_not_depend_on_the_call():
    """The same rows, bit for bit, in calls of every kernel, with any k, alone and among others; scales of 0, -0 and NaN among them."""
    K, N = 1152, 4102
    c = w8_inputs(72, LARGE, K, N)
    c["sx"][:4] = np.array([0.0, -0.0, np.nan, -0.5], np.float32)
    c["sw"][0, :3] = np.array([np.inf, np.nan, -1.0], np.float32)
    dw = w8_device(c)
    d, w, t = dw
    want = run_w8(c, torch.float32, dw)                         # 256 x 256 tiles
    assert (want[:2, 2:] == 0).all() and (want[1] == 0).all() and not torch.signbit(want[1]).any()
    bits = want.view(torch.int32)
    print("k", flush=True)
    for k in (2, 3, 5):
        assert torch.equal(run_w8(dict(c, k=k), torch.float32, dw).view(torch.int32), bits), k
    print("alone", flush=True)
    for a, b in ((0, 1), (0, 4), (0, 16), (0, 40), (100, 129)): # rows of expert 0: one, a few, two tiles of 32
        off = torch.tensor([0] + [b - a] * 5, dtype=torch.int32, device=DEV)
        Y = torch.empty(b - a, N, device=DEV)
        L.w4a8_moe_gemm_w8a8(t["Xq"][a:b], t["sx"][a:b], None, 1, off, 5, b - a, w.blob, w.stride, d, Y, L.W4A8_OUT_F32)
        assert torch.equal(Y.view(torch.int32), bits[a:b]), (a, b)
    print("narrow", flush=True)
    narrow = w8_inputs(72, LARGE, K, N)
    narrow.update(sx=c["sx"], sw=c["sw"][:, :2306].copy(), codes=narrow["codes"][:, :, :2306].copy())
    assert torch.equal(run_w8(narrow, torch.float32).view(torch.int32), bits[:, :2306])        # 128 x 128 tiles


# ------------------------------------------------------------------------------------------- layers
@pytest.mark.parametrize("T,E,k,H,I,hot", [(3, 16, 4, 384, 128, None), (40, 8, 3, 256, 640, None), (300, 4, 2, 1152, 1280, 1)])
def test_w8_layer_of_unequal_widths_against_the_oracle(T, E, k, H, I, hot):
    """H and I apart: a channel's one scale is given to the oracle as the scales of its groups of 128, which is the same sum."""
    X, ids, w = routed(91, T, E, k, H, hot=hot)
    wts = weights8(92, E, H, I)
    per_group = {e: (cgu, np.repeat(sgu, H // 128, axis=0), None, cd, np.repeat(sd, I // 128, axis=0), None)
                 for e, (cgu, sgu, _, cd, sd, _) in wts[4].items()}
    print("layer", T, E, k, H, I, flush=True)
    ref = O.moe_layer(X.float().cpu().numpy(), ids.cpu().numpy(), w.cpu().numpy(), lambda e: per_group[e], E, I, 128)
    check_moe(run8(X, ids, w, E, wts), ref, {e: per_group[e] for e in np.unique(ids.cpu().numpy())}, 128)


# ------------------------------------------------------------------------------------------- refusals on device tensors
def test_refusals_leave_the_output_alone():
    """Wrong types, CPU tensors among device ones, gaps and overlaps: refused before anything is launched."""
    i32 = dict(dtype=torch.int32, device=DEV)
    x, ids, w, d = torch.randn(4, 64, device=DEV), torch.full((4, 2), -7, **i32), torch.full((4, 2), -7.0, device=DEV), L.route_desc(64, 2)
    bad = [lambda: L.w4a8_moe_route(x, d, ids.long(), w), lambda: L.w4a8_moe_route(x, d, ids, w.half()),
           lambda: L.w4a8_moe_route(x.cpu(), d, ids, w), lambda: L.w4a8_moe_route(x, d, ids, w, bias=torch.zeros(64)),
           lambda: L.w4a8_moe_route(x, d, ids, w, bias=torch.zeros(64, dtype=torch.float64, device=DEV)),
           lambda: L.w4a8_moe_route(x[:1].expand(4, 64), d, ids, w), lambda: L.w4a8_moe_route(x.double(), d, ids, w),
           lambda: L.w4a8_moe_route(x, d, ids.t().contiguous().t(), w)]
    dw = L.desc(128, 32, 128, False, bits=8)
    size = L.w4a8_packed_size(dw)
    blob, xq, sx = torch.zeros(2, size, dtype=torch.uint8, device=DEV), torch.zeros(4, 128, dtype=torch.int8, device=DEV), torch.zeros(4, device=DEV)
    off, ga, Y = torch.tensor([0, 2, 4], **i32), torch.zeros(4, **i32), torch.full((4, 32), 7.0, dtype=torch.bfloat16, device=DEV)

    def w8(xq=xq, sx=sx, ga=ga, off=off, blob=blob, stride=size, Y=Y, out=L.W4A8_OUT_BF16):
        L.w4a8_moe_gemm_w8a8(xq, sx, ga, 1, off, 2, 4, blob, stride, dw, Y, out)

    Y8 = torch.full((8, 32), 7, dtype=torch.uint8, device=DEV)
    bad += [lambda: w8(xq=xq.to(torch.uint8)), lambda: w8(sx=sx.half()), lambda: w8(ga=ga.long()), lambda: w8(ga=ga.cpu()), lambda: w8(off=off.long()),
            lambda: w8(off=torch.zeros(3, 2, **i32)[:, 0]), lambda: w8(ga=torch.zeros(8, **i32)[::2]), lambda: w8(Y=Y.half()),
            lambda: w8(Y=Y8[:4]), lambda: w8(out=L.W4A8_OUT_F32), lambda: w8(blob=blob[:1].expand(2, size)), lambda: w8(stride=-size)]
    X, W = torch.zeros(4, 64, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 32, 64, dtype=torch.bfloat16, device=DEV)
    for f in (L.w4a8_moe_gemm_w16a16, L.w4a8_moe_gemm_silu_w16a16):
        y = Y if f is L.w4a8_moe_gemm_w16a16 else Y[:, :16]
        bad += [lambda f=f, y=y: f(X.half(), ga, 1, off, W, y), lambda f=f, y=y: f(X.float(), ga, 1, off, W.float(), y),
                lambda f=f, y=y: f(X, ga.long(), 1, off, W, y), lambda f=f, y=y: f(X, ga, 1, off, W.cpu(), y),
                lambda f=f, y=y: f(X, ga, 1, torch.zeros(6, **i32)[::2], W, y), lambda f=f, y=y: f(X, ga, 1, off, W, y.half()),
                lambda f=f, y=y: f(X, ga, 1, off, W, y[:1].expand(4, y.shape[1])), lambda f=f, y=y: f(X, ga, 1, off, W[:1].expand(2, 32, 64), y)]
    for i, call_it in enumerate(bad):
        with pytest.raises((ValueError, L.W4A8Error)):
            call_it()
    torch.cuda.synchronize()
    assert (ids == -7).all() and (w == -7).all() and (Y == 7).all() and (Y8 == 7).all()
    w8()                                                        # and what they were refused for is all that was wrong
    L.w4a8_moe_gemm_w16a16(X, ga, 1, off, W, Y)
    L.w4a8_moe_gemm_silu_w16a16(X, ga, 1, off, W, Y[:, :16])
    L.w4a8_moe_route(x, d, ids, w)
    torch.cuda.synchronize()
    assert (Y == 0).all() and (ids >= 0).all()
