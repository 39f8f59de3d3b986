"""The router against its float64 definition: ids exactly, weights to the rounding of float32.

Weight bound: softmax and sigmoid in float32 err by the rounding of the argument x - max (2^-24 |x - max|, absolute in the
exponent), an exponential good to 2 units, a sum of at most 1024 terms added in a tree or in lanes (at most 32 deep), two
divisions and the scale: together under (|x - max| + 40) 2^-23 relative."""
import numpy as np
import pytest
import torch

import moe_token_int8_amd as L
from moe_formats_cases import DEV, route_reference

pytestmark = pytest.mark.gpu
SCORES = {"softmax": L.W4A8_ROUTE_SOFTMAX, "sigmoid": L.W4A8_ROUTE_SIGMOID}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    L.lib()


def call(x, bias, k, score, renorm=False, scale=1.0, groups=1, keep=1, stream=None):
    T, E = x.shape
    ids = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
    w = torch.full((T, k), -7.0, device=DEV)
    d = L.route_desc(E, k, SCORES[score], renorm, scale, groups, keep)
    L.w4a8_moe_route(x, d, ids, w, bias=bias, stream=stream)
    return ids, w


def check(x, bias, k, score, renorm=False, scale=1.0, groups=1, keep=1):
    ids, w = call(x, bias, k, score, renorm, scale, groups, keep)
    torch.cuda.synchronize()
    xs = x.float().cpu().numpy()
    ri, rw = route_reference(xs, None if bias is None else bias.cpu().numpy(), x.shape[1], k, score, renorm, scale,
                             groups, keep)
    assert np.array_equal(ids.cpu().numpy(), ri)
    got = w.cpu().numpy().astype(np.float64)
    assert np.array_equal(np.isnan(got), np.isnan(rw))
    fin = np.where(np.isfinite(xs), xs, 0.0).astype(np.float64)
    spread = (fin.max(1) - fin.min(1))[:, None]
    ok = ~np.isnan(rw)
    bound = (spread + 40) * 2.0 ** -23 * np.abs(rw) + 1e-37
    assert (np.abs(got - rw)[ok] <= np.broadcast_to(bound, rw.shape)[ok]).all()


@pytest.mark.parametrize("E,k,T", [(1, 1, 1), (2, 2, 5), (8, 2, 64), (60, 6, 301), (64, 8, 17), (65, 5, 33), (256, 8, 130),
                                   (257, 9, 31), (512, 16, 9), (1000, 64, 7), (1024, 10, 12)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_sizes(E, k, T, score, with_bias):
    print("route", E, k, T, score, with_bias, flush=True)
    g = torch.Generator().manual_seed(E * 100 + k)
    for dt in TYPES.values():
        x = (torch.randn(T, E, generator=g) * 2).to(dt).to(DEV)
        bias = (torch.randn(E, generator=g) * 0.2).to(DEV) if with_bias else None
        check(x, bias, k, score)
        check(x, bias, k, score, renorm=True, scale=2.5)


@pytest.mark.parametrize("E,groups,keep,k", [(256, 8, 4, 8), (256, 8, 1, 8), (256, 8, 8, 6), (64, 2, 1, 4), (60, 4, 3, 6),
                                             (1024, 1024, 20, 20), (1024, 128, 3, 8), (160, 5, 2, 32), (512, 4, 2, 8)])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups(E, groups, keep, k, with_bias, score):
    print("route groups", E, groups, keep, k, with_bias, score, flush=True)
    g = torch.Generator().manual_seed(E + groups)
    x = (torch.randn(65, E, generator=g) * 2)
    x[::7, : E // 2] = -torch.inf                               # whole groups masked
    bias = (torch.randn(E, generator=g) * 0.2).to(DEV) if with_bias else None
    check(x.to(DEV), bias, k, score, renorm=True, groups=groups, keep=keep)


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("groups,keep", [(1, 1), (8, 3)])
def test_ties_go_to_the_lowest_index(with_bias, groups, keep):
    g = torch.Generator().manual_seed(5)
    x = torch.randint(-2, 3, (200, 256), generator=g).float()   # five values over 256 experts
    x[0] = 1.25
    bias = torch.randint(0, 2, (256,), generator=g).float().to(DEV) * 0.5 if with_bias else None
    for score in SCORES:
        for dt in TYPES.values():
            check(x.to(dt).to(DEV), bias, 8, score, groups=groups, keep=keep)


def test_signed_zeros_are_equal():
    x = torch.zeros(3, 70)
    x[0, :35], x[1, 35:] = -0.0, -0.0
    for score in SCORES:
        check(x.to(DEV), None, 5, score)


def test_extreme_logits():
    x = torch.tensor([[3e38, -3e38, 0.0, 1.0], [-3e38, -3e38, -3e38, -3e38], [80.0, 90.0, 100.0, 100.5], [-200.0, -100.0, -150.0, -90.0],
                      [1e-45, 0.0, -1e-45, 2e-45]])
    for score in SCORES:
        for bias in (None, torch.tensor([0.0, 0.25, -0.25, 0.0]).to(DEV)):
            check(x.to(DEV), bias, 3, score)
            check(x.to(DEV), bias, 3, score, renorm=True)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("groups,keep", [(1, 1), (4, 2)])
def test_masked_and_poisoned_rows(score, with_bias, groups, keep):
    g = torch.Generator().manual_seed(11)
    x = torch.randn(12, 64, generator=g)
    x[1] = -torch.inf                                           # a padded token
    x[2, 3:] = -torch.inf                                       # three experts for six places
    x[3, 5] = torch.nan
    x[4] = torch.nan
    x[5, 60] = torch.inf
    x[6, 0], x[6, 1] = torch.nan, -torch.inf
    x[7, 1::2] = -torch.inf
    x[8, 63] = torch.finfo(torch.float32).min
    bias = (torch.randn(64, generator=g) * 0.1).to(DEV) if with_bias else None
    check(x.to(DEV), bias, 6, score, groups=groups, keep=keep)
    check(x.to(DEV), bias, 6, score, renorm=True, groups=groups, keep=keep)


def test_bias_masks_and_poisons():
    g = torch.Generator().manual_seed(12)
    x = torch.randn(9, 40, generator=g).to(DEV)
    bias = torch.zeros(40)
    bias[4:30] = -torch.inf
    check(x, bias.to(DEV), 20, "sigmoid")                       # 14 experts for 20 places
    bias[35] = torch.nan
    check(x, bias.to(DEV), 5, "softmax")


def test_strided_rows_and_offset_start():
    g = torch.Generator().manual_seed(13)
    for dt in TYPES.values():
        full = torch.randn(50, 101, generator=g).to(dt).to(DEV)
        full[:, 73:] = torch.nan                                # next to the rows that are read
        full[:, :1] = torch.nan
        check(full[:, 1:73], None, 7, "softmax", renorm=True)
        check(full[1::2, 1:73], None, 7, "sigmoid")


def test_neighbouring_buffers_are_left_alone():
    x = torch.randn(5, 64, device=DEV)
    ids, w = torch.full((9, 4), -7, dtype=torch.int32, device=DEV), torch.full((9, 4), -7.0, device=DEV)
    L.w4a8_moe_route(x, L.route_desc(64, 4), ids[2:7], w[2:7])
    torch.cuda.synchronize()
    for t in (ids, w):
        assert (t[:2] == -7).all() and (t[7:] == -7).all() and (t[2:7] != -7).all()


def test_no_tokens():
    ids, w = call(torch.empty(0, 64, device=DEV), None, 4, "softmax")
    assert ids.shape == (0, 4)


def test_many_tokens_other_stream_and_graph():
    """More tokens than one round of workgroups, captured and replayed on other logits."""
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(20001, 128, generator=g, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        eager = [t.clone() for t in call(x, None, 8, "softmax", True)]
    torch.cuda.current_stream().wait_stream(s)
    top = torch.topk(x, 8, dim=1)                               # distinct float32 logits: no ties to settle
    assert torch.equal(eager[0].long(), top.indices)
    ids, w = torch.empty_like(eager[0]), torch.empty_like(eager[1])
    d = L.route_desc(128, 8, renormalize=True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.w4a8_moe_route(x, d, ids, w)
    for i in range(3):
        x.copy_(torch.randn(x.shape, generator=g, device=DEV))
        graph.replay()
        torch.cuda.synchronize()
        want = call(x, None, 8, "softmax", True)
        assert torch.equal(ids, want[0]) and torch.equal(w, want[1])


@pytest.mark.parametrize("E,groups,keep,k", [(200, 8, 3, 5), (56, 8, 2, 7), (36, 4, 4, 8), (252, 4, 2, 12), (768, 3, 1, 8),
                                             (1024, 2, 1, 8), (40, 20, 7, 8), (130, 13, 2, 20),
                                             (200, 100, 30, 8), (1020, 3, 2, 8)])             # the last two: more than the lanes hold
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_that_end_inside_a_lane(E, groups, keep, k, with_bias, score):
    print("route odd groups", E, groups, keep, k, with_bias, score, flush=True)
    g = torch.Generator().manual_seed(2 * E + groups)
    for dt in TYPES.values():
        x = (torch.randn(65, E + 4, generator=g) * 2).to(dt).to(DEV)[:, :E]     # rows further apart than E
        bias = (torch.randn(E, generator=g) * 0.2).to(DEV) if with_bias else None
        check(x, bias, k, score, renorm=True, groups=groups, keep=keep)


def test_sigmoid_far_from_zero():
    """Logits from -700 to 700: scores from 1e-304 to 1, by the sign of the logit one minus almost nothing or almost nothing."""
    x = torch.linspace(-700, 700, 256).repeat(3, 1).to(DEV)
    x[1] = x[1].flip(0)
    x[2] = x[2] - 400                                           # the smallest are below what a score tells apart, none is chosen
    check(x, None, 8, "sigmoid")
    check(x, torch.zeros(256, device=DEV), 8, "sigmoid")
    check(x[:, :100].contiguous(), torch.zeros(100, device=DEV), 8, "sigmoid")
