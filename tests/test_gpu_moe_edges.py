"""Inputs of the router and of the grouped products on which forms of the same operator once disagreed, or left their
definition: each is checked in every form that takes it."""
import numpy as np
import pytest
import torch

import moe_token_int8_amd as L
from moe_formats_cases import DEV, offsets_of
from test_gpu_moe_route import call, check

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
