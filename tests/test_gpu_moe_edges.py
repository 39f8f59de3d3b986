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
