"""Sizes that the MX calls refuse: a layer that is refused has no workspace size, and tile numbers fit 32 bits."""
import ctypes
import json
import os
import subprocess
import sys

import pytest

import moe_token_int8_amd as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(1 << 20)                                    # aligned, never dereferenced
FP4, FP8 = L.W4A8_MX_FP4, L.W4A8_MX_FP8


def layer(T, k, H, I, E, fmt):
    return L.lib().w4a8_moe_forward_mx(P, P, P, T, k, E, fmt, P, 1 << 40, P, 1 << 40, H, I, P, 1 << 62, P, None)


# T, k, H, I, E
REFUSED = [(4, 2, 64, 40, 4), (4, 2, 64, 15, 4), (4, 2, 64, 32, 1025), (4, 2, 1 << 19, 1 << 13, 4), (4, 2, 1 << 13, 1 << 19, 4),
           (1 << 20, 1, 1 << 14, 32, 4), (1 << 23, 2, 1025, 32, 4), (1 << 24, 1, 1 << 20, 16, 1)]


@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("s", REFUSED)
def test_no_workspace_for_a_refused_layer(s, fmt):
    assert layer(*s, fmt) in (L.W4A8_EINVAL, L.W4A8_EUNSUPPORTED)
    assert L.lib().w4a8_moe_mx_workspace_size(*s, fmt) == 0


def test_workspace_at_the_limits():
    size = L.lib().w4a8_moe_mx_workspace_size
    for s in [((1 << 24) - 1, 1, 1024, 16, 1024), ((1 << 23) - 1, 2, 2048, 16, 1), (4, 2, 64, 32, 1024), (0, 2, 64, 32, 4), (1 << 21, 8, 64, 16, 8)]:
        assert size(*s, FP8) > 0, s
