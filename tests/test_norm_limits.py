"""Sizes at the limits of the norm around a block: a launch has less than 2^32 work-items."""
import ctypes
import json
import os
import subprocess
import sys

import pytest

import moe_token_int8_amd as L

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p(1 << 20)                                    # aligned, never dereferenced

CHILD = r"""
import ctypes, json, sys
import moe_token_int8_amd as L
lib, n, f = L.lib(), ctypes.c_int(0), 1 << 20
if lib.hipGetDeviceCount(ctypes.byref(n)) == 0 and n.value > 0:
    sys.exit(77)
d = ctypes.byref(L.norm_desc())
print(json.dumps([lib.w4a8_norm_residual(f, 0, H, f, 0, H, None, 0, None, f, d, M, H, f, H, f, H, None) for M, H in json.loads(sys.argv[1])]))
"""


@pytest.mark.parametrize("H", [8193, 16384, 16385, 65536])
def test_rows_of_1024_threads(H):
    """Rows of more than 8192 take 1024 threads: 2^22 of them would be 2^32 work-items."""
    a = (P, L.W4A8_BF16, H, P, L.W4A8_BF16, H, None, 0, None, P, ctypes.byref(L.norm_desc()), 1 << 22, H, P, H)
    assert L.lib().w4a8_norm_residual(*a, P, H, None) == L.W4A8_EUNSUPPORTED
    assert L.lib().w4a8_norm_residual_quant(*a, L.W4A8_MX_FP8, P, P, None) == L.W4A8_EUNSUPPORTED


def test_most_rows_pass_the_checks():
    """In a process that sees no GPU the launch then fails, and the made-up pointers are never used."""
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1", CUDA_VISIBLE_DEVICES="-1")
    sizes = [(1 << 22, 1), (1 << 22, 513), (1 << 22, 8192), ((1 << 22) - 1, 8193), ((1 << 22) - 1, 65536)]
    r = subprocess.run([sys.executable, "-c", CHILD, json.dumps(sizes)], capture_output=True, text=True, env=env, timeout=120, cwd=ROOT)
    if r.returncode == 77:
        pytest.skip("a GPU stays visible to the child")
    assert r.returncode == 0, r.stderr
    assert json.loads(r.stdout) == [L.W4A8_EHIP] * len(sizes)
