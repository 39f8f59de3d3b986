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


CHILD = r"""
import ctypes, json, sys
import moe_token_int8_amd as L
lib, n, f = L.lib(), ctypes.c_int(0), 1 << 20
if lib.hipGetDeviceCount(ctypes.byref(n)) == 0 and n.value > 0:
    sys.exit(77)
out = []
for op, E, rows, N in json.loads(sys.argv[1]):
    a = (f, f, 0, None, 1, f, E, rows, rows, f, L.w4a8_mx_packed_size(64, 2 * N if op in ("silu", "quantized") else N), 64, N)
    out.append(lib.w4a8_mx_gemm(f, f, 0, rows, f, 64, N, f, N, 1, None) if op == "dense" else lib.w4a8_moe_gemm_mx(*a, f, N, 1, None) if op == "moe"
               else lib.w4a8_moe_gemm_silu_mx(*a, f, N, 0, None) if op == "silu" else lib.w4a8_moe_gemm_silu_mx_quant(*a, 0, f, f, None))
print(json.dumps(out))
"""


def test_tile_numbers_fit_32_bits():
    """Row tiles of 32 (and one more for each expert) by blocks of 64 weight columns are fewer than 2^32.  (In a process that sees no GPU the
    launch of what is taken fails, and the made-up pointers are never used.)"""
    calls = [("dense", 1, 1 << 24, 1 << 20), ("dense", 1, 1 << 24, 1 << 19), ("dense", 1, 1 << 24, (1 << 19) - 64), ("dense", 1, (1 << 24) - 32, 1 << 19),
             ("dense", 1, 1 << 20, 1 << 20), ("moe", 1024, 1 << 24, (1 << 19) - 64), ("moe", 1024, 1 << 24, (1 << 19) - 1024),
             ("silu", 8, 1 << 24, 1 << 18), ("silu", 8, 1 << 24, (1 << 18) - 64), ("quantized", 8, 1 << 24, 1 << 18), ("quantized", 8, 1 << 24, (1 << 18) - 64)]
    want = [(rows // 32 + E) * -(-(2 * N if op in ("silu", "quantized") else N) // 64) for op, E, rows, N in calls]
    want = [L.W4A8_EUNSUPPORTED if n >= 1 << 32 else L.W4A8_EHIP for n in want]
    assert want.count(L.W4A8_EHIP) == 5
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1", CUDA_VISIBLE_DEVICES="-1")
    r = subprocess.run([sys.executable, "-c", CHILD, json.dumps(calls)], capture_output=True, text=True, env=env, timeout=120, cwd=ROOT)
    if r.returncode == 77:
        pytest.skip("a GPU stays visible to the child")
    assert r.returncode == 0, r.stderr
    assert json.loads(r.stdout) == want
