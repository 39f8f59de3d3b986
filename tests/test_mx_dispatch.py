"""Which kernels the microscaled (MX) products choose, read from the log (W4A8_LOG) of calls made in a child process that sees no
GPU: the choice is made on the host from the sizes, the launch then fails and the made-up pointers are never used."""
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import ctypes, json, sys
import moe_token_int8_amd as L
lib, n, f = L.lib(), ctypes.c_int(0), 1 << 20
if lib.hipGetDeviceCount(ctypes.byref(n)) == 0 and n.value > 0:
    sys.exit(77)
for op, fmt, E, rows, K, N, src in json.loads(sys.argv[1]):
    size = L.w4a8_mx_packed_size(K, N if op in ("dense", "moe") else 2 * N)
    a = (f, f, fmt, f if src else None, 1, f, E, rows, src or rows, f, size, K, N)
    if op == "dense":
        st = lib.w4a8_mx_gemm(f, f, fmt, rows, f, K, N, f, N, 1, None)
    elif op == "moe":
        st = lib.w4a8_moe_gemm_mx(*a, f, N, 1, None)
    elif op == "silu":
        st = lib.w4a8_moe_gemm_silu_mx(*a, f, N, 0, None)
    else:
        st = lib.w4a8_moe_gemm_silu_mx_quant(*a, fmt, f, f, None)
    assert st == L.W4A8_EHIP, (op, E, rows, K, N, st)
"""


def kernels_of(calls):
    """What the log says for calls (operator, format, E, rows, K, N, rows of the gathered source or 0), one text each."""
    env = dict(os.environ, W4A8_LOG="1", HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1", CUDA_VISIBLE_DEVICES="-1")
    r = subprocess.run([sys.executable, "-c", CHILD, json.dumps(calls)], capture_output=True, text=True, env=env, timeout=120, cwd=ROOT)
    if r.returncode == 77:
        pytest.skip("a GPU stays visible to the child")
    assert r.returncode == 0, r.stderr
    names = [line.split("-> ")[1] for line in r.stderr.splitlines() if line.startswith("w4a8: ")]
    assert len(names) == len(calls)
    return names


STREAM, KERNELS = "mx_stream_kernel", ["mx_stream_kernel"] + [
    f"mx_tile_kernel ({tile})" for tile in ("32 x 128", "32 x 256", "64 x 256", "128 x 256", "128 x 512")]


@pytest.mark.parametrize("op", ["dense", "moe", "silu", "quantized"])
@pytest.mark.parametrize("fmt", [0, 1])
def test_kernels_by_size(op, fmt):
    """Few rows of one matrix stream, and many rows and columns take the widest tiles."""
    E = 1 if op == "dense" else 8
    names = kernels_of([(op, fmt, E, rows * E, 4096, 4096, 0) for rows in (1, 16, 64, 256, 1024, 8192)])
    assert (names[0] == STREAM if E == 1 else KERNELS.index(names[0]) <= 3) and names[-1] == KERNELS[-1], names


def test_far_gather_streams():
    """Gathered rows past 32-bit offsets from the first are out of the tile kernel's reach."""
    K, src = 65536, 0xe0000000 // 65536
    names = kernels_of([("moe", fmt, 4, 4096, K, 512, s) for fmt, s in ((1, src - 1), (1, src), (0, src), (0, 2 * src))])
    assert [n == STREAM for n in names] == [False, True, False, True], names


def test_every_kernel_has_a_size_in_the_tests():
    """The sizes of tests/test_gpu_mx_kernels.py run every kernel in every product, in both formats."""
    from test_gpu_mx_kernels import SIZES

    for op, sizes in SIZES.items():
        for fmt in (0, 1):
            names = kernels_of([(op, fmt, len(c), sum(c), K, N, 0) for c, K, N in sizes])
            assert set(names) == set(KERNELS), (op, fmt, names)
