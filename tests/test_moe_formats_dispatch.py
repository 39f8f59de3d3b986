"""Which kernels the grouped products choose, read from the log (W4A8_LOG) of calls made in a child process that sees no GPU:
the choice is made on the host from the sizes, the launch then fails and the made-up pointers are never used."""
import json
import os
import subprocess
import sys

import pytest

from test_gpu_moe_edges import W8_FORMS
from test_gpu_moe_tile_edges import SPLITS, TILES
from test_gpu_moe_tiles import LARGE, MIXED

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import ctypes, json, sys
import moe_token_int8_amd as L
lib, n, f = L.lib(), ctypes.c_int(0), 1 << 20
if lib.hipGetDeviceCount(ctypes.byref(n)) == 0 and n.value > 0:
    sys.exit(77)
for op, gather, k, E, rows, K, N in json.loads(sys.argv[1]):
    g = f if gather else None
    if op == "w8":
        d = L.desc(K, N, K, False, bits=8)
        st = lib.w4a8_moe_gemm_w8a8(f, f, g, k, f, E, rows, rows, f, L.w4a8_packed_size(d), ctypes.byref(d), f, 0, None)
    elif op == "w16":
        st = lib.w4a8_moe_gemm_w16a16(f, 0, K, g, k, f, E, rows, rows, f, N * K, K, K, N, f, N, 0, None)
    else:
        st = lib.w4a8_moe_gemm_silu_w16a16(f, 0, K, g, k, f, E, rows, rows, f, 2 * N * K, K, K, N, f, N, None)
    assert st == L.W4A8_EHIP, (op, E, rows, K, N, st)
"""


def kernels_of(calls):
    """What the log says for calls (operator, gathered, k, E, rows, K, N), one text each."""
    env = dict(os.environ, W4A8_LOG="1", HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1", CUDA_VISIBLE_DEVICES="-1")
    r = subprocess.run([sys.executable, "-c", CHILD, json.dumps(calls)], capture_output=True, text=True, env=env, timeout=120, cwd=ROOT)
    if r.returncode == 77:
        pytest.skip("a GPU stays visible to the child")
    assert r.returncode == 0, r.stderr
    names = [line.split("-> ")[1] for line in r.stderr.splitlines() if line.startswith("w4a8: w4a8_moe_gemm")]
    assert len(names) == len(calls)
    return names


def test_no_launch_of_2_to_the_32_work_items():
    """The paired form's 16-row class has ceil(N / 16) workgroups of 512 for an expert: with 1024 experts, N = 131071 and 131057
    give 8192 each, 2^32 work-items in all, which no launch may have; those take 32-row tiles, whose grid is small."""
    names = kernels_of([("silu", False, 1, 1024, 1040, 8, n) for n in (131071, 131057, 131056, 131072)] +
                       [("silu", False, 1024, 1024, 16384, 8, n) for n in (65535, 65521, 65536)])
    one = "moe_grouped_stream_kernel (32-row tiles)"
    assert [n == one for n in names] == [True, True, False, True, True, True, True], names


SMALL, BIG = "moe_grouped_tile_kernel (128 x 128)", "moe_grouped_tile_kernel (256 x 256)"


def test_log_names_the_tiles():
    """The sizes at which tests/test_gpu_moe_tiles.py means to reach each tile size, in every product, do."""
    rows, E = sum(LARGE), len(LARGE)
    small = [("w8", 1152, 2306), ("w8", 1280, 2049), ("w8", 1152, 2047), ("w16", 1096, 2050), ("w16", 1152, 2051), ("w16", 1096, 2047),
             ("silu", 1096, 1100), ("silu", 1280, 1153)]
    big = [("w8", 1152, 4102), ("w8", 1280, 4097), ("w8", 1152, 4095), ("w16", 1096, 4100), ("w16", 1152, 4099), ("w16", 1096, 4095),
           ("silu", 1096, 2060), ("silu", 1280, 2051)]
    for want, shapes in ((SMALL, small), (BIG, big)):
        names = kernels_of([(op, False, 1, E, rows, K, N) for op, K, N in shapes] +
                           [(op, True, 3, E, rows + 70, K, N) for op, K, N in shapes])
        assert all(n.endswith(want) for n in names), (want, names)
    rows, E = sum(MIXED), len(MIXED)
    names = kernels_of([("w16", True, 4, E, rows + 3, 2200, 4100), ("w8", True, 4, E, rows + 3, 2304, 4100),
                        ("w16", True, 4, E, rows + 3, 2200, 2050), ("silu", False, 1, E, rows, 2200, 1030)])
    assert [n.endswith(BIG) for n in names] == [True, True, False, False] and all(n.endswith(SMALL) for n in names[2:]), names


def test_forms_of_the_edge_tests():
    """tests/test_gpu_moe_edges.py runs the kernel that each of its forms is named for."""
    names = kernels_of([("w8", True, 2, len(c), sum(c), K, N) for c, K, N in W8_FORMS.values()])
    assert all(form.split(",")[0] in name for form, name in zip(W8_FORMS, names)), names


@pytest.mark.parametrize("tile", list(TILES))
def test_tiles_of_the_tile_edge_tests(tile):
    """Every size in tests/test_gpu_moe_tile_edges.py reaches the tile size it is listed under, however its rows are gathered."""
    N, I = TILES[tile]
    assert all(sum(s) <= sum(LARGE) for s in SPLITS)
    names = kernels_of([(op, g, k, len(LARGE), sum(LARGE), K, n) for op, K, n in (("w8", 1152, N), ("w16", 1096, N), ("silu", 1096, I))
                        for g, k in ((False, 1), (True, 1), (True, 2), (True, 3))])
    assert all(n.endswith(f"({tile})") for n in names), names
