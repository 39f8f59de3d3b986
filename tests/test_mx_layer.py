"""The MX expert layer: the workspaces that it takes, and its steps over slices of the output's columns."""
import json
import os
import subprocess
import sys

import pytest
import torch

import moe_token_int8_amd as L
from mx_cases import DEV, FP4, FP8
from test_gpu_mx_kernels import SENTINEL, layer_inputs, steps, worst

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def up(x, unit):
    return -(-x // unit) * unit


def of_16_bit_outputs(T, k, H, I, E):
    """What a serving program may keep for a layer: the codes of tokens and of h with their scales in a byte each, the routing, the
    experts' outputs in 16 bits, and 64 KiB for the pieces' ends."""
    return 2 * T * up(H, 128) + T * k * (2 * up(I, 128) + 2 * H + 8) + 4 * E + 65536


def least(T, k, H, I, E, fmt):
    """The pieces in front of the experts' outputs, and 64 columns of those."""
    row = lambda K: up(K, 128) // (2 if fmt == FP4 else 1)  # noqa: E731
    R = T * k
    pieces = [T * row(H), T * up(H, 128) // 32, 4 * R, 4 * E + 4, 4 * R, R * row(I), R * up(I, 128) // 32]
    return sum(up(p, 256) for p in pieces) + 256 * R


SIZES = [(T, k, H, I, E) for T in (1, 2, 5, 16, 64, 300, 512, 1500, 8192) for k in (1, 2, 6, 8) for E in (8, 64, 256)
         for H, I in ((128, 16), (129, 48), (300, 2048), (1000, 16), (4096, 1408), (5555, 176), (7168, 2048))]

CHILD = r"""
import ctypes, json, sys
import moe_token_int8_amd as L
lib, n, f = L.lib(), ctypes.c_int(0), 1 << 20
if lib.hipGetDeviceCount(ctypes.byref(n)) == 0 and n.value > 0:
    sys.exit(77)
print(json.dumps([lib.w4a8_moe_forward_mx(f, f, f, T, k, E, fmt, f, L.w4a8_mx_packed_size(H, 2 * I), f, L.w4a8_mx_packed_size(I, H), H, I,
                                          f, ws, f, None) for T, k, H, I, E, fmt, ws in json.loads(sys.stdin.read())]))
"""


def test_workspaces_taken():
    """A workspace that leaves room for 64 columns passes the checks (in a process that sees no GPU the first launch then fails, and the
    made-up pointers are never used), one byte less does not; that of 16-bit outputs suffices at every size."""
    calls, want = [], []
    for s in SIZES:
        for fmt in (FP4, FP8):
            for ws, status in ((least(*s, fmt), L.W4A8_EHIP), (least(*s, fmt) - 1, L.W4A8_ESIZE), (of_16_bit_outputs(*s), L.W4A8_EHIP),
                               (L.w4a8_moe_mx_workspace_size(*s, fmt), L.W4A8_EHIP)):
                calls.append((*s, fmt, ws)), want.append(status)
    env = dict(os.environ, HIP_VISIBLE_DEVICES="-1", ROCR_VISIBLE_DEVICES="-1", CUDA_VISIBLE_DEVICES="-1")
    r = subprocess.run([sys.executable, "-c", CHILD], input=json.dumps(calls), capture_output=True, text=True, env=env, timeout=120, cwd=ROOT)
    if r.returncode == 77:
        pytest.skip("a GPU stays visible to the child")
    assert r.returncode == 0, r.stderr
    assert [(c, g) for c, g, w in zip(calls, json.loads(r.stdout), want) if g != w] == []


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("T,k,E,H,I", [(7, 2, 4, 64, 32), (400, 3, 5, 65, 48), (200, 4, 9, 129, 96), (300, 2, 3, 577, 144), (90, 6, 64, 1030, 80),
                                       (1, 8, 16, 7168, 128), (700, 6, 7, 1216, 64), (40, 2, 3, 64, 16)])
def test_layer_in_slices(T, k, E, H, I, fmt):
    """Slices of every kind (one of all columns, equal ones, a last one of one column or of a few, H that 4 does not divide) give the bits of
    the whole, which are those of the steps; what the workspace held and what lies behind it does not matter."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    GU, DN, down, x, logits = layer_inputs(T, k, E, H, I, fmt, T)
    ids = logits.topk(min(k, E), 1).indices.to(torch.int32).repeat(1, k)[:, :k].contiguous()
    w = torch.rand(T, k, device=DEV)
    if T > 4:
        ids[1] = -1

    def layer(size):
        ws = torch.full((size + 256,), 0xff, dtype=torch.uint8, device=DEV)
        rows = torch.full((T + 2, H), SENTINEL, dtype=torch.bfloat16, device=DEV)
        for _ in range(2):
            L.w4a8_moe_forward_mx(x, ids, w, E, fmt, GU, GU.shape[1], DN, DN.shape[1], I, ws[:size], rows[1:T + 1])
        assert (rows[0] == SENTINEL).all() and (rows[-1] == SENTINEL).all() and (ws[size:] == 0xff).all()
        return rows[1:T + 1]

    full, need = L.w4a8_moe_mx_workspace_size(T, k, H, I, E, fmt), least(T, k, H, I, E, fmt)
    out = layer(full)
    want, bound = steps(x, ids, w, fmt, E, GU, DN, down, H, I)
    assert worst(out, want, bound) <= 0
    for size in (of_16_bit_outputs(T, k, H, I, E), need, need + 128 * 4 * T * k, full - 256, need + (full - need) // 3):
        if size >= need:
            assert torch.equal(layer(size), out), size


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [FP4, FP8])
@pytest.mark.parametrize("T", [3, 130, 900])
def test_layer_in_slices_captured(T, fmt):
    """A layer in slices captured into a graph, replayed with its own eager work between on another stream with another workspace, on new
    inputs each time."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    k, E, H, I = 4, 12, 700, 112
    GU, DN, _, x, logits = layer_inputs(T, k, E, H, I, fmt, T)
    ids, w = logits.topk(k, 1).indices.to(torch.int32).contiguous(), torch.rand(T, k, device=DEV)
    size = least(T, k, H, I, E, fmt) + 192 * 4 * T * k                    # three slices of 256 columns
    ws, full = (torch.empty(n, dtype=torch.uint8, device=DEV) for n in (size, L.w4a8_moe_mx_workspace_size(T, k, H, I, E, fmt)))
    out, eager = torch.empty_like(x), torch.empty_like(x)

    def layer(work, o):
        L.w4a8_moe_forward_mx(x, ids, w, E, fmt, GU, GU.shape[1], DN, DN.shape[1], I, work, o)

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        layer(ws, out)
    for i in range(4):
        x *= -1.25 if i % 2 else 0.7
        ids.copy_(ids.flip(0))
        out.fill_(SENTINEL), ws.fill_(0xff)
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            layer(full, eager)
        torch.cuda.synchronize()
        assert torch.equal(out, eager)
