"""Microscaled (MX) quantisation and products, and the norm around a block: cases, inputs and plain forms.

MX matrices [R, K] keep 32 neighbours along K as a block with one power-of-two scale 2^(b - 127) (a byte b, E8M0) and elements
in E2M1 ("fp4", two to a byte, the first in the low half) or E4M3 ("fp8").  Rows are padded with zeros to a multiple of 128.
Weights are fp4, in the order of the matrix instructions' operands (`_pack`); activations fp4 or fp8, row by row.

  quant  rows -> codes and scales -> the values that these stand for
  gemm   Y = X W^T
  moe    grouped product: rows sorted by expert, each with its expert's weights
  silu   grouped gate/up product with silu(gate) * up in its epilogue
  layer  one expert layer from bfloat16 to bfloat16: quantise, gate/up, quantise again, down, weighted sum per token
  norm   r' = r + alpha g u, u = X or its RMS norm times p;  h = RMS norm of r' times w, kept in 16 bits or quantised

Expert e owns the sorted rows [offsets[e], offsets[e + 1]); row r reads activation row sorted_rows[r] // k with a gather, or
row r.  Rows at or past offsets[E] belong to nobody (padded tokens) and keep what the output held.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # the rows of a small decode step in front of a fused gate/up projection
        {"name": "quant_decode", "op": "quant", "M": 8, "K": 4096, "fmt": "fp8", "dtype": "bf16"},
        # a long prompt of wide rows
        {"name": "quant_prompt", "op": "quant", "M": 8192, "K": 7168, "fmt": "fp4", "dtype": "bf16"},
        # fused gate/up projection of a small decode step
        {"name": "gemm_decode", "op": "gemm", "M": 8, "K": 4096, "N": 14336, "fmt": "fp8", "out": "bf16"},
        # down projection of a prompt, activations in 4 bits
        {"name": "gemm_prompt", "op": "gemm", "M": 4096, "K": 14336, "N": 4096, "fmt": "fp4", "out": "bf16"},
        # down product of a large decode step: about two rows for each of 256 experts
        {"name": "moe_decode", "op": "moe", "T": 64, "E": 256, "k": 8, "K": 2048, "N": 7168, "gather": False, "fmt": "fp8",
         "out": "bf16", "zipf": 0.0, "pad": 0.0},
        # gate/up product of a skewed, padded prompt of odd length and width, kept in float32
        {"name": "moe_ragged", "op": "moe", "T": 4153, "E": 64, "k": 6, "K": 4096, "N": 2815, "gather": True, "fmt": "fp4",
         "out": "f32", "zipf": 0.5, "pad": 0.05},
        # gate/up product of one token
        {"name": "silu_token", "op": "silu", "T": 1, "E": 64, "k": 6, "K": 4096, "N": 1408, "gather": True, "fmt": "fp8",
         "out": "bf16", "zipf": 0.0, "pad": 0.0},
        # gate/up product of a long prompt
        {"name": "silu_prompt", "op": "silu", "T": 8192, "E": 64, "k": 6, "K": 4096, "N": 1408, "gather": True, "fmt": "fp8",
         "out": "bf16", "zipf": 0.5, "pad": 0.0},
        # a layer of a skewed serving batch
        {"name": "layer_batch", "op": "layer", "T": 512, "E": 64, "k": 6, "K": 4096, "N": 1408, "fmt": "fp8", "zipf": 1.1,
         "pad": 0.0},
        # a layer of a large decode step of few rows an expert
        {"name": "layer_decode", "op": "layer", "T": 64, "E": 256, "k": 8, "K": 7168, "N": 2048, "fmt": "fp4", "zipf": 0.0,
         "pad": 0.0},
        # the norm in front of a projection, for the tokens of a small decode step
        {"name": "norm_decode", "op": "norm", "M": 8, "K": 4096, "x": "bf16", "res": "bf16", "post": False, "gate": "", "alpha": 1.0,
         "fmt": "fp8"},
        # a long prompt with a norm on both sides of the block, a gate for each token and a float32 residual stream
        {"name": "norm_prompt", "op": "norm", "M": 8192, "K": 7168, "x": "bf16", "res": "f32", "post": True, "gate": "token",
         "alpha": 0.5, "fmt": ""},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quant", "gemm", "moe", "silu", "layer", "norm"))
    fmt = rng.choice(("fp4", "fp8"))
    if op in ("quant", "norm"):
        M, K = _log(rng, 1, 8192), _log(rng, 32, 8192)
        while M * K > 8192 * 7168:
            M //= 2
        if op == "quant":
            return {"op": op, "M": M, "K": K, "fmt": fmt, "dtype": rng.choice(("bf16", "f16", "f32"))}
        return {"op": op, "M": M, "K": K, "x": rng.choice(("bf16", "f16")), "res": rng.choice(("bf16", "f32")),
                "post": rng.random() < 0.5, "gate": rng.choice(("", "channel", "token")), "alpha": rng.choice((1.0, 0.22)),
                "fmt": rng.choice(("", "fp8"))}
    out = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "gemm":
        M, K, N = _log(rng, 1, 8192), _log(rng, 64, 14336), _log(rng, 16, 14336)
        while M * K * N > 4096 * 14336 * 4096:
            M //= 2
        return {"op": op, "M": max(M, 1), "K": K, "N": N, "fmt": fmt, "out": out}
    E = _log(rng, 4, 256)
    k = rng.randint(1, min(E, 8))
    K = _log(rng, 128, 7168)
    N = _log(rng, 16, 4096) if op == "moe" else 16 * max(1, _log(rng, 16, 2048) // 16)
    T = _log(rng, 1, 8192)
    wide = {"moe": 1, "silu": 2, "layer": 3}[op] * N
    while T * k * K * wide > 49152 * 4096 * 2816 or E * T * (K + wide) > 64 * 8192 * (4096 + 2816) or E * K * wide > 256 * 7168 * 6144:
        T, E = max(1, T // 2), max(k, E * 3 // 4)
    c = {"op": op, "T": T, "E": E, "k": k, "K": K, "N": N, "fmt": fmt, "zipf": rng.choice((0.0, 0.5, 1.1)),
         "pad": rng.choice((0.0, 0.0, 0.1))}
    if op != "layer":
        c["gather"] = True if op == "silu" else rng.random() < 0.5
        c["out"] = out if op == "moe" else rng.choice(("bf16", "f16"))
    return c


# ---------------------------------------------------------------------------------------------- the format
def _up(x, unit):
    return -(-x // unit) * unit


def _encode(x, fmt):
    """Element codes [R, K32] and scale bytes [R, K32 / 32] of float32 rows, K padded to whole blocks: the scale is the power of
    two under the block's largest value, less the format's largest exponent; elements to nearest even, saturating.  A block with
    a NaN or an infinity has the scale NaN (255) and codes 0."""
    R, K = x.shape
    if K % 32:
        x = torch.cat((x, x.new_zeros(R, _up(K, 32) - K)), 1)
    bits = x.view(torch.int32) & 0x7fffffff
    top = bits.view(R, -1, 32).amax(2)
    bad = top >= 0x7f800000
    b = ((top >> 23) - (2 if fmt == "fp4" else 8)).clamp_min(0)
    up = ((254 - b) << 23).view(torch.float32)
    y = (x.view(R, -1, 32) * up[:, :, None])
    a = y.abs().clamp_max(6.0 if fmt == "fp4" else 448.0)
    # spacing of the element grid: one unit of the mantissa (1 or 3 bits) at the value's exponent, not below the least
    man, least = (1, 0) if fmt == "fp4" else (3, -6)
    e = ((a.view(torch.int32) >> 23) - 127).clamp_min(least)
    q = torch.round(a * ((127 - e + man) << 23).view(torch.float32)).to(torch.int32)      # in units, 0 .. 2^(man + 1)
    mag = torch.where(q < (1 << man), q, q + ((e - least) << man))                          # carries go on into the exponent
    sign = torch.signbit(x.view(R, -1, 32)).to(torch.int32) << (3 if fmt == "fp4" else 7)
    code = torch.where(bad[:, :, None], 0, mag | sign).to(torch.uint8).view(R, -1)
    return code, torch.where(bad, 255, b).to(torch.uint8)


def _store(code, scale, fmt):
    """Codes and scales as they are kept: rows padded to 128, two fp4 codes a byte."""
    R, K = code.shape
    full = torch.zeros(R, _up(K, 128), dtype=torch.uint8, device=code.device)
    full[:, :K] = code
    s = torch.zeros(R, full.shape[1] // 32, dtype=torch.uint8, device=code.device)
    s[:, : scale.shape[1]] = scale
    return (full[:, 0::2] | (full[:, 1::2] << 4) if fmt == "fp4" else full), s


def _values(code):
    """float32 values of fp4 codes (0 .. 15)."""
    a = (code & 7).float()
    v = torch.where(a < 4, a * 0.5, torch.where(a < 6, a - 2, 2 * a - 8))
    return torch.where(code > 7, -v, v)


def _scales(s):
    """float32 values of scale bytes: 2^(b - 127), NaN for 255."""
    v = torch.where(s == 0, 0x00400000, s.to(torch.int32) << 23).view(torch.float32)
    return torch.where(s == 255, math.nan, v)


def _decode(q, s, fmt, K):
    """float32 values [R, K] of stored rows."""
    if fmt == "fp4":
        v = torch.stack((_values(q & 15), _values(q >> 4)), 2).view(q.shape[0], -1)
    else:
        v = q.view(torch.float8_e4m3fn).float()
    return (v.view(q.shape[0], -1, 32) * _scales(s)[:, :, None]).view(q.shape[0], -1)[:, :K]


def _sizes(N, K):
    """Where the scales of a packed fp4 matrix start, and its bytes."""
    codes = _up(N, 16) * _up(K, 128) // 2
    at = _up(codes, 256)
    return codes, at, _up(at + _up(N, 64) * _up(K, 128) // 32, 256)


def _pack(code, scale, out):
    """Packed weights [N, K] into `out`: codes by 16 columns x 128 k, 16 bytes for each (quarter of the 128, column), then the scales
    by 64 columns x 128 k, 4 bytes (the column in each of four 16s) for each (quarter, column)."""
    N, K = code.shape
    N16, N64, K1 = _up(N, 16), _up(N, 64), _up(K, 128) // 128
    q, s = _store(code, scale, "fp4")
    full = torch.zeros(N16, K1 * 64, dtype=torch.uint8, device=code.device)
    full[:N] = q
    codes, at, _ = _sizes(N, K)
    out[:codes] = full.view(N16 // 16, 16, K1, 4, 16).permute(0, 2, 3, 1, 4).reshape(-1)
    sf = torch.zeros(N64, K1 * 4, dtype=torch.uint8, device=code.device)
    sf[:N] = s
    out[at:at + N64 * K1 * 4] = sf.view(N64 // 64, 4, 16, K1, 4).permute(0, 3, 4, 2, 1).reshape(-1)


def _unpack(blobs, N, K):
    """float32 weights [experts, N, K] of packed blobs."""
    n, K1 = blobs.shape[0], _up(K, 128) // 128
    codes, at, _ = _sizes(N, K)
    q = blobs[:, :codes].view(n, -1, K1, 4, 16, 16).permute(0, 1, 4, 2, 3, 5).reshape(n, _up(N, 16), -1)[:, :N]
    s = blobs[:, at:at + _up(N, 64) * K1 * 4].view(n, -1, K1, 4, 16, 4).permute(0, 1, 5, 4, 2, 3).reshape(n, _up(N, 64), -1)[:, :N]
    return _decode(q.reshape(n * N, -1), s.reshape(n * N, -1), "fp4", K).view(n, N, K)


# ---------------------------------------------------------------------------------------------- inputs
def _routing(c, g):
    """Chosen experts and weights of each token, and the rows in expert order, as the framework's align step leaves them."""
    T, E, k = c["T"], c["E"], c["k"]
    z = torch.randn(T, E, device=DEV, generator=g)
    if c["zipf"]:
        rank = torch.randperm(E, device=DEV, generator=g) + 1
        z = z - c["zipf"] * torch.log(rank.float())
    ids = z.topk(k, dim=1).indices
    w = torch.softmax(z, 1).gather(1, ids)
    if c["pad"]:
        gone = (torch.rand(T, 1, device=DEV, generator=g) < c["pad"]) & (torch.arange(T, device=DEV)[:, None] > 0)
        ids, w = torch.where(gone, -1, ids), torch.where(gone, 0.0, w)
    flat = torch.where(ids < 0, E, ids).reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return ids.to(torch.int32), w, order.to(torch.int32), offsets, counts.tolist()


def _rows(g, M, K, dtype):
    """Activations: normal values, a few channels much larger than the others."""
    x = torch.randn(M, K, device=DEV, generator=g)
    x[:, torch.randint(0, K, (max(1, K // 1000),), device=DEV, generator=g)] *= 20
    return x.to(DTYPES[dtype])


def _experts(g, E, N, K):
    """Packed weights of E experts, and the bytes of one."""
    size = _sizes(N, K)[2]
    blobs = torch.zeros(E, size, dtype=torch.uint8, device=DEV)
    for e in range(E):
        _pack(*_encode(torch.randn(N, K, device=DEV, generator=g) * 0.02, "fp4"), blobs[e])
    return blobs


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    K = c["K"]
    s = {"c": c}
    if c["op"] == "quant":
        s["X"] = _rows(g, c["M"], K, c["dtype"])
        s["Xq"], s["sx"] = _buffers(c["M"], K, c["fmt"])
        s["Y"] = torch.empty(c["M"], K, dtype=DTYPES[c["dtype"]], device=DEV)
        return s
    if c["op"] == "norm":
        M = c["M"]
        s["X"] = _rows(g, M, K, c["x"])
        s["r"] = (torch.randn(M, K, device=DEV, generator=g) * 3).to(DTYPES[c["res"]])
        s["w"] = 1 + 0.2 * torch.randn(K, device=DEV, generator=g)
        s["p"] = 1 + 0.2 * torch.randn(K, device=DEV, generator=g) if c["post"] else None
        s["gate"] = None if not c["gate"] else torch.randn(M if c["gate"] == "token" else 1, K, device=DEV, generator=g).to(DTYPES[c["x"]])
        s["out"] = torch.empty_like(s["r"])
        s["h"] = torch.empty(M, K, dtype=DTYPES[c["x"]], device=DEV)
        if c["fmt"]:
            s["Xq"], s["sx"] = _buffers(M, K, c["fmt"])
        return s
    if c["op"] == "gemm":
        s["Xq"], s["sx"] = _store(*_encode(_rows(g, c["M"], K, "f32"), c["fmt"]), c["fmt"])
        s["W"] = _experts(g, 1, c["N"], K)[0]
        s["Y"] = torch.empty(c["M"], c["N"], dtype=DTYPES[c["out"]], device=DEV)
        return s
    E, k, N, T = c["E"], c["k"], c["N"], c["T"]
    rows = T * k
    ids, w, order, offsets, counts = _routing(c, g)
    s |= {"offsets": offsets, "rows": rows, "cap": max(max(counts), 1), "counts": counts}
    s["W"] = _experts(g, E, N if c["op"] == "moe" else 2 * N, K)
    if c["op"] == "layer":
        s |= {"ids": ids, "w": w, "order": order, "X": _rows(g, T, K, "bf16"), "Wd": _experts(g, E, K, N),
              "Y": torch.empty(T, K, dtype=torch.bfloat16, device=DEV)}
        # the workspace that a serving program keeps: both activations' codes, the routing and the experts' outputs
        s["ws"] = torch.empty(2 * T * _up(K, 128) + rows * (2 * _up(N, 128) + 2 * K + 8) + 4 * E + 65536, dtype=torch.uint8, device=DEV)
        return s
    s["gather"] = order if c["gather"] else None
    s["Xq"], s["sx"] = _store(*_encode(_rows(g, T if c["gather"] else rows, K, "f32"), c["fmt"]), c["fmt"])
    s["Y"] = torch.zeros(rows, N, dtype=DTYPES[c["out"]], device=DEV)
    return s


def _buffers(M, K, fmt):
    return (torch.empty(M, _up(K, 128) // (2 if fmt == "fp4" else 1), dtype=torch.uint8, device=DEV),
            torch.empty(M, _up(K, 128) // 32, dtype=torch.uint8, device=DEV))


# ---------------------------------------------------------------------------------------------- one pass
def run(state):
    c = state["c"]
    if own:
        return _run_own(c, state)
    if c["op"] == "quant":
        return _decode(*_store(*_encode(state["X"].float(), c["fmt"]), c["fmt"]), c["fmt"], c["K"]).to(state["X"].dtype)
    if c["op"] == "norm":
        return _plain_norm(c, state)
    if c["op"] == "gemm":
        x, W = _decode(state["Xq"], state["sx"], c["fmt"], c["K"]), _unpack(state["W"][None], c["N"], c["K"])[0]
        return (x @ W.t()).to(DTYPES[c["out"]])
    if c["op"] == "layer":
        return _plain_layer(c, state)
    x = _decode(state["Xq"], state["sx"], c["fmt"], c["K"])
    return _plain_grouped(c, state, x, state["gather"], c["op"] == "silu", state["W"]).to(DTYPES[c["out"]])


def _fmt(c):
    import moe_token_int8_amd as L

    return L.W4A8_MX_FP4 if c["fmt"] == "fp4" else L.W4A8_MX_FP8


def _run_own(c, s):
    import moe_token_int8_amd as L

    K = c["K"]
    if c["op"] == "quant":
        L.w4a8_mx_quant(s["X"], _fmt(c), s["Xq"], s["sx"])
        L.w4a8_mx_dequant(s["Xq"], s["sx"], _fmt(c), s["Y"])
        return s["Y"]
    if c["op"] == "norm":
        d = L.norm_desc(eps=1e-6, eps_post=1e-5, alpha=c["alpha"])
        if not c["fmt"]:
            L.w4a8_norm_residual(s["X"], s["r"], d, s["w"], s["out"], s["h"], post_w=s["p"], gate=s["gate"])
        else:
            L.w4a8_norm_residual_quant(s["X"], s["r"], d, s["w"], s["out"], _fmt(c), s["Xq"], s["sx"], post_w=s["p"], gate=s["gate"])
            L.w4a8_mx_dequant(s["Xq"], s["sx"], _fmt(c), s["h"])
        return {"residual": s["out"], "h": s["h"]}
    if c["op"] == "gemm":
        L.w4a8_mx_gemm(s["Xq"], s["sx"], _fmt(c), s["W"], K, c["N"], s["Y"])
    elif c["op"] == "moe":
        L.w4a8_moe_gemm_mx(s["Xq"], s["sx"], _fmt(c), s["gather"], c["k"], s["offsets"], c["E"], s["W"], s["W"].shape[1], K, s["Y"])
    elif c["op"] == "silu":
        L.w4a8_moe_gemm_silu_mx(s["Xq"], s["sx"], _fmt(c), s["gather"], c["k"], s["offsets"], c["E"], s["W"], s["W"].shape[1], K,
                                s["Y"])
    else:
        L.w4a8_moe_forward_mx(s["X"], s["ids"], s["w"], c["E"], _fmt(c), s["W"], s["W"].shape[1], s["Wd"], s["Wd"].shape[1], c["N"],
                              s["ws"], s["Y"])
    return s["Y"]


def _plain_norm(c, s):
    x = s["X"].float()
    if s["p"] is not None:
        x = x * torch.rsqrt((x * x).mean(1, keepdim=True) + 1e-5) * s["p"]
    if s["gate"] is not None:
        x = x * s["gate"].float()
    r = (s["r"].float() + c["alpha"] * x).to(s["r"].dtype)
    f = r.float()
    h = (f * torch.rsqrt((f * f).mean(1, keepdim=True) + 1e-6) * s["w"]).to(s["X"].dtype)
    if c["fmt"]:
        h = _decode(*_store(*_encode(h.float(), c["fmt"]), c["fmt"]), c["fmt"], c["K"]).to(h.dtype)
    return {"residual": r, "h": h}


def _plain_grouped(c, s, x, gather, pair, blobs):
    """Grouped product of float32 rows x, in float32; rows of nobody are zeros."""
    rows, cap, K, E = s["rows"], s["cap"], x.shape[1], c["E"]
    N = c["N"] * 2 if pair else (c["N"] if c["op"] != "layer" else c["K"])
    off = s["offsets"].long()
    r = torch.arange(rows, device=DEV)
    e = torch.searchsorted(off[1:].contiguous(), r, right=True)
    owned = e < E
    e = e.clamp_max(E - 1)
    x = x[gather.long() // c["k"]] if gather is not None else x
    if rows < E:  # fewer rows than experts: each row with its own expert's weights
        y = torch.bmm(_unpack(blobs[e], N, K), x[:, :, None])[:, :, 0]
    else:  # every expert's rows padded to the longest; a last slot takes the rows of nobody
        slot = torch.where(owned, r - off[e], cap)
        xp = torch.zeros(E, cap + 1, K, device=DEV)
        xp[e, slot] = x
        y = torch.bmm(_unpack(blobs, N, K), xp[:, :cap].transpose(1, 2).contiguous()).transpose(1, 2)[e, slot.clamp_max(cap - 1)]
    if pair:
        gate, up = y[:, : N // 2], y[:, N // 2:]
        y = gate / (1 + torch.exp(-gate)) * up
    return torch.where(owned[:, None], y, 0.0)


def _plain_layer(c, s):
    x = _decode(*_store(*_encode(s["X"].float(), c["fmt"]), c["fmt"]), c["fmt"], c["K"])
    h = _plain_grouped(c, s, x, s["order"], True, s["W"])
    h = _decode(*_store(*_encode(h, c["fmt"]), c["fmt"]), c["fmt"], c["N"])
    y = _plain_grouped(c, s, h, None, False, s["Wd"])
    out = torch.zeros(c["T"] * c["k"], c["K"], device=DEV)
    out[s["order"].long()] = y
    return (out.view(c["T"], c["k"], -1) * s["w"][:, :, None]).sum(1).to(torch.bfloat16)


# ---------------------------------------------------------------------------------------------- what a pass needs
def _size(fmt, M, K):
    return M * (K / 2 if fmt == "fp4" else K) + M * K / 32


def work(case):
    c = case
    K = c["K"]
    if c["op"] in ("quant", "norm"):
        M = c["M"]
        size = {"bf16": 2, "f16": 2, "f32": 4}
        if c["op"] == "quant":
            return {"bytes": 2 * M * K * size[c["dtype"]], "flops": 4 * M * K}
        gate = {"": 0, "channel": 2 * K, "token": 2 * M * K}[c["gate"]]
        return {"bytes": M * K * (2 * size[c["x"]] + 2 * size[c["res"]]) + gate + 4 * K * (2 if c["post"] else 1), "flops": 10 * M * K}
    N = c["N"]
    out = {"bf16": 2, "f16": 2, "f32": 4}[c.get("out", "bf16")]
    if c["op"] == "gemm":
        return {"bytes": _size("fp4", N, K) + _size(c["fmt"], c["M"], K) + c["M"] * N * out, "flops": 2 * c["M"] * K * N}
    T, E, k = c["T"] * (1 - c["pad"]), c["E"], c["k"]
    rows = T * k
    share = [(i + 1.0) ** -c["zipf"] for i in range(E)]
    active = min(rows, sum(1 - (1 - min(1.0, k * p / sum(share))) ** T for p in share))  # experts with any row
    if c["op"] == "layer":
        return {"bytes": active * _size("fp4", 3 * N, K) + T * K * 4, "flops": 6 * rows * K * N}
    width = 2 * N if c["op"] == "silu" else N
    return {"bytes": active * _size("fp4", width, K) + _size(c["fmt"], T if c["gather"] else rows, K) + rows * N * out,
            "flops": 2 * rows * K * width}


# ---------------------------------------------------------------------------------------------- in 64 bits
def _nearest(x, fmt):
    """float64 values that float64 rows [R, K] are kept as: a search over the format's values, block by block."""
    grid = list(E2M1) if fmt == "fp4" else [m / 8 * 2.0 ** -6 for m in range(8)] + [
        (1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8) if e < 8 or m < 7]
    grid = torch.tensor(grid, dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    R, K = x.shape
    out = torch.empty_like(x)
    for first in range(0, K, 4096):
        part = x[:, first:first + 4096]
        n = part.shape[1]
        part = torch.nn.functional.pad(part, (0, -n % 32)).view(R, -1, 32)
        top = part.abs().amax(2, keepdim=True)
        step = torch.exp2((torch.frexp(top)[1] - 1 - (2 if fmt == "fp4" else 8)).clamp_min(-127).double())
        step = torch.where(top == 0, 2.0 ** -127, step)
        a = (part / step).abs()
        i = torch.bucketize(a.contiguous(), mid)                       # a tie goes to the lower value here
        tie = (i < len(mid)) & (a == mid[i.clamp_max(len(mid) - 1)]) & (i % 2 == 1)
        v = grid[torch.where(tie, i + 1, i)]
        out[:, first:first + n] = (torch.copysign(v, part) * step).view(R, -1)[:, :n]
    return out


def _weights64(blob, N, K):
    """float64 weights [N, K] of one packed blob: where each element and its scale are kept."""
    n = torch.arange(N, device=DEV)[:, None]
    k = torch.arange(K, device=DEV)[None, :]
    K1 = _up(K, 128) // 128
    byte = blob[((n // 16 * K1 + k // 128) * 64 + k % 128 // 32 * 16 + n % 16) * 16 + k % 32 // 2].long()
    code = torch.where(k % 2 == 1, byte // 16, byte % 16)
    b = blob[_sizes(N, K)[1] + ((n // 64 * K1 + k // 128) * 64 + k % 128 // 32 * 16 + n % 16) * 4 + n % 64 // 16].double()
    v = torch.tensor(E2M1, dtype=torch.float64, device=DEV)[code % 8] * torch.exp2(b - 127)
    return torch.where(code >= 8, -v, v)


def _rows64(q, s, fmt, K):
    """float64 values of stored activation rows."""
    if fmt == "fp4":
        k = torch.arange(K, device=DEV)
        code = (q[:, k // 2].long() >> (k % 2 * 4)) & 15
        v = torch.tensor(E2M1 + tuple(-x for x in E2M1), dtype=torch.float64, device=DEV)[code]
    else:
        v = q[:, :K].contiguous().view(torch.float8_e4m3fn).double()
    return v * torch.exp2(s.double() - 127).repeat_interleave(32, 1)[:, :K]


def exact(case, seed):
    """The definitions in 64 bits, expert by expert."""
    c = case
    s = prepare(case, seed)
    K = c["K"]
    if c["op"] == "quant":
        return _nearest(s["X"].double(), c["fmt"])
    if c["op"] == "norm":
        x = s["X"].double()
        if s["p"] is not None:
            x = x / torch.sqrt(x.square().mean(1, keepdim=True) + 1e-5) * s["p"].double()
        if s["gate"] is not None:
            x = x * s["gate"].double()
        r = s["r"].double() + c["alpha"] * x
        kept = r.to(s["r"].dtype).double()
        h = kept / torch.sqrt(kept.square().mean(1, keepdim=True) + 1e-6) * s["w"].double()
        return {"residual": r, "h": _nearest(h.to(s["X"].dtype).double(), c["fmt"]) if c["fmt"] else h}
    if c["op"] == "gemm":
        return _rows64(s["Xq"], s["sx"], c["fmt"], K) @ _weights64(s["W"], c["N"], K).t().contiguous()
    N, k = c["N"], c["k"]
    layer = c["op"] == "layer"
    x = _nearest(s["X"].double(), c["fmt"]) if layer else _rows64(s["Xq"], s["sx"], c["fmt"], K)
    out = torch.zeros(c["T"] if layer else s["rows"], K if layer else N, dtype=torch.float64, device=DEV)
    gather = s["order"] if layer else s["gather"]
    first = 0
    for e, count in enumerate(s["counts"]):
        if count:
            row = gather[first:first + count].long() if gather is not None else torch.arange(first, first + count, device=DEV)
            src = row // k if gather is not None else row
            y = x[src] @ _weights64(s["W"][e], N if c["op"] == "moe" else 2 * N, K).t().contiguous()
            if c["op"] != "moe":
                y = y[:, :N] * torch.sigmoid(y[:, :N]) * y[:, N:]
            if layer:
                y = _nearest(y, c["fmt"]) @ _weights64(s["Wd"][e], K, N).t().contiguous()
                out.index_add_(0, src, y * s["w"].double().reshape(-1)[row][:, None])
            else:
                out[first:first + count] = y
        first += count
    return out
