"""Expert routing and expert-grouped products in 8 and 16 bits: cases, inputs and plain forms.

The operators of one mixture-of-experts layer whose experts are kept in 8-bit codes or unquantized:

  route  router scores -> top-k expert ids and weights
  w8     grouped product of int8 codes, one scale per token and one per output channel
  w16    grouped product in bfloat16 or float16
  silu   grouped gate/up product in 16 bits with silu(gate) * up in its epilogue

Rows are routed rows sorted by expert: expert e owns the rows [offsets[e], offsets[e + 1]), and row r reads activation
row sorted_rows[r] // k when a gather is given (gate/up products: X holds tokens) or row r (down products: X holds
routed rows).  Rows at or past offsets[E] belong to nobody (padded tokens) and keep what the output held.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # one token of a decode step: 256 experts, sigmoid scores with a selection bias
        {"name": "route_token", "op": "route", "T": 1, "E": 256, "k": 8, "score": "sigmoid", "bias": True, "renorm": True,
         "scale": 2.5, "groups": 1, "keep": 1, "dtype": "f32", "masked": 0.0, "pad": 0.0},
        # an odd serving batch, softmax over few experts in bfloat16 (ties are common), some experts masked, padded rows
        {"name": "route_batch", "op": "route", "T": 301, "E": 60, "k": 6, "score": "softmax", "bias": False, "renorm": False,
         "scale": 1.0, "groups": 1, "keep": 1, "dtype": "bf16", "masked": 0.1, "pad": 0.1},
        # a long prompt: 256 experts in 8 groups of which 4 are kept
        {"name": "route_prompt", "op": "route", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "bias": True,
         "renorm": True, "scale": 2.5, "groups": 8, "keep": 4, "dtype": "f32", "masked": 0.0, "pad": 0.0},
        # gate/up product of a single token
        {"name": "w8_token", "op": "w8", "T": 1, "E": 64, "k": 6, "K": 4096, "N": 2816, "gather": True, "out": "bf16",
         "zipf": 0.0, "pad": 0.0},
        # gate/up product of a large decode step: about two rows for each of 256 experts
        {"name": "w8_decode", "op": "w8", "T": 64, "E": 256, "k": 8, "K": 7168, "N": 4096, "gather": True, "out": "bf16",
         "zipf": 0.0, "pad": 0.0},
        # down product of a skewed, padded batch: one expert has most tokens, odd width, float32 output
        {"name": "w8_ragged", "op": "w8", "T": 509, "E": 64, "k": 6, "K": 1408, "N": 4095, "gather": False, "out": "f32",
         "zipf": 1.1, "pad": 0.05},
        # gate/up product of a long prompt
        {"name": "w8_prompt", "op": "w8", "T": 8192, "E": 64, "k": 6, "K": 4096, "N": 2816, "gather": True, "out": "bf16",
         "zipf": 0.5, "pad": 0.0},
        # down product of a single token, float16
        {"name": "w16_token", "op": "w16", "T": 1, "E": 64, "k": 6, "K": 1408, "N": 4096, "gather": False, "dtype": "f16",
         "out": "f16", "zipf": 0.0, "pad": 0.0},
        # down product of a large decode step
        {"name": "w16_decode", "op": "w16", "T": 64, "E": 256, "k": 8, "K": 2048, "N": 7168, "gather": False,
         "dtype": "bf16", "out": "bf16", "zipf": 0.0, "pad": 0.0},
        # down product of a long prompt
        {"name": "w16_prompt", "op": "w16", "T": 8192, "E": 64, "k": 6, "K": 1408, "N": 4096, "gather": False,
         "dtype": "bf16", "out": "bf16", "zipf": 0.5, "pad": 0.0},
        # gate/up of a small odd batch: a few rows for each expert
        {"name": "silu_batch", "op": "silu", "T": 33, "E": 64, "k": 6, "K": 4096, "N": 1408, "gather": True,
         "dtype": "bf16", "out": "bf16", "zipf": 0.0, "pad": 0.0},
        # gate/up of a prompt of odd length
        {"name": "silu_prompt", "op": "silu", "T": 4153, "E": 64, "k": 6, "K": 4096, "N": 1408, "gather": True,
         "dtype": "bf16", "out": "bf16", "zipf": 0.5, "pad": 0.02},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "w8", "w16", "silu"))
    E = _log(rng, 4, 256)
    k = rng.randint(1, min(E, 8))
    pad = rng.choice((0.0, 0.0, 0.1))
    if op == "route":
        T = _log(rng, 1, 16384)
        groups = rng.choice((1, 1, 4, 8))
        groups = groups if E % groups == 0 and E // groups >= 2 else 1
        keep = max(rng.randint(1, groups), -(-k * groups // E))
        return {"op": op, "T": T, "E": E, "k": k, "score": rng.choice(("softmax", "sigmoid")), "bias": rng.random() < 0.5,
                "renorm": rng.random() < 0.5, "scale": rng.choice((1.0, 2.5)), "groups": groups, "keep": keep,
                "dtype": rng.choice(("f32", "bf16")), "masked": rng.choice((0.0, 0.2)), "pad": pad}
    # the least unit of K is 128 for the packed 8-bit codes and 8 for the 16-bit rows
    unit, top = (128, 7168) if op == "w8" else (8, 4096)
    K = max(unit, _log(rng, 128, top) // unit * unit)
    N = _log(rng, 16, 4096 if op != "silu" else 2048)
    T = _log(rng, 1, 8192)
    c = {"op": op, "T": T, "E": E, "k": k, "K": K, "N": N, "gather": True if op == "silu" else rng.random() < 0.5,
         "zipf": rng.choice((0.0, 0.5, 1.1)), "pad": pad}
    if op == "w8":
        c["out"] = rng.choice(("bf16", "f32"))
    else:
        c["dtype"] = rng.choice(("bf16", "f16"))
        c["out"] = rng.choice((c["dtype"], c["dtype"], "f32")) if op == "w16" else c["dtype"]
    # no more than the largest listed case costs: weights, arithmetic and the padded plain form
    width = 2 * N if op == "silu" else N
    while T * c["k"] * K * width > 49152 * 4096 * 2816 or E * T * (K + width) > 64 * 8192 * (4096 + 2816):
        T //= 2
    c["T"] = max(1, T)
    return c


# ---------------------------------------------------------------------------------------------- inputs
def _routing(c, g):
    """Routed rows in expert order, as the framework's align step leaves them."""
    T, E, k = c["T"], c["E"], c["k"]
    z = torch.randn(T, E, device=DEV, generator=g)
    if c["zipf"]:
        rank = torch.randperm(E, device=DEV, generator=g) + 1
        z = z - c["zipf"] * torch.log(rank.float())
    ids = z.topk(k, dim=1).indices
    if c["pad"]:
        ids = torch.where((torch.rand(T, 1, device=DEV, generator=g) < c["pad"]) & (torch.arange(T, device=DEV)[:, None] > 0),
                          E, ids)
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    return order.to(torch.int32), offsets, counts.tolist()


def _codes(g, *shape):
    t = torch.empty(shape, dtype=torch.int8, device=DEV)
    for part in t.view(-1).split(1 << 28):
        part.copy_((torch.randn(part.shape, device=DEV, generator=g) * 40).round_().clamp_(-127, 127))
    return t


def _normal(g, dtype, std, *shape):
    t = torch.empty(shape, dtype=dtype, device=DEV)
    for part in t.view(-1).split(1 << 28):
        part.copy_(torch.randn(part.shape, device=DEV, generator=g) * std)
    return t


def _blob(codes, scales):
    """Packed blobs of 8-bit per-channel weights [E, N, K], as the framework lays them out: a 256-byte header (read on the
    host only, blank here), codes in superblocks of 16 columns x 128 k, then one float32 scale per column."""
    E, N, K = codes.shape
    n16 = -(-N // 16) * 16
    codes_end = 256 + n16 * K
    scales_off = -(-codes_end // 256) * 256
    total = -(-(scales_off + n16 * 4) // 256) * 256
    blob = torch.zeros(E, total, dtype=torch.uint8, device=DEV)
    for e in range(E):
        full = torch.zeros(n16, K, dtype=torch.int8, device=DEV)
        full[:N] = codes[e]
        sb = full.view(n16 // 16, 16, K // 128, 2, 4, 16).permute(0, 2, 4, 1, 3, 5)  # tile, block, quarter, column, half, k
        blob[e, 256:codes_end] = sb.reshape(-1).view(torch.uint8)
        s = torch.zeros(n16, device=DEV)
        s[:N] = scales[e]
        blob[e, scales_off:scales_off + n16 * 4] = s.view(torch.uint8)
    return blob


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV).manual_seed(seed)
    if c["op"] == "route":
        T, E = c["T"], c["E"]
        logits = torch.randn(T, E, device=DEV, generator=g) * 2
        if c["masked"]:
            gone = torch.rand(E, device=DEV, generator=g) < c["masked"]
            gone[: c["k"]] = False
            logits[:, gone] = -math.inf
        if c["pad"]:
            gone = torch.rand(T, device=DEV, generator=g) < c["pad"]
            gone[0] = False
            logits[gone] = -math.inf
        return {"c": c, "logits": logits.to(DTYPES[c["dtype"]]),
                "bias": torch.randn(E, device=DEV, generator=g) * 0.1 if c["bias"] else None,
                "ids": torch.empty(T, c["k"], dtype=torch.int32, device=DEV),
                "w": torch.empty(T, c["k"], dtype=torch.float32, device=DEV)}
    E, k, K, N = c["E"], c["k"], c["K"], c["N"]
    rows = c["T"] * k
    order, offsets, counts = _routing(c, g)
    s = {"c": c, "offsets": offsets, "rows": rows, "cap": max(max(counts), 1), "counts": counts,
         "gather": order if c["gather"] else None}
    src = c["T"] if c["gather"] else rows
    s["Y"] = torch.zeros(rows, N, dtype=DTYPES[c["out"]], device=DEV)
    if c["op"] == "w8":
        s["Xq"] = _codes(g, src, K)
        s["sx"] = (torch.rand(src, device=DEV, generator=g) + 0.5) * (4 / 127)
        sw = (torch.rand(E, N, device=DEV, generator=g) + 0.5) * (0.08 / 127)
        s["blob"] = _blob(_codes(g, E, N, K), sw)
    else:
        s["X"] = _normal(g, DTYPES[c["dtype"]], 1.0, src, K)
        s["W"] = _normal(g, DTYPES[c["dtype"]], 0.02, E, 2 * N if c["op"] == "silu" else N, K)
    return s


# ---------------------------------------------------------------------------------------------- one pass
def run(state):
    c = state["c"]
    if own:
        return _run_own(c, state)
    if c["op"] == "route":
        return _plain_route(c, state)
    return _plain_grouped(c, state)


def _run_own(c, s):
    import moe_token_int8_amd as L

    if c["op"] == "route":
        d = L.route_desc(c["E"], c["k"], L.W4A8_ROUTE_SIGMOID if c["score"] == "sigmoid" else L.W4A8_ROUTE_SOFTMAX,
                         renormalize=c["renorm"], scale=c["scale"], n_group=c["groups"], topk_group=c["keep"])
        L.w4a8_moe_route(s["logits"], d, s["ids"], s["w"], bias=s["bias"])
        return {"ids": s["ids"], "w": s["w"]}
    if c["op"] == "w8":
        d = L.desc(c["K"], c["N"], c["K"], False, bits=8)
        L.w4a8_moe_gemm_w8a8(s["Xq"], s["sx"], s["gather"], c["k"], s["offsets"], c["E"], s["rows"], s["blob"],
                             s["blob"].shape[1], d, s["Y"], L.W4A8_OUT_F32 if c["out"] == "f32" else L.W4A8_OUT_BF16)
    elif c["op"] == "w16":
        L.w4a8_moe_gemm_w16a16(s["X"], s["gather"], c["k"], s["offsets"], s["W"], s["Y"])
    else:
        L.w4a8_moe_gemm_silu_w16a16(s["X"], s["gather"], c["k"], s["offsets"], s["W"], s["Y"])
    return s["Y"]


def _plain_route(c, s):
    """In 64 bits: the order of two experts may hang on the last digit of their scores."""
    T, E, k, G = c["T"], c["E"], c["k"], c["groups"]
    x = s["logits"].double()
    if c["score"] == "softmax":
        top = x.max(1, keepdim=True).values
        p = torch.exp(x - torch.where(torch.isinf(top), 0.0, top))
        p = p / p.sum(1, keepdim=True).clamp_min(1e-300)
    else:
        p = 1 / (1 + torch.exp(-x))
    rank = x if s["bias"] is None else torch.where(torch.isinf(x), x, p + s["bias"].double())
    if G > 1:
        by = rank.view(T, G, E // G).sort(dim=2, descending=True).values
        best = by[:, :, 0] if s["bias"] is None else by[:, :, 0] + torch.where(torch.isinf(by[:, :, 1]), 0.0, by[:, :, 1])
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, : c["keep"]]
        keep = torch.zeros(T, G, dtype=torch.bool, device=x.device).scatter_(1, kept, True)
        rank = torch.where(keep[:, :, None].expand(T, G, E // G).reshape(T, E), rank, -math.inf)
    order = rank.sort(dim=1, descending=True, stable=True)
    ids, there = order.indices[:, :k], ~torch.isinf(order.values[:, :k])
    w = torch.where(there, p.gather(1, ids), 0.0)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True).clamp_min(1e-300)
    return {"ids": torch.where(there, ids, -1).to(torch.int32), "w": (w * c["scale"]).float()}


def _weights(c, s, which):
    """float32 weights [experts, rows of W, K] of the experts `which` (None: all), and their channel scales or None."""
    if c["op"] != "w8":
        return (s["W"] if which is None else s["W"][which]).float(), None
    K, N = c["K"], c["N"]
    n16 = -(-N // 16) * 16
    b = s["blob"] if which is None else s["blob"][which]
    q = b[:, 256:256 + n16 * K].view(torch.int8).view(-1, n16 // 16, K // 128, 4, 16, 2, 16)
    q = q.permute(0, 1, 4, 2, 5, 3, 6).reshape(-1, n16, K)[:, :N].float()
    at = -(-(256 + n16 * K) // 256) * 256
    return q, b[:, at:at + n16 * 4].contiguous().view(torch.float32)[:, :N]


def _plain_grouped(c, s):
    rows, cap, K = s["rows"], s["cap"], c["K"]
    off = s["offsets"].long()
    r = torch.arange(rows, device=DEV)
    e = torch.searchsorted(off[1:].contiguous(), r, right=True)
    owned = e < c["E"]
    e = e.clamp_max(c["E"] - 1)
    src = (s["gather"].long() // c["k"]) if s["gather"] is not None else r
    x = (s["Xq"] if c["op"] == "w8" else s["X"])[src].float()
    if rows < c["E"]:  # fewer rows than experts: each row with its own expert's weights
        W, sw = _weights(c, s, e)
        y = torch.bmm(W, x[:, :, None])[:, :, 0]
    else:  # every expert's rows padded to the longest; a last slot takes the rows of nobody
        W, sw = _weights(c, s, None)
        slot = torch.where(owned, r - off[e], cap)
        xp = torch.zeros(c["E"], cap + 1, K, device=DEV)
        xp[e, slot] = x
        y = torch.bmm(W, xp[:, :cap].transpose(1, 2).contiguous()).transpose(1, 2)[e, slot.clamp_max(cap - 1)]
        sw = sw if sw is None else sw[e]
    if c["op"] == "w8":
        y = y * s["sx"][src][:, None] * sw
    elif c["op"] == "silu":
        gate, up = y[:, : c["N"]], y[:, c["N"]:]
        y = gate / (1 + torch.exp(-gate)) * up
    return torch.where(owned[:, None], y, 0.0).to(DTYPES[c["out"]])


# ---------------------------------------------------------------------------------------------- what a pass needs
def work(case):
    c = case
    if c["op"] == "route":
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": c["T"] * c["E"] * size + (4 * c["E"] if c["bias"] else 0) + 8 * c["T"] * c["k"],
                "flops": 8 * c["T"] * c["E"]}
    T, E, k, K = c["T"] * (1 - c["pad"]), c["E"], c["k"], c["K"]
    width = 2 * c["N"] if c["op"] == "silu" else c["N"]
    rows = T * k
    share = [(i + 1.0) ** -c["zipf"] for i in range(E)]
    active = min(rows, sum(1 - (1 - min(1.0, k * p / sum(share))) ** T for p in share))  # experts with any row
    size = 1 if c["op"] == "w8" else 2
    out = 4 if c["out"] == "f32" else 2
    x = (T if c["gather"] else rows) * K * size
    return {"bytes": active * K * width * size + x + rows * c["N"] * out, "flops": 2 * rows * K * width}


def exact(case, seed):
    """The definitions in 64 bits, row by row of the router and expert by expert of the products."""
    c = case
    s = prepare(case, seed)
    if c["op"] == "route":
        return _exact_route(c, s)
    out = torch.zeros(s["rows"], c["N"], dtype=torch.float64, device=DEV)
    X = (s["Xq"] if c["op"] == "w8" else s["X"])
    if c["op"] == "w8":  # where the packed layout keeps the code of channel n at depth k
        n = torch.arange(c["N"], device=DEV)[:, None]
        d = torch.arange(c["K"], device=DEV)[None, :]
        at = 256 + (n // 16 * (c["K"] // 128) + d // 128) * 2048 + (d % 64 // 16 * 16 + n % 16) * 32 + d % 128 // 64 * 16 + d % 16
        scales_at = -(-(256 + -(-c["N"] // 16) * 16 * c["K"]) // 256) * 256
    first = 0
    for e, count in enumerate(s["counts"]):
        last = first + count
        if count:
            src = s["gather"][first:last].long() // c["k"] if s["gather"] is not None else torch.arange(first, last, device=DEV)
            x = X[src].double()
            if c["op"] == "w8":
                raw = s["blob"][e]
                W = raw.view(torch.int8)[at].double()
                sw = raw[scales_at:scales_at + 4 * c["N"]].clone().view(torch.float32).double()
                y = (x @ W.t().contiguous()) * s["sx"][src].double()[:, None] * sw[None, :]
            else:
                y = x @ s["W"][e].double().t().contiguous()
                if c["op"] == "silu":
                    y = y[:, : c["N"]] * torch.sigmoid(y[:, : c["N"]]) * y[:, c["N"]:]
            out[first:last] = y
        first = last
    return out


def _exact_route(c, s):
    """Only the weights: the ids are whole numbers."""
    x = s["logits"].double().cpu()
    if c["T"] > 4096:
        x = x.to(DEV)
    bias = None if s["bias"] is None else s["bias"].double().to(x.device)
    p = torch.softmax(x, 1) if c["score"] == "softmax" else torch.sigmoid(x)
    p = torch.nan_to_num(p, 0.0)  # a row with every expert masked
    rank = p.clone() if bias is None else p + bias
    if bias is None and c["score"] == "softmax":
        rank = x.clone()
    rank[x == -math.inf] = -math.inf
    if c["groups"] > 1:
        each = rank.view(c["T"], c["groups"], -1)
        two = each.topk(2, dim=2).values
        best = two[..., 0] if bias is None else two[..., 0] + two[..., 1].masked_fill(two[..., 1] == -math.inf, 0.0)
        dropped = best.argsort(dim=1, descending=True, stable=True)[:, c["keep"]:]
        each.scatter_(1, dropped[:, :, None].expand(-1, -1, each.shape[2]), -math.inf)
    best = rank.topk(c["k"], dim=1)
    w = p.gather(1, best.indices).masked_fill(best.values == -math.inf, 0.0)
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return {"ids": None, "w": (w * c["scale"]).to(DEV)}
