"""The mixture-of-experts and 4-bit operators as their callers run them, for measurement.

Five operators:
  route    scores of a router -> the experts of each token, their weights, and
           the plan (offsets, rows, slots) that sorts (token, expert) pairs by
           expert;
  convert  BF16 or FP32 -> MXFP4 (E2M1 elements, one E8M0 scale per 32) and
           back to BF16;
  mx4      y = x . W^T with W in MXFP4, x in BF16 or quantised to MXFP4 too;
  experts  products grouped by expert over ragged rows, plain (fp32 out) or
           gated (silu(gate) * up, BF16 out), weights BF16, UWF1 or MXFP4;
  mlp      route, gated product, down product and the weighted sum over a
           token's experts.

``own`` false: the plain form, elementary torch operations in 32 bits, rounded
once at the end.  ``own`` true: the library's calls.
"""
import math
import random

import torch

own = False
DEV = "cuda:0"


# ---------------------------------------------------------------- cases -----

def listed():
    return [
        # one decoded token's routing: a pure latency call
        {"name": "route_token", "op": "route", "tokens": 1, "experts": 64, "topk": 4, "scoring": "softmax_topk",
         "bf16": False, "pad": 0},
        # a long prompt's routing from BF16 scores, its padded tokens masked to -inf
        {"name": "route_prompt", "op": "route", "tokens": 16001, "experts": 160, "topk": 6, "scoring": "sigmoid",
         "bf16": True, "pad": 500},
        # a few activation rows of an odd block count
        {"name": "convert_rows", "op": "convert", "rows": 37, "cols": 4128, "fp32": True},
        # the 8B gate's weights, converted once at load
        {"name": "convert_gate8b", "op": "convert", "rows": 14336, "cols": 4096, "fp32": False},
        # decode: one token through the 8B gate
        {"name": "mx4_token", "op": "mx4", "batch": 1, "n": 14336, "k": 4096, "act": "bf16"},
        # a ragged decode batch through an odd-sized projection
        {"name": "mx4_batch45", "op": "mx4", "batch": 45, "n": 5001, "k": 8224, "act": "bf16"},
        # a prompt through the 70B gate with its activations in 4 bits as well
        {"name": "mx4_prompt", "op": "mx4", "batch": 1024, "n": 28672, "k": 8192, "act": "mx4"},
        # decode: one token through two of eight 8B-sized experts
        {"name": "experts_token", "op": "experts", "form": "bf16", "gated": True, "tokens": 1, "experts": 8, "topk": 2,
         "n": 14336, "k": 4096, "pad": 0},
        # a decode batch from losslessly compressed experts
        {"name": "experts_uwf1", "op": "experts", "form": "uwf1", "gated": False, "tokens": 24, "experts": 32,
         "topk": 4, "n": 2048, "k": 4096, "pad": 0},
        # a prompt over many small experts
        {"name": "experts_prompt", "op": "experts", "form": "bf16", "gated": True, "tokens": 4096, "experts": 64,
         "topk": 8, "n": 1408, "k": 2048, "pad": 0},
        # a decode batch through the whole layer with 4-bit experts
        {"name": "mlp_decode", "op": "mlp", "form": "mx4", "tokens": 37, "experts": 32, "topk": 4, "n": 2048,
         "k": 4096, "pad": 3},
        # a ragged prompt through the whole layer
        {"name": "mlp_prompt", "op": "mlp", "form": "bf16", "tokens": 3001, "experts": 64, "topk": 6, "n": 1408,
         "k": 2048, "pad": 41},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["route", "convert", "mx4", "experts", "experts", "mlp"])
    if op == "route":
        tokens = _log(rng, 1, 16000)
        e = rng.randint(4, 256)
        return {"op": op, "tokens": tokens, "experts": e, "topk": rng.randint(1, min(8, e)),
                "scoring": rng.choice(["softmax", "softmax_topk", "sigmoid"]), "bf16": rng.random() < 0.5,
                "pad": rng.randint(0, tokens // 3)}
    if op == "convert":
        return {"op": op, "rows": _log(rng, 1, 12000), "cols": 32 * _log(rng, 2, 150), "fp32": rng.random() < 0.5}
    if op == "mx4":
        n, k = _log(rng, 200, 16000), 32 * _log(rng, 8, 256)
        return {"op": op, "batch": _log(rng, 1, 1100), "n": n, "k": k, "act": rng.choice(["bf16", "mx4"])}
    form = rng.choice(["bf16", "mx4", "uwf1"])
    e = rng.choice([4, 8, 16, 24, 32, 60])
    c = {"op": op, "form": form, "tokens": _log(rng, 1, 3000), "experts": e, "topk": rng.randint(1, min(e, 6)),
         "n": 64 * _log(rng, 2, 24), "k": 64 * _log(rng, 4, 32)}
    c["pad"] = rng.randint(0, c["tokens"] // 4)
    if op == "experts":
        c["gated"] = rng.random() < 0.5
        if form != "uwf1":   # UWF1 rows are whole groups of 64; the other forms take any N
            c["n"] += rng.choice([0, 1, 8, 33])
    return c


def _active(c):
    """Experts that receive at least one token, on average (even routing)."""
    t = c["tokens"] - c["pad"]
    return c["experts"] * (1.0 - (1.0 - c["topk"] / c["experts"]) ** t)


_BYTES = {"bf16": 2.0, "mx4": 0.5 + 1 / 32, "uwf1": 1.5}   # per weight, as the caller holds it


def work(c):
    op = c["op"]
    if op == "route":
        pairs = c["tokens"] * c["topk"]
        return {"bytes": c["tokens"] * c["experts"] * (2 if c["bf16"] else 4) + pairs * 16 + 4 * (c["experts"] + 1),
                "flops": 4.0 * c["tokens"] * c["experts"]}
    if op == "convert":
        e = c["rows"] * c["cols"]
        return {"bytes": e * ((4 if c["fp32"] else 2) + 2 * (0.5 + 1 / 32) + 2), "flops": 4.0 * e}
    if op == "mx4":
        b, n, k = c["batch"], c["n"], c["k"]
        return {"bytes": n * k * _BYTES["mx4"] + 2 * b * k + 4 * b * n, "flops": 2.0 * b * n * k}
    t = c["tokens"] - c["pad"]
    s, n, k = t * c["topk"], c["n"], c["k"]
    w = _active(c) * n * k * _BYTES[c["form"]]
    if op == "experts":
        m = 2 if c["gated"] else 1
        return {"bytes": m * w + 2 * t * k + s * n * (2 if c["gated"] else 4), "flops": 2.0 * m * s * n * k}
    return {"bytes": 3 * w + 2 * t * k + 2 * c["tokens"] * k + 4 * c["tokens"] * c["experts"],
            "flops": 6.0 * s * n * k}


# --------------------------------------------------------------- inputs -----

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def _logits(g, c, dtype=torch.float32):
    """Router scores: some experts are liked more than others; padded tokens are -inf throughout."""
    liked = torch.randn(c["experts"], generator=g, device=DEV) * 0.5
    x = torch.randn(c["tokens"], c["experts"], generator=g, device=DEV) * 1.5 + liked
    if c["pad"]:
        x[torch.randperm(c["tokens"], generator=g, device=DEV)[:c["pad"]]] = float("-inf")
    return x.to(dtype)


def _inputs(c, seed):
    g = _gen(seed)
    op = c["op"]
    if op == "route":
        return {"logits": _logits(g, c, torch.bfloat16 if c["bf16"] else torch.float32)}
    if op == "convert":
        spread = torch.exp2(torch.randn(c["rows"], 1, generator=g, device=DEV) * 2)
        x = torch.randn(c["rows"], c["cols"], generator=g, device=DEV) * 0.02 * spread
        return {"x": x if c["fp32"] else x.to(torch.bfloat16)}
    if op == "mx4":
        e, s = _quantise(_normal(g, c["n"], c["k"], scale=0.02))
        return {"elem": e, "scale": s, "x": _normal(g, c["batch"], c["k"])}
    s = {"x": _normal(g, c["tokens"], c["k"]), "logits": _logits(g, c)}
    names = [("gate", c["n"], c["k"])]
    if op == "mlp" or c["gated"]:
        names.append(("up", c["n"], c["k"]))
    if op == "mlp":
        names.append(("down", c["k"], c["n"]))
    for name, n, k in names:
        w = _normal(g, c["experts"], n, k, scale=0.02)
        s[name] = _quantise(w.view(-1, k)) if c["form"] == "mx4" else w
    if op == "experts":
        s["plan"] = _plan(_route(s["logits"], c["topk"], "softmax_topk")[0], c["experts"])
        s["counts"] = s["plan"][0].tolist()   # a caller of the plain form splits its rows on the host
        s["pairs"] = s["counts"][-1]
    return s


def _scale_stride(k):
    return 4 * ((k + 127) // 128)


def prepare(c, seed):
    s = dict(_inputs(c, seed), case=c)
    op = c["op"]
    if not own:
        return s
    from decode_gemm_exp_amd import uw
    if op == "route":
        s["routing"] = uw.Routing(c["tokens"], c["experts"], c["topk"], DEV)
    elif op == "convert":
        s["elem"] = torch.empty(c["rows"], c["cols"] // 2, dtype=torch.uint8, device=DEV)
        s["scale"] = torch.empty(c["rows"], _scale_stride(c["cols"]), dtype=torch.uint8, device=DEV)
        s["out"] = torch.empty(c["rows"], c["cols"], dtype=torch.bfloat16, device=DEV)
    elif op == "mx4":
        s["y"] = torch.empty(c["batch"], c["n"], dtype=torch.float32, device=DEV)
        s["act"] = uw.ACT_MX4 if c["act"] == "mx4" else uw.ACT_BF16
        s["ws"] = torch.empty(max(16, uw.uw_workspace_size_mx4(c["n"], c["k"], c["batch"], s["act"])),
                              dtype=torch.uint8, device=DEV)
    else:
        for name in ("gate", "up", "down"):
            if name in s:
                n, k = (c["k"], c["n"]) if name == "down" else (c["n"], c["k"])
                s["h_" + name] = _handle(uw, c, s[name], n, k)
        s["routing"] = uw.Routing(c["tokens"], c["experts"], c["topk"], DEV)
        if op == "experts":
            offsets, rows, slots = s["plan"]
            s["routing"].offsets.copy_(offsets)
            s["routing"].rows.copy_(rows)
            s["routing"].slots.copy_(slots)
            s["y"] = torch.zeros(c["tokens"] * c["topk"], c["n"], device=DEV,
                                 dtype=torch.bfloat16 if c["gated"] else torch.float32)
        else:
            s["y"] = torch.empty(c["tokens"], c["k"], dtype=torch.bfloat16, device=DEV)
            s["ws"] = torch.empty(max(16, uw.uw_workspace_size_expert_mlp(s["h_gate"], s["h_down"], c["tokens"],
                                                                          c["topk"])), dtype=torch.uint8, device=DEV)
    return s


def _handle(uw, c, w, n, k):
    """The experts' weights as a server keeps them."""
    if c["form"] == "mx4":
        return uw.uw_experts_mx4(w[0], w[1], c["experts"], n, k)
    if c["form"] == "bf16":
        return uw.uw_experts_bf16(w, c["experts"], n, k)
    ms = []
    for e in range(c["experts"]):
        m = uw.uw_compress(w[e], n, k)
        uw.uw_transcode_palette(m, None)
        uw.uw_drop_stream(m)
        ms.append(m)
    return uw.uw_experts_uwf1(ms)


# ------------------------------------------------------------- plain form ---

def _route(logits, topk, scoring):
    """ids (-1: none) and weights; the k largest selectable scores, ties to the lower index."""
    l = logits.float()
    dead = torch.isnan(l) | (l == float("-inf"))
    key = torch.where(dead, float("-inf"), l)
    top, ids = torch.sort(key, dim=1, descending=True, stable=True)
    top, ids = top[:, :topk], ids[:, :topk].to(torch.int32)
    none = top == float("-inf")
    if scoring == "sigmoid":
        w = torch.where(none, 0.0, 1.0 / (1.0 + torch.exp(-top)))
        w = w / w.sum(1, keepdim=True).clamp_min(torch.finfo(torch.float32).tiny)
    else:
        high = torch.where(top[:, :1] == float("-inf"), 0.0, top[:, :1])
        w = torch.where(none, 0.0, torch.exp(top - high))
        total = torch.exp(key - high).sum(1, keepdim=True) if scoring == "softmax" else w.sum(1, keepdim=True)
        w = w / total.clamp_min(torch.finfo(torch.float32).tiny)
    return torch.where(none, -1, ids), torch.where(none, 0.0, w)


def _plan(ids, experts):
    """offsets [E+1], rows [pairs] (slot -> token), slots [pairs] (pair -> slot, -1 none)."""
    topk = ids.shape[1]
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, experts, flat)
    order = torch.sort(key, stable=True)[1]
    counts = (key[:, None] == torch.arange(experts, device=flat.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    place = torch.arange(flat.numel(), device=flat.device)
    rows = torch.where(place < offsets[-1], order // topk, 0).to(torch.int32)
    slots = torch.empty_like(flat).scatter_(0, order, place)
    return offsets, rows, torch.where(flat < 0, -1, slots).to(torch.int32).view(ids.shape)


def _e2m1(a):
    """Non-negative values -> the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even code."""
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.clamp(torch.round(a / step) * step, max=6.0)


def _mx4_blocks(x):
    """(values before scaling, exponent of each block's scale); finite inputs."""
    b = x.float().reshape(x.shape[0], -1, 32)
    _, e = torch.frexp(b.abs().amax(2, keepdim=True))   # amax = f 2^e, f in [.5, 1): floor(log2) = e - 1
    e = torch.where(b.abs().amax(2, keepdim=True) == 0, -127, (e - 3).clamp(-127, 125))
    v = torch.ldexp(torch.ldexp(b, -(e // 2)), -(e - e // 2))
    return torch.copysign(_e2m1(v.abs()), v), e


def _mx4_values(x):
    v, e = _mx4_blocks(x)
    return torch.ldexp(torch.ldexp(v, e // 2), e - e // 2).reshape(x.shape)


def _quantise(x):
    """Packed elements [rows][cols/2] and scales [rows][stride] of finite x."""
    v, e = _mx4_blocks(x)
    a = v.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(v).to(torch.uint8) << 3)).reshape(x.shape[0], -1, 2)
    scale = torch.zeros(x.shape[0], _scale_stride(x.shape[1]), dtype=torch.uint8, device=x.device)
    scale[:, :x.shape[1] // 32] = (e.reshape(x.shape[0], -1) + 127).to(torch.uint8)
    return code[:, :, 0] | (code[:, :, 1] << 4), scale


def _table(dtype):
    t = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(t + [-v for v in t], dtype=dtype, device=DEV)


def _dequantise(elem, scale):
    r, half = elem.shape
    t = _table(torch.float32)
    v = torch.stack([t[(elem & 15).int()], t[(elem >> 4).int()]], 2).reshape(r, -1, 32)
    e = scale[:, :v.shape[1], None].int() - 127
    return torch.ldexp(v, e).reshape(r, 2 * half)


def _expert(s, name, e, dtype=torch.float32):
    w = s[name]
    if s["case"]["form"] != "mx4":
        return w[e].to(dtype)
    n = w[0].shape[0] // s["case"]["experts"]
    return _dequantise(w[0][e * n:(e + 1) * n], w[1][e * n:(e + 1) * n]).to(dtype)


def _silu(g):
    return g / (1.0 + torch.exp(-g))


def _plain_experts(s, counts, rows, gated, n):
    """[pairs, N] in fp32, rows past the last pair zero."""
    out = torch.zeros(rows.numel(), n, device=DEV)
    for e in range(len(counts) - 1):
        a, b = counts[e], counts[e + 1]
        if a < b:
            x = s["x"][rows[a:b]].float()
            y = x @ _expert(s, "gate", e).t()
            out[a:b] = _silu(y) * (x @ _expert(s, "up", e).t()) if gated else y
    return out


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "route":
        ids, w = _route(s["logits"], c["topk"], c["scoring"])
        return (ids, w) + _plan(ids, c["experts"])
    if op == "convert":
        return _mx4_values(s["x"]).to(torch.bfloat16)
    if op == "mx4":
        x = _mx4_values(s["x"]) if c["act"] == "mx4" else s["x"].float()
        return x @ _dequantise(s["elem"], s["scale"]).t()
    if op == "experts":
        y = _plain_experts(s, s["counts"], s["plan"][1], c["gated"], c["n"])
        return y.to(torch.bfloat16) if c["gated"] else y
    ids, w = _route(s["logits"], c["topk"], "softmax_topk")
    offsets, rows, slots = _plan(ids, c["experts"])
    counts = offsets.tolist()
    h = _plain_experts(s, counts, rows, True, c["n"])
    d = torch.zeros(rows.numel(), c["k"], device=DEV)
    for e in range(c["experts"]):
        a, b = counts[e], counts[e + 1]
        if a < b:
            d[a:b] = h[a:b] @ _expert(s, "down", e).t()
    y = torch.where(slots[..., None] < 0, 0.0, d[slots.clamp_min(0).long()] * w[..., None])
    return y.sum(1).to(torch.bfloat16)


# -------------------------------------------------------- the library's -----

def run(s):
    if not own:
        return _run_plain(s)
    from decode_gemm_exp_amd import uw
    c = s["case"]
    op = c["op"]
    if op == "route":
        r = s["routing"]
        uw.uw_route_experts(s["logits"], r, c["scoring"])
        return r.ids, r.weights, r.offsets, r.rows, r.slots
    if op == "convert":
        uw.uw_quantize_mx4(s["x"], s["elem"], s["scale"])
        uw.uw_dequantize_mx4(s["elem"], s["scale"], s["out"])
        return s["out"]
    if op == "mx4":
        uw.uw_matmul_mx4(s["elem"], s["scale"], s["x"], s["y"], s["ws"], s["act"])
        return s["y"]
    r = s["routing"]
    if op == "experts":
        if c["gated"]:
            uw.uw_matmul_experts_gated(s["h_gate"], s["h_up"], r.offsets, r.rows, s["x"], s["y"])
        else:
            uw.uw_matmul_experts(s["h_gate"], r.offsets, r.rows, s["x"], s["y"])
        return s["y"]
    uw.uw_route_experts(s["logits"], r, "softmax_topk")
    uw.uw_expert_mlp(s["h_gate"], s["h_up"], s["h_down"], r, s["x"], s["y"], s["ws"])
    return s["y"]


# ------------------------------------------------------------- in 64 bits ---

def _exact_values(x):
    """MXFP4 of x by its definition: the scale from log2's floor, the element by counting the midpoints below."""
    b = x.double().unflatten(1, (-1, 32))
    amax = b.abs().max(2, keepdim=True).values
    e = (torch.frexp(amax)[1].double() - 3).clamp(-127.0, 125.0)
    e = torch.where(amax > 0, e, -127.0)
    q = (b * torch.exp2(-e)).abs()
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=x.device)
    code = torch.zeros_like(q, dtype=torch.int64)
    for i, mid in enumerate([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]):
        code += (q >= mid) if i % 2 else (q > mid)   # a tie goes to the even code
    return (torch.where(b < 0, -grid[code], grid[code]) * torch.exp2(e)).flatten(1)


def _exact_weight(s, name, e, n):
    c = s["case"]
    if c["form"] != "mx4":
        return s[name][e].double()
    return _exact_mx4(s[name][0][e * n:(e + 1) * n], s[name][1][e * n:(e + 1) * n])


def _exact_mx4(elem, scale):
    lo, hi = elem.long() & 15, elem.long() >> 4
    codes = torch.cat([lo[:, :, None], hi[:, :, None]], 2).flatten(1)
    v = _table(torch.float64)[codes]
    s = torch.exp2(scale.double() - 127.0)[:, :elem.shape[1] // 16]
    return v * s.repeat_interleave(32, dim=1)


def _exact_route(c, logits):
    l = logits.double().nan_to_num(nan=float("-inf"), posinf=float("inf"), neginf=float("-inf"))
    t, n = l.shape
    # the lower index first among equals: order by (-score, index)
    order = torch.argsort(-l, dim=1, stable=True)[:, :c["topk"]]
    top = l.gather(1, order)
    live = top > float("-inf")
    if c.get("scoring", "softmax_topk") == "sigmoid":
        w = torch.sigmoid(top) * live
        w = w / w.sum(1, keepdim=True)
    elif c.get("scoring") == "softmax":
        w = torch.softmax(l, 1).gather(1, order)
    else:
        w = torch.softmax(top, 1)
    ids = torch.where(live, order, -1)
    return ids, torch.where(live, w, 0.0)


def _exact_plan(c, ids):
    pairs = [(e, p) for p, e in enumerate(ids.reshape(-1).tolist()) if e >= 0]
    pairs.sort()
    offsets = [0] * (c["experts"] + 1)
    for e, _ in pairs:
        offsets[e + 1] += 1
    for e in range(c["experts"]):
        offsets[e + 1] += offsets[e]
    rows = [p // c["topk"] for _, p in pairs] + [0] * (ids.numel() - len(pairs))
    slots = [-1] * ids.numel()
    for i, (_, p) in enumerate(pairs):
        slots[p] = i
    as_int = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    return as_int(offsets), as_int(rows), as_int(slots).view(ids.shape)


def exact(c, seed):
    if 6.0 * work(c)["flops"] > 2e13:   # 64-bit products of this size take too long
        return None
    s = dict(_inputs(c, seed), case=c)
    op = c["op"]
    if op == "route":
        ids, w = _exact_route(c, s["logits"])
        return (ids.to(torch.int32), w) + _exact_plan(c, ids)
    if op == "convert":
        return _exact_values(s["x"])
    if op == "mx4":
        x = _exact_values(s["x"]) if c["act"] == "mx4" else s["x"].double()
        return torch.matmul(x, _exact_mx4(s["elem"], s["scale"]).transpose(0, 1))
    ids, w = _exact_route({"topk": c["topk"]}, s["logits"])
    offsets, rows, slots = _exact_plan(c, ids)
    gated = op == "mlp" or c["gated"]
    n, k = c["n"], c["k"]
    h = torch.zeros(ids.numel(), n, dtype=torch.float64, device=DEV)
    d = torch.zeros(ids.numel(), k if op == "mlp" else 1, dtype=torch.float64, device=DEV)
    for e in range(c["experts"]):
        mine = (ids == e).any(1).nonzero().flatten()   # an expert's tokens; a token has an expert once
        if mine.numel() == 0:
            continue
        at = slots[mine][ids[mine] == e].long()
        x = s["x"][mine].double()
        g = torch.matmul(x, _exact_weight(s, "gate", e, n).transpose(0, 1))
        if gated:
            g = g * torch.sigmoid(g) * torch.matmul(x, _exact_weight(s, "up", e, n).transpose(0, 1))
        h[at] = g
        if op == "mlp":
            d[at] = torch.matmul(g, _exact_weight(s, "down", e, k).transpose(0, 1))
    if op == "experts":
        return h
    y = torch.zeros(c["tokens"], k, dtype=torch.float64, device=DEV)
    for j in range(c["topk"]):
        y += torch.where(slots[:, j:j + 1] >= 0, d[slots[:, j].long().clamp(min=0)] * w[:, j:j + 1], 0.0)
    return y
