"""The FP8 operators and the few-token expert layer as their callers run them, for measurement.

Four operators:
  convert  BF16 or FP32 -> E4M3 with one FP32 scale per block of 1 x 128
           (activations) or 128 x 128 (weights), and back to BF16;
  product  y = x . W^T with W in E4M3 and a scale per 128 x 128 block, x in
           BF16 or converted with a scale per 1 x 128 block;
  experts  products grouped by expert over ragged rows from such weights,
           plain (fp32 out) or gated (silu(gate) * up, BF16 out);
  layer    a whole mixture-of-experts layer for a few tokens: router's choice,
           gated product, down product and the weighted sum, weights BF16,
           UWF1, MXFP4 or FP8.

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
        # activations of a decode batch, their last block a quarter
        {"name": "convert_rows", "op": "convert", "rows": 45, "cols": 8224, "block_rows": 1, "fp32": False},
        # the 8B gate's weights, converted once at load
        {"name": "convert_gate8b", "op": "convert", "rows": 14336, "cols": 4096, "block_rows": 128, "fp32": False},
        # decode: one token through the 8B gate
        {"name": "product_token", "op": "product", "batch": 1, "n": 14336, "k": 4096, "act": "bf16"},
        # a ragged decode batch through an odd-sized projection, activations in 8 bits as well
        {"name": "product_batch13", "op": "product", "batch": 13, "n": 5001, "k": 8224, "act": "fp8"},
        # a short prompt through the 8B down projection, activations kept as they are
        {"name": "product_rows333", "op": "product", "batch": 333, "n": 4096, "k": 14336, "act": "bf16"},
        # a prompt through the 70B gate, both operands in 8 bits
        {"name": "product_prompt", "op": "product", "batch": 1024, "n": 28672, "k": 8192, "act": "fp8"},
        # a decode batch over 32 experts
        {"name": "experts_decode", "op": "experts", "gated": True, "tokens": 24, "experts": 32, "topk": 4, "n": 2048,
         "k": 4096, "pad": 0},
        # a ragged prompt over many small experts
        {"name": "experts_prompt", "op": "experts", "gated": False, "tokens": 3001, "experts": 64, "topk": 6,
         "n": 1408, "k": 2048, "pad": 41},
        # one token through eight of 64 small experts: mostly latency
        {"name": "layer_token", "op": "layer", "form": "fp8", "tokens": 1, "experts": 64, "topk": 8, "n": 1408,
         "k": 2048, "scoring": "softmax", "bias": False, "bf16": False, "pad": 0},
        # one token through two of eight 8B-sized experts
        {"name": "layer_token8b", "op": "layer", "form": "bf16", "tokens": 1, "experts": 8, "topk": 2, "n": 14336,
         "k": 4096, "scoring": "softmax_topk", "bias": False, "bf16": True, "pad": 0},
        # five sequences, one of them ended, over losslessly compressed experts
        {"name": "layer_uwf1", "op": "layer", "form": "uwf1", "tokens": 5, "experts": 32, "topk": 4, "n": 2048,
         "k": 4096, "scoring": "softmax_topk", "bias": False, "bf16": False, "pad": 1},
        # a decode batch over many 4-bit experts whose router is balanced by a bias
        {"name": "layer_batch16", "op": "layer", "form": "mx4", "tokens": 16, "experts": 160, "topk": 6, "n": 1408,
         "k": 2048, "scoring": "sigmoid", "bias": True, "bf16": True, "pad": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["convert", "product", "product", "experts", "layer", "layer"])
    if op == "convert":
        return {"op": op, "rows": _log(rng, 1, 12000), "cols": 32 * _log(rng, 1, 150),
                "block_rows": rng.choice([1, 128]), "fp32": rng.random() < 0.5}
    if op == "product":
        return {"op": op, "batch": _log(rng, 1, 1100), "n": _log(rng, 100, 16000), "k": 32 * _log(rng, 2, 256),
                "act": rng.choice(["bf16", "fp8"])}
    e = rng.choice([4, 8, 16, 24, 32, 60])
    c = {"op": op, "experts": e, "topk": rng.randint(1, min(e, 6)), "k": 64 * _log(rng, 2, 32)}
    if op == "experts":
        c["tokens"] = _log(rng, 1, 3000)
        c["gated"] = rng.random() < 0.5
        c["n"] = 64 * _log(rng, 2, 24) + rng.choice([0, 1, 8, 33])
        c["pad"] = rng.randint(0, c["tokens"] // 4)
        return c
    c["form"] = rng.choice(["bf16", "uwf1", "mx4", "fp8"])
    c["tokens"] = rng.randint(1, 16)
    c["n"] = 64 * _log(rng, 2, 24)
    if c["form"] != "uwf1":   # UWF1 rows are whole groups of 64; the other forms take blocks of 32
        c["n"] += rng.choice([0, 32])
        c["k"] += rng.choice([0, 32])
    c["scoring"] = rng.choice(["softmax", "softmax_topk", "sigmoid"])
    c["bias"] = rng.random() < 0.5
    c["bf16"] = rng.random() < 0.5
    c["pad"] = rng.randint(0, c["tokens"] // 4)
    return c


def _active(c):
    """Experts that receive at least one token, on average (even routing)."""
    t = c["tokens"] - c["pad"]
    return c["experts"] * (1.0 - (1.0 - c["topk"] / c["experts"]) ** t)


_BYTES = {"bf16": 2.0, "mx4": 0.5 + 1 / 32, "uwf1": 1.5, "fp8": 1.0 + 4 / 16384}   # per weight, as the caller holds it


def work(c):
    op = c["op"]
    if op == "convert":
        e = c["rows"] * c["cols"]
        return {"bytes": e * ((4 if c["fp32"] else 2) + 2 + 2) + 8 * e / (128 * c["block_rows"]), "flops": 4.0 * e}
    if op == "product":
        b, n, k = c["batch"], c["n"], c["k"]
        return {"bytes": n * k * _BYTES["fp8"] + 2 * b * k + 4 * b * n, "flops": 2.0 * b * n * k}
    t = c["tokens"] - c["pad"]
    s, n, k = t * c["topk"], c["n"], c["k"]
    w = _active(c) * n * k * _BYTES["fp8" if op == "experts" else c["form"]]
    if op == "experts":
        m = 2 if c["gated"] else 1
        return {"bytes": m * w + 2 * t * k + s * n * (2 if c["gated"] else 4), "flops": 2.0 * m * s * n * k}
    return {"bytes": 3 * w + 2 * t * k + 2 * c["tokens"] * k + (2 if c["bf16"] else 4) * c["tokens"] * c["experts"]
            + 8 * c["tokens"] * c["topk"], "flops": 6.0 * s * n * k}


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


def _weights(g, c, form, count, n, k):
    """count matrices [n][k] stacked along rows, as the form keeps them."""
    w = _normal(g, count, n, k, scale=0.02)
    if form == "mx4":
        return _quantise_mx4(w.view(-1, k))
    if form != "fp8":
        return w
    elem = torch.empty(count, n, k, dtype=torch.uint8, device=DEV)
    scale = torch.empty(count, (n + 127) // 128, (k + 127) // 128, device=DEV)
    for e in range(count):   # a matrix at a time: rows of blocks begin anew in each
        v, s = _fp8(w[e], 128)
        elem[e], scale[e] = v.to(torch.float8_e4m3fn).view(torch.uint8), s
    return elem, scale


def _inputs(c, seed):
    g = _gen(seed)
    op = c["op"]
    if op == "convert":
        spread = torch.exp2(torch.randn(c["rows"], 1, generator=g, device=DEV) * 2)
        x = torch.randn(c["rows"], c["cols"], generator=g, device=DEV) * 0.02 * spread
        return {"x": x if c["fp32"] else x.to(torch.bfloat16)}
    if op == "product":
        elem, scale = _weights(g, c, "fp8", 1, c["n"], c["k"])
        loud = torch.exp2(torch.randn(c["k"], generator=g, device=DEV))   # some channels are louder
        x = (torch.randn(c["batch"], c["k"], generator=g, device=DEV) * loud).to(torch.bfloat16)
        return {"elem": elem[0], "scale": scale[0], "x": x}
    s = {"x": _normal(g, c["tokens"], c["k"])}
    s["logits"] = _logits(g, c, torch.bfloat16 if c.get("bf16") else torch.float32)
    s["bias"] = torch.randn(c["experts"], generator=g, device=DEV) * 0.2 if c.get("bias") else None
    names = [("gate", c["n"], c["k"])]
    if op == "layer" or c["gated"]:
        names.append(("up", c["n"], c["k"]))
    if op == "layer":
        names.append(("down", c["k"], c["n"]))
    for name, n, k in names:
        s[name] = _weights(g, c, "fp8" if op == "experts" else c["form"], c["experts"], n, k)
    if op == "experts":
        s["plan"] = _plan(_route(s["logits"], None, c["topk"], "softmax_topk")[0], c["experts"])
        s["counts"] = s["plan"][0].tolist()   # a caller of the plain form splits its rows on the host
    return s


def _scale_stride(k):
    return 4 * ((k + 127) // 128)


def prepare(c, seed):
    s = dict(_inputs(c, seed), case=c)
    op = c["op"]
    if not own:
        return s
    from decode_gemm_exp_amd import uw
    if op == "convert":
        s["elem"] = torch.empty(c["rows"], c["cols"], dtype=torch.float8_e4m3fn, device=DEV)
        s["scale"] = torch.empty(uw.fp8_scale_shape(c["rows"], c["cols"], c["block_rows"]), device=DEV)
        s["out"] = torch.empty(c["rows"], c["cols"], dtype=torch.bfloat16, device=DEV)
    elif op == "product":
        s["y"] = torch.empty(c["batch"], c["n"], dtype=torch.float32, device=DEV)
        s["act"] = uw.ACT_FP8 if c["act"] == "fp8" else uw.ACT_BF16
        s["ws"] = torch.empty(max(16, uw.uw_workspace_size_fp8(c["n"], c["k"], c["batch"], s["act"])),
                              dtype=torch.uint8, device=DEV)
    else:
        for name in ("gate", "up", "down"):
            if name in s:
                n, k = (c["k"], c["n"]) if name == "down" else (c["n"], c["k"])
                s["h_" + name] = _handle(uw, "fp8" if op == "experts" else c["form"], s[name], c["experts"], n, k)
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
            s["ws"] = torch.empty(max(16, uw.uw_workspace_size_expert_layer(s["h_gate"], s["h_down"], c["tokens"],
                                                                            c["topk"])), dtype=torch.uint8, device=DEV)
    return s


def _handle(uw, form, w, count, n, k):
    """The experts' weights as a server keeps them."""
    if form == "fp8":
        return uw.uw_experts_fp8(w[0], w[1], count, n, k)
    if form == "mx4":
        return uw.uw_experts_mx4(w[0], w[1], count, n, k)
    if form == "bf16":
        return uw.uw_experts_bf16(w, count, n, k)
    ms = []
    for e in range(count):
        m = uw.uw_compress(w[e], n, k)
        uw.uw_transcode_palette(m, None)
        uw.uw_drop_stream(m)
        ms.append(m)
    return uw.uw_experts_uwf1(ms)


# ------------------------------------------------------------- plain form ---

def _blocks(x, rows):
    """x padded to whole blocks: [row blocks][rows][column blocks][128]."""
    r, c = -x.shape[0] % rows, -x.shape[1] % 128
    x = torch.nn.functional.pad(x, (0, c, 0, r))
    return x.reshape(x.shape[0] // rows, rows, x.shape[1] // 128, 128)


def _fp8(x, rows):
    """(E4M3 values before scaling, scale of each block); finite inputs."""
    b = _blocks(x.float(), rows)
    top = b.abs().amax((1, 3), keepdim=True).clamp_min(2.0 ** -110)
    most = torch.full_like(top, 448.0)         # (a tensor: torch multiplies by the inverse of a plain number)
    v = b * (most / top)
    _, e = torch.frexp(v)                      # |v| = f 2^e, f in [.5, 1)
    step = torch.exp2((e - 1).clamp_min(-6) - 3.0)
    v = (torch.round(v / step) * step).clamp(-448.0, 448.0)   # ties to even
    v = v.reshape(b.shape[0] * rows, -1)[:x.shape[0], :x.shape[1]]
    return v, (top / most)[:, 0, :, 0]


def _scaled(v, scale, rows):
    """Values times their block's scale."""
    full = scale.repeat_interleave(rows, 0)[:v.shape[0]].repeat_interleave(128, 1)[:, :v.shape[1]]
    return v * full


def _e4m3(elem):
    return elem.view(torch.float8_e4m3fn).float()


def _route(logits, bias, topk, scoring):
    """ids (-1: none) and weights; the k largest selectable keys, ties to the lower index."""
    l = logits.float()
    key = l if bias is None else l + bias
    dead = torch.isnan(l) | (l == float("-inf"))
    key = torch.where(dead, float("-inf"), key)
    _, ids = torch.sort(key, dim=1, descending=True, stable=True)
    ids = ids[:, :topk]
    none = key.gather(1, ids) == float("-inf")
    top = torch.where(none, float("-inf"), l.gather(1, ids))
    if scoring == "sigmoid":
        w = torch.where(none, 0.0, 1.0 / (1.0 + torch.exp(-top)))
        w = w / w.sum(1, keepdim=True).clamp_min(torch.finfo(torch.float32).tiny)
    else:
        live = torch.where(dead, float("-inf"), l)
        high = live.amax(1, keepdim=True)
        high = torch.where(high == float("-inf"), 0.0, high)
        w = torch.where(none, 0.0, torch.exp(top - high))
        total = torch.exp(live - high).sum(1, keepdim=True) if scoring == "softmax" else w.sum(1, keepdim=True)
        w = w / total.clamp_min(torch.finfo(torch.float32).tiny)
    return torch.where(none, -1, ids).to(torch.int32), torch.where(none, 0.0, w)


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


def _quantise_mx4(x):
    """MXFP4 elements [rows][cols/2] and scales [rows][stride] of finite x (inputs only)."""
    b = x.float().reshape(x.shape[0], -1, 32)
    top = b.abs().amax(2, keepdim=True)
    _, e = torch.frexp(top)
    e = torch.where(top == 0, -127, (e - 3).clamp(-127, 125))
    v = torch.ldexp(b, -e)
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.clamp(torch.round(a / step) * step, max=6.0)
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(v).to(torch.uint8) << 3)).reshape(x.shape[0], -1, 2)
    scale = torch.zeros(x.shape[0], _scale_stride(x.shape[1]), dtype=torch.uint8, device=x.device)
    scale[:, :x.shape[1] // 32] = (e.reshape(x.shape[0], -1) + 127).to(torch.uint8)
    return code[:, :, 0] | (code[:, :, 1] << 4), scale


def _table(dtype):
    t = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    return torch.tensor(t + [-v for v in t], dtype=dtype, device=DEV)


def _mx4(elem, scale):
    r, half = elem.shape
    t = _table(torch.float32)
    v = torch.stack([t[(elem & 15).int()], t[(elem >> 4).int()]], 2).reshape(r, -1, 32)
    return torch.ldexp(v, scale[:, :v.shape[1], None].int() - 127).reshape(r, 2 * half)


def _expert(s, name, e):
    w, c = s[name], s["case"]
    form = "fp8" if c["op"] == "experts" else c["form"]
    if form == "fp8":
        return _scaled(_e4m3(w[0][e]), w[1][e], 128)
    if form == "mx4":
        n = w[0].shape[0] // c["experts"]
        return _mx4(w[0][e * n:(e + 1) * n], w[1][e * n:(e + 1) * n])
    return w[e].float()


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
    if op == "convert":
        v, scale = _fp8(s["x"], c["block_rows"])
        return scale, _scaled(v, scale, c["block_rows"]).to(torch.bfloat16)
    if op == "product":
        x = _scaled(*_fp8(s["x"], 1), 1) if c["act"] == "fp8" else s["x"].float()
        return x @ _scaled(_e4m3(s["elem"]), s["scale"], 128).t()
    if op == "experts":
        y = _plain_experts(s, s["counts"], s["plan"][1], c["gated"], c["n"])
        return y.to(torch.bfloat16) if c["gated"] else y
    ids, w = _route(s["logits"], s["bias"], c["topk"], c["scoring"])
    offsets, rows, slots = _plan(ids, c["experts"])
    counts = offsets.tolist()
    h = _plain_experts(s, counts, rows, True, c["n"])
    d = torch.zeros(rows.numel(), c["k"], device=DEV)
    for e in range(c["experts"]):
        a, b = counts[e], counts[e + 1]
        if a < b:
            d[a:b] = h[a:b] @ _expert(s, "down", e).t()
    y = torch.where(slots[..., None] < 0, 0.0, d[slots.clamp_min(0).long()] * w[..., None])
    return ids, w, y.sum(1).to(torch.bfloat16)


# -------------------------------------------------------- the library's -----

def run(s):
    if not own:
        return _run_plain(s)
    from decode_gemm_exp_amd import uw
    c = s["case"]
    op = c["op"]
    if op == "convert":
        uw.uw_quantize_fp8(s["x"], s["elem"], s["scale"], c["block_rows"])
        uw.uw_dequantize_fp8(s["elem"], s["scale"], s["out"], c["block_rows"])
        return s["scale"], s["out"]
    if op == "product":
        uw.uw_matmul_fp8(s["elem"], s["scale"], s["x"], s["y"], s["ws"], s["act"])
        return s["y"]
    r = s["routing"]
    if op == "experts":
        if c["gated"]:
            uw.uw_matmul_experts_gated(s["h_gate"], s["h_up"], r.offsets, r.rows, s["x"], s["y"])
        else:
            uw.uw_matmul_experts(s["h_gate"], r.offsets, r.rows, s["x"], s["y"])
        return s["y"]
    uw.uw_expert_layer(s["h_gate"], s["h_up"], s["h_down"], s["logits"], r, s["x"], s["y"], s["ws"], c["scoring"],
                       s["bias"])
    return r.ids, r.weights, s["y"]


# ------------------------------------------------------------- in 64 bits ---

def _exact_fp8(x, rows):
    """x's values and scales by the definition: scale and its inverse are FP32 numbers by it, and the scaled value
    is one before it is rounded to E4M3; block by block of columns."""
    x = x.double()
    parts, scales = [], []
    for k in range(0, x.shape[1], 128):
        b = x[:, k:k + 128]
        top = torch.stack([r.abs().max() for r in b.split(rows)]) if rows > 1 else b.abs().max(1).values
        top = top.clamp(min=2.0 ** -110)
        most = torch.full_like(top, 448.0)
        inv, scale = (most / top).float().double(), (top / most).float().double()
        per = lambda t: torch.repeat_interleave(t, rows)[:x.shape[0], None]  # noqa: E731
        q = (b * per(inv)).float().to(torch.float8_e4m3fn).double()
        parts.append(q * per(scale))
        scales.append(scale)
    return torch.cat(parts, 1), torch.stack(scales, 1)


def _exact_weights(elem, scale):
    """E4M3 bytes by their fields, times the scale of row / 128, column / 128."""
    b = elem.long()
    e, m = (b >> 3) & 15, (b & 7).double()
    v = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))
    v = torch.where((b & 127) == 127, float("nan"), v) * torch.where(b >= 128, -1.0, 1.0)
    i = torch.arange(elem.shape[0], device=elem.device) // 128
    j = torch.arange(elem.shape[1], device=elem.device) // 128
    return v * scale.double()[i][:, j]


def _exact_expert(s, name, e):
    c, w = s["case"], s[name]
    form = "fp8" if c["op"] == "experts" else c["form"]
    if form == "fp8":
        return _exact_weights(w[0][e], w[1][e])
    if form != "mx4":
        return w[e].double()
    n = w[0].shape[0] // c["experts"]
    elem, scale = w[0][e * n:(e + 1) * n], w[1][e * n:(e + 1) * n]
    codes = torch.cat([(elem.long() & 15)[:, :, None], (elem.long() >> 4)[:, :, None]], 2).flatten(1)
    f = torch.exp2(scale.double() - 127.0)[:, :elem.shape[1] // 16]
    return _table(torch.float64)[codes] * f.repeat_interleave(32, dim=1)


def _exact_route(logits, bias, topk, scoring):
    l = logits.double().nan_to_num(nan=float("-inf"), posinf=float("inf"), neginf=float("-inf"))
    key = l if bias is None else (logits.float() + bias).double()   # keys are FP32 sums by definition
    key = torch.where(l > float("-inf"), key, float("-inf"))
    order = torch.argsort(-key, dim=1, stable=True)[:, :topk]   # the lower index first among equals
    live = key.gather(1, order) > float("-inf")
    top = torch.where(live, l.gather(1, order), float("-inf"))
    if scoring == "sigmoid":
        w = torch.sigmoid(top) * live
        w = w / w.sum(1, keepdim=True)
    elif scoring == "softmax":
        w = torch.softmax(l, 1).gather(1, order)
    else:
        w = torch.softmax(top, 1)
    return torch.where(live, order, -1), torch.where(live, w, 0.0)


def exact(c, seed):
    if 6.0 * work(c)["flops"] > 4e13:   # 64-bit products of this size take too long
        return None
    s = dict(_inputs(c, seed), case=c)
    op = c["op"]
    if op == "convert":
        v, scale = _exact_fp8(s["x"], c["block_rows"])
        return scale, v
    if op == "product":
        x = _exact_fp8(s["x"], 1)[0] if c["act"] == "fp8" else s["x"].double()
        return torch.matmul(x, _exact_weights(s["elem"], s["scale"]).transpose(0, 1))
    layer = op == "layer"
    ids, w = _exact_route(s["logits"], s["bias"], c["topk"], c["scoring"] if layer else "softmax_topk")
    pairs = sorted((e, p) for p, e in enumerate(ids.reshape(-1).tolist()) if e >= 0)
    n, k, gated = c["n"], c["k"], layer or c["gated"]
    h = torch.zeros(ids.numel(), n, dtype=torch.float64, device=DEV)   # by slot, the pairs sorted by expert
    y = torch.zeros(c["tokens"], k, dtype=torch.float64, device=DEV)
    for e in sorted({e for e, _ in pairs}):
        at = [i for i, (q, _) in enumerate(pairs) if q == e]
        mine = torch.tensor([pairs[i][1] for i in at], device=DEV)
        x = s["x"][mine // c["topk"]].double()
        g = torch.matmul(x, _exact_expert(s, "gate", e).transpose(0, 1))
        if gated:
            g = g * torch.sigmoid(g) * torch.matmul(x, _exact_expert(s, "up", e).transpose(0, 1))
        h[at[0]:at[-1] + 1] = g
        if layer:   # a token has an expert once
            d = torch.matmul(g, _exact_expert(s, "down", e).transpose(0, 1))
            y[mine // c["topk"]] += d * w.flatten()[mine][:, None]
    return (ids.to(torch.int32), w, y) if layer else h
