"""The layer from the router's scores in one call, against plain 64-bit implementations
and against the calls it stands for.

Tolerance, derived: h as in tests/test_gpu_experts.py (FP8: k + 16 steps for k); then
with m = sum over a token's experts of w |h| . |D|, each of the at most n products is
exact in FP32, a window's sum is weighted and scaled by at most four roundings and added
to those before it, in all at most 2 n + 16 steps of 2^-23 for up to 16 experts (n / 128 + 1
windows each, eight waves); weights are off by 2^-16 relative (exponentials, sums and
quotients in FP32) and the result is rounded to BF16, 2^-8 relative.
"""
import numpy as np
import pytest
import torch

from tests import test_gpu_fp8_blocks as fp8
from tests.test_gpu_experts import grouped_ref, h_ref, make_set, plan_ref, route_ref, weights

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FORMS = ["bf16", "mx4", "uwf1", "fp8"]


@pytest.fixture(scope="module")
def uw():
    from decode_gemm_exp_amd import uw as _uw
    return _uw


def any_set(uw, form, w):
    return fp8.make_set(uw, w) if form == "fp8" else make_set(uw, form, w)


def layer_ref(ids, w, experts, x, gv, uv, dv):
    off, rows, slots = plan_ref(ids, experts)
    rows = torch.from_numpy(rows)
    n, k = gv.shape[1:]
    f = (k + 16) / k
    (a, am), (b, bm) = grouped_ref(off, rows, x, gv), grouped_ref(off, rows, x, uv)
    hv, ht = h_ref(a, am * f, b, bm * f, k)
    out = torch.zeros(len(x), k, dtype=torch.float64)
    tol, mag = torch.zeros_like(out), torch.zeros_like(out)
    for t in range(len(x)):
        for j in range(ids.shape[1]):
            s = int(slots[t, j])
            if s >= 0:
                d, wt = dv[int(ids[t, j])], float(w[t, j])
                out[t] += wt * (hv[s] @ d.T)
                tol[t] += wt * (ht[s] @ d.abs().T)
                mag[t] += wt * ((hv[s].abs() + ht[s]) @ d.abs().T)
    tol += ((2 * n + 16) * 2.0 ** -23 + 2.0 ** -16) * mag
    return out, tol + 2.0 ** -8 * (out.abs() + tol)


def build(uw, g, gf, df, experts, n, k):
    gate, gv = any_set(uw, gf, weights(g, experts, n, k))
    up, uv = any_set(uw, gf, weights(g, experts, n, k, outliers=False))
    down, dv = any_set(uw, df, weights(g, experts, k, n))
    return (gate, up, down), (gv, uv, dv)


def run(uw, sets, l, x, topk, scoring="softmax_topk", bias=None, ws_fill=255):
    tokens, experts = l.shape
    r = uw.Routing(tokens, experts, topk, DEV)
    r.rows.fill_(-7)
    out = torch.full((tokens, sets[0].k), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = torch.full((uw.uw_workspace_size_expert_layer(sets[0], sets[2], tokens, topk),), ws_fill, dtype=torch.uint8,
                    device=DEV)
    uw.uw_expert_layer(*sets, l, r, x, out, ws, scoring, bias)
    return r, out


def same_routing(a, b):
    return all(torch.equal(p, q) for p, q in
               ((a.ids, b.ids), (a.weights, b.weights), (a.offsets, b.offsets), (a.rows, b.rows), (a.slots, b.slots)))


def routed(uw, l, topk, scoring, bias=None):
    r = uw.Routing(*l.shape, topk, DEV)
    r.rows.fill_(-7)
    uw.uw_route_experts(l, r, scoring, bias)
    return r


CASES = [(1, 1, 1, 64, 64), (1, 4, 2, 64, 128), (2, 64, 8, 192, 320), (3, 8, 3, 128, 192), (4, 5, 5, 320, 128),
         (5, 65, 6, 64, 256), (7, 16, 2, 704, 448), (8, 300, 7, 64, 128), (9, 6, 4, 128, 576), (13, 256, 6, 192, 64),
         (16, 16, 16, 64, 192), (16, 40, 1, 256, 128)]


@pytest.mark.parametrize("tokens,experts,topk,n,k", CASES)
@pytest.mark.parametrize("form", FORMS + ["mixed"])
def test_layer(uw, form, tokens, experts, topk, n, k):
    g = torch.Generator().manual_seed(tokens + experts)
    gf, df = ("fp8", "mx4") if form == "mixed" else (form, form)
    if form != "uwf1":
        n, k = n + 32, k + 96                  # tails of the windows and of the blocks
    sets, vals = build(uw, g, gf, df, experts, n, k)
    l = torch.randn(tokens, experts, generator=g)
    if tokens > 4:
        l[2:4] = float("-inf")                 # padded tokens
        l[4, 1:] = float("-inf")               # one expert left
    x = torch.randn(tokens, k, generator=g).bfloat16()
    scoring = ["softmax", "softmax_topk", "sigmoid"][tokens % 3]
    r, out = run(uw, sets, l.to(DEV), x.to(DEV), topk, scoring)
    assert same_routing(r, routed(uw, l.to(DEV), topk, scoring))
    ids, w = route_ref(l, topk, scoring)
    ref, tol = layer_ref(ids, w, experts, x, *vals)
    got = out.double().cpu()
    assert bool(((got - ref).abs() <= tol).all())
    if tokens > 4:
        assert bool((got[2:4] == 0).all())
    again = run(uw, sets, l.to(DEV), x.to(DEV), topk, scoring, ws_fill=0)[1]
    assert torch.equal(out, again), "two calls differ"


@pytest.mark.parametrize("tokens", [0, 1, 2, 4, 8, 15, 16, 17, 40, 300])
@pytest.mark.parametrize("scoring", ["softmax", "softmax_topk", "sigmoid", "sigmoid_biased"])
def test_routing_is_the_routers(uw, tokens, scoring):
    """ids, weights and plan are uw_route_experts' bit for bit, with a bias, BF16 scores (ties), strided rows,
    masked scores and tokens, at every kernel for a number of experts."""
    for experts, topk in ((3, 3), (64, 8), (65, 2), (256, 16), (257, 5), (1024, 16)):
        g = torch.Generator().manual_seed(experts + tokens)
        sets, _ = build(uw, g, "bf16", "bf16", experts, 32, 32)
        wide = torch.randn(tokens, experts + 5, generator=g)
        wide[torch.rand(wide.shape, generator=g) < 0.2] = float("-inf")
        if tokens > 1:
            wide[1] = float("nan")
        x = torch.randn(tokens, 32, generator=g).bfloat16().to(DEV)
        bias = torch.randn(experts, generator=g).to(DEV)
        for dt in (torch.float32, torch.bfloat16):
            l = wide.to(dt).to(DEV)[:, :experts]
            r, out = run(uw, sets, l, x, topk, scoring, bias)
            assert same_routing(r, routed(uw, l, topk, scoring, bias))
            if tokens:
                assert out.isfinite().all()
            if tokens > 1:
                assert bool((out[1] == 0).all())


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("tokens", [6, 40])
def test_layer_is_the_two_calls(uw, form, tokens):
    """What uw_route_experts and uw_expert_mlp give: the same beyond UW_LAYER_TOKENS, within the sums' order below."""
    g = torch.Generator().manual_seed(21)
    experts, topk, n, k = 9, 3, 192, 320
    sets, _ = build(uw, g, form, form, experts, n, k)
    l, x = torch.randn(tokens, experts, generator=g).to(DEV), torch.randn(tokens, k, generator=g).bfloat16().to(DEV)
    _, out = run(uw, sets, l, x, topk)
    r = routed(uw, l, topk, "softmax_topk")
    two = torch.empty_like(out)
    ws = torch.empty(uw.uw_workspace_size_expert_mlp(sets[0], sets[2], tokens, topk), dtype=torch.uint8, device=DEV)
    uw.uw_expert_mlp(*sets, r, x, two, ws)
    if tokens > 16:
        assert torch.equal(out, two)
    else:   # both are within half a BF16 step of sums that agree far closer
        big = two.double().abs().amax(1, keepdim=True)
        assert bool(((out.double() - two.double()).abs() <= 2.0 ** -7 * two.double().abs() + 2.0 ** -12 * big).all())


@pytest.mark.parametrize("form", FORMS)
def test_not_finite_values_stay_with_their_tokens(uw, form):
    """A token with an infinity or a NaN in x spoils its own row alone; an expert with a NaN or infinite down
    weight spoils that output of its tokens alone, and no output of a token without the expert."""
    g = torch.Generator().manual_seed(12)
    experts, topk, n, k = 6, 2, 128, 192
    for tokens in (3, 6, 16):
        sets, _ = build(uw, g, form, form, experts, n, k)
        l, x = torch.randn(tokens, experts, generator=g).to(DEV), torch.randn(tokens, k, generator=g).bfloat16().to(DEV)
        l[0, 5] = 9.0                          # token 0 has expert 5,
        l[1:, 5] = float("-inf")               # no other has
        _, clean = run(uw, sets, l, x, topk)
        bad = x.clone()
        bad[1, k - 1] = float("nan")
        bad[2, 0] = float("inf")
        _, out = run(uw, sets, l, bad, topk)
        assert out[1].isnan().all() and not out[2].isfinite().any()
        keep = [t for t in range(tokens) if t not in (1, 2)]
        assert torch.equal(out[keep], clean[keep])
        down = sets[2]
        if form == "bf16":
            down.keep.view(experts, k, n)[5, 3, 7] = float("inf")
            down.keep.view(experts, k, n)[5, 190, n - 1] = float("nan")
        elif form == "fp8":
            down.keep[0].view(torch.uint8)[5, 3, 7] = 0x7F
            down.keep[0].view(torch.uint8)[5, 190, n - 1] = 0xFF
        elif form == "mx4":
            down.keep[1].view(experts, k, -1)[5, 3, 0] = 255
            down.keep[1].view(experts, k, -1)[5, 190, n // 32 - 1] = 255
        else:
            continue
        _, out = run(uw, sets, l, x, topk)
        assert not out[0, 3].isfinite() and not out[0, 190].isfinite()
        rest = torch.ones(k, dtype=torch.bool, device=DEV)
        rest[3] = rest[190] = False
        assert torch.equal(out[0, rest], clean[0, rest]) and torch.equal(out[1:], clean[1:])


@pytest.mark.parametrize("form", FORMS)
def test_larger_layer(uw, form):
    """Sizes at which every wave has several windows, experts' windows straddle waves and the output has more
    blocks than the chip: against the two calls' products."""
    g = torch.Generator().manual_seed(31)
    for tokens, experts, topk, n, k in ((1, 16, 4, 1408, 2048), (6, 8, 2, 2112, 1024), (16, 12, 3, 1024, 4224)):
        sets, vals = build(uw, g, form, form, experts, n, k)
        l, x = torch.randn(tokens, experts, generator=g), torch.randn(tokens, k, generator=g).bfloat16()
        _, out = run(uw, sets, l.to(DEV), x.to(DEV), topk, "softmax")
        ids, w = route_ref(l, topk, "softmax")
        ref, tol = layer_ref(ids, w, experts, x, *vals)
        assert bool(((out.double().cpu() - ref).abs() <= tol).all())


def test_captured_layers_share_a_workspace(uw):
    """Two captured layers of different token counts with one workspace, replayed in turn with other tokens and
    other routings, eager work between."""
    g = torch.Generator().manual_seed(17)
    experts, topk, n, k = 70, 3, 96, 160
    sets, _ = build(uw, g, "fp8", "mx4", experts, n, k)
    ws = torch.empty(max(uw.uw_workspace_size_expert_layer(sets[0], sets[2], t, topk) for t in (3, 16, 40)),
                     dtype=torch.uint8, device=DEV)
    jobs = []
    for tokens in (3, 16, 40):
        l, x = torch.zeros(tokens, experts, device=DEV), torch.zeros(tokens, k, dtype=torch.bfloat16, device=DEV)
        r, out = uw.Routing(tokens, experts, topk, DEV), torch.empty(tokens, k, dtype=torch.bfloat16, device=DEV)

        def step(l=l, x=x, r=r, out=out):
            uw.uw_expert_layer(*sets, l, r, x, out, ws)

        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        jobs.append((graph, l, x, r, out, step))
    seen = []
    for i in range(4):
        for _, l, x, _, out, _ in jobs:
            l.copy_(torch.randn(l.shape, generator=g))
            x.copy_(torch.randn(x.shape, generator=g))
            if i == 2:
                l[:, 1:] = float("-inf")       # every token to one expert
            out.zero_()
        for graph, *_ in jobs:
            graph.replay()
        torch.cuda.synchronize()
        got = [(j[4].clone(), j[3].ids.clone()) for j in jobs]
        for _, _, _, r, out, step in jobs:
            out.zero_()
            r.ids.zero_()
            step()
        torch.cuda.synchronize()
        for (a, b), j in zip(got, jobs):
            assert torch.equal(a, j[4]) and torch.equal(b, j[3].ids)
        seen.append(got[0][0])
    assert not torch.equal(seen[0], seen[1])


def test_two_streams_at_once(uw):
    """Layers on two streams with their own workspaces give what they give alone."""
    g = torch.Generator().manual_seed(5)
    tokens, experts, topk, n, k = 11, 24, 4, 1056, 1024
    sets, _ = build(uw, g, "mx4", "fp8", experts, n, k)
    nb = uw.uw_workspace_size_expert_layer(sets[0], sets[2], tokens, topk)
    jobs = []
    for _ in range(2):
        jobs.append((torch.randn(tokens, experts, generator=g).to(DEV), torch.randn(tokens, k, generator=g).bfloat16().to(DEV),
                     uw.Routing(tokens, experts, topk, DEV), torch.empty(tokens, k, dtype=torch.bfloat16, device=DEV),
                     torch.empty(nb, dtype=torch.uint8, device=DEV), torch.cuda.Stream()))
    alone = []
    for l, x, r, out, ws, _ in jobs:
        uw.uw_expert_layer(*sets, l, r, x, out, ws)
        torch.cuda.synchronize()
        alone.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for l, x, r, out, ws, s in jobs:
            with torch.cuda.stream(s):
                uw.uw_expert_layer(*sets, l, r, x, out, ws)
    torch.cuda.synchronize()
    for (_, _, _, out, _, _), a in zip(jobs, alone):
        assert torch.equal(out, a)


def test_layer_from_conversion_on(uw):
    """As a server runs them: BF16 experts converted once, then decode steps and a prompt through the same sets."""
    g = torch.Generator().manual_seed(40)
    experts, topk, n, k = 12, 2, 160, 288
    sets, vals = build(uw, g, "fp8", "fp8", experts, n, k)
    for tokens in (1, 16, 17, 200, 1):
        l, x = torch.randn(tokens, experts, generator=g), torch.randn(tokens, k, generator=g).bfloat16()
        r, out = run(uw, sets, l.to(DEV), x.to(DEV), topk, "sigmoid")
        ids, w = route_ref(l, topk, "sigmoid")
        assert np.array_equal(r.ids.cpu().numpy(), ids)
        ref, tol = layer_ref(ids, w, experts, x, *vals)
        assert bool(((out.double().cpu() - ref).abs() <= tol).all())
