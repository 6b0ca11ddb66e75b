"""The router's choice by sigmoid(logit) + bias against a plain 64-bit implementation.

The key in FP32 is off by at most the exponential's, the sum's and the
quotient's roundings, 2^-23 relative each, of a sigmoid of at most 1, and the
last addition's 2^-24 of the key: below 2^-20 for |bias| <= 2.  Inputs are drawn
so that the keys that decide a choice are 2^-18 apart at least.
"""
import numpy as np
import pytest
import torch

from tests.test_gpu_experts import DEV, check_plan, route_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def uw():
    from decode_gemm_exp_amd import uw as _uw
    return _uw


def keys(l, bias):
    l, b = l.double().numpy(), bias.double().numpy()
    with np.errstate(over="ignore", invalid="ignore"):
        k = 1.0 / (1.0 + np.exp(-l)) + b
    return np.where(np.isnan(l) | np.isneginf(l) | np.isnan(k), -np.inf, k)


def draw(g, tokens, experts, topk, bias, dtype):
    l = (torch.randn(tokens, experts, generator=g) * 3).to(dtype)
    while True:
        k = -np.sort(-keys(l, bias), 1)[:, :topk + 1]
        near = np.flatnonzero((k[:, :-1] - k[:, 1:] < 2.0 ** -18).any(1))
        if not len(near):
            return l
        l[near] = (torch.randn(len(near), experts, generator=g) * 3).to(dtype)


def check(uw, l, topk, bias):
    """ids by key, ties to the lower index; weights from the sigmoids of the chosen alone; the plan."""
    t, n = l.shape
    r = uw.Routing(t, n, topk, DEV)
    r.rows.fill_(-7)
    uw.uw_route_experts(l.to(DEV), r, "sigmoid_biased", bias.to(DEV))
    k = keys(l, bias)
    order = np.argsort(-k, 1, kind="stable")[:, :topk]
    live = np.take_along_axis(k, order, 1) > -np.inf
    ids = np.where(live, order, -1).astype(np.int32)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    v = np.take_along_axis(l.double().numpy(), order, 1)
    with np.errstate(over="ignore", invalid="ignore"):
        s = np.where(live, 1.0 / (1.0 + np.exp(-v)), 0.0)
        w = np.nan_to_num(s / s.sum(1, keepdims=True))
    # sigmoid's logarithm keeps |l| 2^-24 absolute; exp, log1p and the sum as in test_gpu_experts
    assert np.allclose(r.weights.cpu().double().numpy(), w, rtol=2.0 ** -16, atol=1e-37)
    check_plan(r, ids, n)
    return ids


@pytest.mark.parametrize("tokens,experts,topk", [(1, 64, 4), (7, 24, 6), (200, 16, 3), (300, 256, 8), (90, 300, 5),
                                                 (2000, 160, 8), (40, 1024, 16)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_bias_on_the_score(uw, tokens, experts, topk, dtype):
    g = torch.Generator().manual_seed(tokens + experts)
    bias = torch.rand(experts, generator=g) * 0.6 - 0.3
    l = draw(g, tokens, experts, topk, bias, dtype)
    ids = check(uw, l, topk, bias)
    if tokens >= 40:   # it is not the choice by logit + bias
        assert not np.array_equal(ids, route_ref(l, topk, "sigmoid", bias)[0])


def test_bias_on_the_score_specials(uw):
    n = 8
    g = torch.Generator().manual_seed(3)
    bias = torch.tensor([0.1, -0.2, 0.3, float("-inf"), 2.0, 0.0, float("nan"), -0.1])
    l = draw(g, 30, n, 5, bias, torch.float32)
    l[1] = float("-inf")                                  # a padded token
    l[2] = float("nan")
    l[3, 4] = float("-inf")                               # masked, whatever its bias
    l[4, 4], l[4, 0] = float("nan"), float("inf")
    l[5, 1:] = float("-inf")                              # one left
    l[6] = -200.0                                         # sigmoids of zero: the bias alone
    l[7] = torch.finfo(torch.float32).min
    r = uw.Routing(30, n, 5, DEV)
    uw.uw_route_experts(l.to(DEV), r, "sigmoid_biased", bias.to(DEV))
    ids, w = r.ids.cpu(), r.weights.cpu()
    ok = [i for i in range(30) if i not in (6, 7)]        # (there every sigmoid is zero: their weights are not ratios of them)
    r2 = check(uw, l[ok], 5, bias)
    assert np.array_equal(ids[ok].numpy(), r2)
    assert (ids[1] == -1).all() and (ids[2] == -1).all() and (w[1:3] == 0).all()
    assert ids[5].tolist() == [0, -1, -1, -1, -1] and w[5].tolist() == [1.0, 0.0, 0.0, 0.0, 0.0]
    assert ids[6].tolist() == ids[7].tolist() == [4, 2, 0, 5, 7]
    assert torch.allclose(w[6:8].double(), torch.full((2, 5), 0.2, dtype=torch.float64), rtol=2.0 ** -20)
    assert not ((ids == 3) | (ids == 6)).any()


def test_equal_scores_go_to_the_lower_index(uw):
    """Sigmoids that are 1 in FP32 tie with a bias; without one the choice is by logit."""
    l = torch.tensor([[30.0, 40.0, 50.0, 20.0], [0.5, 0.5, 0.5, 0.5], [-0.0, 0.0, -0.0, 0.0]])
    r = uw.Routing(3, 4, 3, DEV)
    uw.uw_route_experts(l.to(DEV), r, "sigmoid_biased", torch.zeros(4, device=DEV))
    assert r.ids.cpu().tolist() == [[0, 1, 2]] * 3
    uw.uw_route_experts(l.to(DEV), r, "sigmoid_biased")
    assert r.ids.cpu().tolist() == [[2, 1, 0], [0, 1, 2], [0, 1, 2]]
    want = [r.ids.clone(), r.weights.clone()]
    uw.uw_route_experts(l.to(DEV), r, "sigmoid")
    assert torch.equal(want[0], r.ids) and torch.equal(want[1], r.weights)


def test_bias_on_the_score_captured(uw):
    """Choice and plan in one graph, replayed on new scores with eager work between."""
    g = torch.Generator().manual_seed(8)
    tokens, experts, topk = 500, 64, 6
    l, bias = torch.zeros(tokens, experts, device=DEV), torch.zeros(experts, device=DEV)
    r = uw.Routing(tokens, experts, topk, DEV)
    step = lambda: uw.uw_route_experts(l, r, "sigmoid_biased", bias)  # noqa: E731
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        l.copy_(torch.randn(tokens, experts, generator=g))
        bias.copy_(torch.randn(experts, generator=g) * 0.2)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (r.ids, r.weights, r.offsets, r.rows, r.slots)]
        r.ids.zero_()
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (r.ids, r.weights, r.offsets, r.rows, r.slots)))
