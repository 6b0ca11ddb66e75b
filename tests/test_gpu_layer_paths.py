"""The layer's down product in every form and in every split of its MFMAs' rows and columns, against plain
64-bit implementations; tolerances as in tests/test_gpu_layer.py.
"""
import pytest
import torch

from tests import test_gpu_layer as layer
from tests.test_gpu_experts import make_set, route_ref, weights
from tests.test_gpu_experts_edges import two_bands

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def uw():
    from decode_gemm_exp_amd import uw as _uw
    return _uw


def split(tokens, experts, topk, k):
    """Places of k in an MFMA's rows, and columns for an expert's tokens, on 256 CUs."""
    most = min(tokens, -(-2 * tokens * topk // experts) + 1)
    if k // 16 >= 256 or most > 8:
        return 1, 16 if most > 4 else 4
    if k // 8 >= 256 or most > 4:
        return 2, 8 if most > 4 else 4 if most > 2 else 2
    return 4, 4


def one_band(g, e, n, k):
    """Sixteen consecutive exponents, equally frequent, are every palette: a run; rarer ones make verbatim groups."""
    w = torch.exp2(-4.0 - torch.randint(0, 16, (e, n, k), generator=g)) * (1 + torch.rand(e, n, k, generator=g) * 0.99)
    w = torch.where(torch.rand(w.shape, generator=g) < 0.5, w, -w)
    far = torch.exp2(torch.randint(-60, 20, w.shape, generator=g).float())
    return torch.where(torch.rand(w.shape, generator=g) < 0.004, far, w)


# Rows of the down weights from shorter than a place's share of a window to several windows with a cut-off last one.
CASES = [(16, 6, 3, 416, 96, (1, 16)), (8, 8, 3, 160, 4128, (1, 16)), (5, 12, 2, 288, 4128, (1, 4)),
         (8, 8, 3, 416, 160, (2, 8)), (7, 6, 2, 1056, 2080, (2, 8)), (16, 40, 3, 288, 2080, (2, 4)),
         (4, 5, 1, 544, 2080, (2, 4)), (2, 8, 2, 160, 2080, (2, 2)), (16, 130, 4, 96, 2080, (2, 2)),
         (4, 16, 2, 1568, 160, (4, 4)), (16, 40, 3, 96, 416, (4, 4))]


@pytest.mark.parametrize("tokens,experts,topk,n,k,how", CASES)
@pytest.mark.parametrize("form", ["bf16", "mx4", "fp8", "uwf1", "uwf1_one_band", "uwf1_two_bands"])
def test_down_product(uw, form, tokens, experts, topk, n, k, how):
    """Tokens spread over the experts, and all of them on one expert: as many items as its tokens fill."""
    g = torch.Generator().manual_seed(experts + n)
    if form.startswith("uwf1"):
        n, k = (n + 63) // 64 * 64, (k + 63) // 64 * 64   # whole groups
    assert split(tokens, experts, topk, k) == how
    base = form[:4]
    gate, gv = layer.any_set(uw, base, weights(g, experts, n, k))
    up, uv = layer.any_set(uw, base, weights(g, experts, n, k))
    bands = {"uwf1_one_band": one_band, "uwf1_two_bands": two_bands}.get(form)
    w = bands(g, experts, k, n) if bands else weights(g, experts, k, n, outliers=base == "uwf1")
    down, dv = layer.any_set(uw, base, w)
    x = torch.randn(tokens, k, generator=g).bfloat16()
    for crowded in (False, True):
        l = torch.randn(tokens, experts, generator=g)
        if crowded:
            l[:, experts // 2] += 20.0
        _, out = layer.run(uw, (gate, up, down), l.to(DEV), x.to(DEV), topk, "softmax_topk")
        ids, wt = route_ref(l, topk, "softmax_topk")
        assert not crowded or (ids[:, 0] == experts // 2).all()
        ref, tol = layer.layer_ref(ids, wt, experts, x, gv, uv, dv)
        assert bool(((out.double().cpu() - ref).abs() <= tol).all()), "crowded" if crowded else "spread"


@pytest.mark.parametrize("tokens", [3, 6, 16])
def test_not_finite_uwf1_down_weights_stay_with_their_tokens(uw, tokens):
    """An infinity and a NaN among the down weights of an expert spoil those outputs of its tokens alone."""
    g = torch.Generator().manual_seed(12)
    experts, topk, n, k = 6, 2, 128, 192
    gate, up = make_set(uw, "uwf1", weights(g, experts, n, k))[0], make_set(uw, "uwf1", weights(g, experts, n, k))[0]
    w = weights(g, experts, k, n)
    bad = w.clone()
    bad[5, 3, 7], bad[5, 190, n - 1] = float("inf"), float("nan")
    l, x = torch.randn(tokens, experts, generator=g).to(DEV), torch.randn(tokens, k, generator=g).bfloat16().to(DEV)
    l[0, 5] = 9.0                              # token 0 has expert 5,
    l[1:, 5] = float("-inf")                   # no other has
    _, clean = layer.run(uw, (gate, up, make_set(uw, "uwf1", w)[0]), l, x, topk)
    _, out = layer.run(uw, (gate, up, make_set(uw, "uwf1", bad)[0]), l, x, topk)
    assert not out[0, 3].isfinite() and out[0, 190].isnan()
    rest = torch.ones(k, dtype=torch.bool, device=DEV)
    rest[3] = rest[190] = False
    assert torch.equal(out[0, rest], clean[0, rest]) and torch.equal(out[1:], clean[1:])
