"""Routing of up to 64 pairs, which one wave does alone: lanes hand ids, counts and first slots to each other."""
import numpy as np
import pytest
import torch

from tests.test_gpu_experts import DEV, check_plan, check_route

pytestmark = pytest.mark.gpu
SIZES = [(1, 1, 1), (1, 16, 16), (2, 1024, 16), (4, 16, 16), (4, 1024, 16), (5, 64, 12), (8, 65, 8), (9, 7, 7), (16, 5, 4),
         (21, 300, 3), (32, 2, 2), (63, 129, 1), (64, 1, 1), (64, 1000, 1)]


@pytest.fixture(scope="module")
def uw():
    from decode_gemm_exp_amd import uw as _uw
    return _uw


@pytest.mark.parametrize("tokens,experts,topk", SIZES)
def test_choice_and_plan(uw, tokens, experts, topk):
    g = torch.Generator().manual_seed(64 * tokens + experts)
    l = torch.randn(tokens, experts, generator=g)
    for scoring in ("softmax", "softmax_topk", "sigmoid"):
        check_route(uw, l, topk, scoring)
    l[tokens // 2] = float("-inf")
    check_route(uw, l, topk, "softmax_topk")
    l[:] = 0.25                                   # every token the same experts
    check_route(uw, l.bfloat16(), topk, "sigmoid", ld=experts + 1)


@pytest.mark.parametrize("tokens,experts,topk", SIZES)
def test_plan_of_given_ids(uw, tokens, experts, topk):
    g = torch.Generator().manual_seed(tokens + experts)
    r = uw.Routing(tokens, experts, topk, DEV)
    few = torch.randint(0, 2, (tokens, topk), generator=g) * (experts - 1)
    every = torch.randint(-1, experts + 1, (tokens, topk), generator=g)
    for ids in (every, few, torch.full((tokens, topk), experts - 1), torch.full((tokens, topk), -1),
                torch.arange(tokens * topk).view(tokens, topk) % experts, experts - 1 - few):
        ids = ids.to(torch.int32)
        for _ in range(2):
            r.rows.fill_(-7)
            uw.uw_plan_experts(ids.to(DEV), r)
            check_plan(r, np.where((ids >= 0) & (ids < experts), ids, -1), experts)
