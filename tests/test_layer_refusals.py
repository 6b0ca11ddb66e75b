"""What the layer's calls refuse before anything is enqueued, on the host alone: no device is touched."""
import ctypes

import pytest

INVALID, UNSUPPORTED = -1, -2
P = 4096   # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def uw():
    from decode_gemm_exp_amd import uw as _uw
    return _uw


def bf16_set(uw, count=4, n=64, k=64):
    h = ctypes.c_void_p()
    assert uw._lib.uw_experts_bf16(P, count, n, k, 0, ctypes.byref(h)) == 0
    return h


def layer(uw, gate, down, tokens=4, topk=2, type=0, bias=None, logits=P, ids=P, weights=P, off=P, rows=P, slots=P):
    return uw._lib.uw_expert_layer(gate, gate, down, logits, type, tokens, 1 << 12, bias, topk, 1, ids, weights, off,
                                   rows, slots, P, P, P, 1 << 62, None)


@pytest.mark.parametrize("tokens", [1, 16, 17, 400])
def test_layer_refuses_misaligned_arrays(uw, tokens):
    """Four bytes for every array of integers and floats, two for BF16 scores, in both forms of the call."""
    h = bf16_set(uw)
    for name in ("logits", "ids", "weights", "off", "rows", "slots", "bias"):
        for by in (1, 2, 3):
            assert layer(uw, h, h, tokens, **{name: P + by}) == INVALID, (name, by)
    assert layer(uw, h, h, tokens, type=1, logits=P + 1) == INVALID
    uw._lib.uw_free_experts(h)


@pytest.mark.parametrize("n,k", [(1 << 20, 32), (32, 1 << 20)])
def test_products_of_too_many_threads(uw, n, k):
    """One of the two products would be 2^32 GPU threads: refused before the router, or the other product, runs."""
    gate, down = bf16_set(uw, 1024, n, k), bf16_set(uw, 1024, k, n)
    f = uw._lib.uw_free_experts
    # 512 threads for each of 4096 (gated: 8192) tiles of columns by 1024 + 70400 / 64 chunks of rows
    assert layer(uw, gate, down, 4400, 16) == UNSUPPORTED
    assert uw._lib.uw_expert_mlp(gate, gate, down, 4400, 16, P, P, P, P, P, P, P, 1 << 62, None) == UNSUPPORTED
    f(gate), f(down)


def test_sets_that_do_not_fit_each_other(uw):
    """gate and up of different shape or form, before a device is asked for."""
    gate, wide, few, down = bf16_set(uw), bf16_set(uw, n=96), bf16_set(uw, count=3), bf16_set(uw)
    fp8 = ctypes.c_void_p()
    assert uw._lib.uw_experts_fp8(P, P, 4, 64, 64, 0, 0, ctypes.byref(fp8)) == 0
    for tokens in (4, 40):
        for up, want in ((wide, INVALID), (few, INVALID), (fp8, UNSUPPORTED)):
            assert uw._lib.uw_expert_layer(gate, up, down, P, 0, tokens, 4, None, 2, 1, P, P, P, P, P, P, P, P, 1 << 62,
                                           None) == want
            assert uw._lib.uw_expert_mlp(gate, up, down, tokens, 2, P, P, P, P, P, P, P, 1 << 62, None) == want
    for h in (gate, wide, few, down, fp8):
        uw._lib.uw_free_experts(h)
