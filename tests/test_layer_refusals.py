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
