"""What the FP8 calls and the layer call refuse, on the host alone: no device is touched."""
import ctypes

import pytest
import torch

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -7
P = 4096   # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def uw():
    from decode_gemm_exp_amd import uw as _uw
    return _uw


def bf16_set(uw, count=4, n=64, k=64):
    h = ctypes.c_void_p()
    assert uw._lib.uw_experts_bf16(P, count, n, k, 0, ctypes.byref(h)) == 0
    return h


def test_conversion_refusals(uw):
    q, d = uw._lib.uw_quantize_fp8, uw._lib.uw_dequantize_fp8
    assert q(None, 1, 4, 64, 64, 1, P, P, None) == INVALID
    assert q(P, 1, 4, 64, 64, 1, None, P, None) == INVALID
    assert q(P, 1, 4, 64, 64, 1, P, None, None) == INVALID
    assert q(P, 2, 4, 64, 64, 1, P, P, None) == INVALID          # type
    for rows in (0, 2, 64, -1):
        assert q(P, 1, 4, 64, 64, rows, P, P, None) == INVALID   # blocks are 1 x 128 or 128 x 128
        assert d(P, P, 4, 64, rows, P, 64, None) == INVALID
    assert q(P, 1, -1, 64, 64, 1, P, P, None) == INVALID
    assert q(P, 1, 4, 0, 64, 1, P, P, None) == INVALID
    assert q(P, 1, 4, 48, 64, 1, P, P, None) == UNSUPPORTED      # columns go by 32
    assert q(P, 1, (1 << 20) + 1, 64, 64, 1, P, P, None) == UNSUPPORTED
    assert q(P, 1, 4, 64, 32, 1, P, P, None) == INVALID          # rows overlap
    assert q(P, 1, 4, 64, 68, 1, P, P, None) == UNSUPPORTED      # rows not on 16 bytes
    assert q(P + 2, 1, 4, 64, 64, 1, P, P, None) == INVALID
    assert q(P, 1, 4, 64, 64, 1, P + 4, P, None) == INVALID
    assert q(P, 1, 4, 64, 64, 1, P, P + 2, None) == INVALID
    assert q(P, 1, 0, 64, 64, 1, P, P, None) == 0                # nothing to do
    assert d(None, P, 4, 64, 1, P, 64, None) == INVALID
    assert d(P, None, 4, 64, 1, P, 64, None) == INVALID
    assert d(P, P, 4, 64, 1, None, 64, None) == INVALID
    assert d(P, P, 4, 40, 1, P, 64, None) == UNSUPPORTED
    assert d(P, P, 4, 64, 1, P, 60, None) == INVALID
    assert d(P, P, 4, 64, 1, P, 65, None) == UNSUPPORTED
    assert d(P, P, 4, 64, 1, P + 8, 64, None) == INVALID
    assert d(P, P, 0, 64, 128, P, 64, None) == 0


def test_product_refusals(uw):
    n = ctypes.c_size_t()
    size = uw._lib.uw_workspace_size_fp8
    assert size(64, 64, 4, 0, None) == INVALID
    assert size(64, 64, 4, 1, ctypes.byref(n)) == INVALID        # 4-bit activations are another call's
    assert size(64, 64, 4, 3, ctypes.byref(n)) == INVALID
    assert size(64, 64, -1, 0, ctypes.byref(n)) == INVALID
    assert size(0, 64, 4, 0, ctypes.byref(n)) == INVALID
    assert size(64, 65, 4, 0, ctypes.byref(n)) == UNSUPPORTED
    assert size(64, 64, 1 << 31, 0, ctypes.byref(n)) == UNSUPPORTED
    assert size(1 << 20, 64, 1 << 30, 2, ctypes.byref(n)) == UNSUPPORTED   # more GPU threads than a launch has
    assert size((1 << 20) + 1, 64, 4, 0, ctypes.byref(n)) == UNSUPPORTED
    assert size(64, (1 << 20) + 32, 4, 0, ctypes.byref(n)) == UNSUPPORTED
    assert size(64, 64, 4, 0, ctypes.byref(n)) == 0 and n.value == 0
    m = uw._lib.uw_matmul_fp8
    assert m(None, P, 64, 64, P, 4, P, 0, None, 0, None) == INVALID
    assert m(P, None, 64, 64, P, 4, P, 0, None, 0, None) == INVALID
    assert m(P, P + 2, 64, 64, P, 4, P, 0, None, 0, None) == INVALID
    assert m(P, P, 64, 64, P + 2, 4, P, 0, None, 0, None) == INVALID
    assert m(P, P, 64, 64, P, 4, P + 8, 0, None, 0, None) == INVALID
    assert m(P, P, 64, 64, P, 4, P, 0, P + 8, 0, None) == INVALID
    assert m(P, P, 64, 64, P, 4, P, 1, None, 0, None) == INVALID
    assert size(64, 64, 4000, 2, ctypes.byref(n)) == 0 and n.value > 0     # x in 8 bits
    assert m(P, P, 64, 64, P, 4000, P, 2, None, 0, None) == WORKSPACE
    assert m(P, P, 64, 64, P, 4000, P, 2, P, n.value - 1, None) == WORKSPACE
    assert m(P, P, 64, 64, P, 0, P, 0, None, 0, None) == 0


def test_sets_refuse(uw):
    h = ctypes.c_void_p()
    mk, r = uw._lib.uw_experts_fp8, ctypes.byref(h)
    assert mk(P, P, 4, 64, 160, 0, 0, r) == 0 and h.value
    uw._lib.uw_free_experts(h)
    for args, want in [((None, P, 4, 64, 64, 0, 0), INVALID), ((P, None, 4, 64, 64, 0, 0), INVALID),
                       ((P + 8, P, 4, 64, 64, 0, 0), INVALID), ((P, P + 2, 4, 64, 64, 0, 0), INVALID),
                       ((P, P, 0, 64, 64, 0, 0), INVALID), ((P, P, 4, 64, 64, 64 * 64 - 16, 0), INVALID),
                       ((P, P, 4, 129, 160, 0, 3), INVALID), ((P, P, 4, 64, 64, 64 * 64 + 8, 0), UNSUPPORTED),
                       ((P, P, 1025, 64, 64, 0, 0), UNSUPPORTED), ((P, P, 4, 64, 48, 0, 0), UNSUPPORTED),
                       ((P, P, 4, 64, 64, 0, 1 << 61), UNSUPPORTED)]:
        assert mk(*args, r) == want and not h.value, args
    assert mk(P, P, 4, 64, 64, 0, 0, None) == INVALID


def test_layer_refusals(uw):
    gate, up, down = bf16_set(uw), bf16_set(uw), bf16_set(uw)
    wide, few = bf16_set(uw, n=96), bf16_set(uw, count=3)
    n = ctypes.c_size_t()
    size = uw._lib.uw_workspace_size_expert_layer
    assert size(None, down, 4, 2, ctypes.byref(n)) == INVALID
    assert size(gate, None, 4, 2, ctypes.byref(n)) == INVALID
    assert size(gate, down, 4, 2, None) == INVALID
    assert size(gate, down, -1, 2, ctypes.byref(n)) == INVALID
    assert size(gate, down, 4, 5, ctypes.byref(n)) == INVALID
    assert size(gate, wide, 4, 2, ctypes.byref(n)) == INVALID      # shapes that are not each other's transposes
    assert size(gate, few, 4, 2, ctypes.byref(n)) == INVALID
    assert size(gate, down, 4, 2, ctypes.byref(n)) == 0
    need = n.value
    assert need >= 2 * 8 * 64
    f = uw._lib.uw_expert_layer

    def call(gate=gate, up=up, down=down, logits=P, type=0, tokens=4, ld=4, topk=2, scoring=1, ids=P, weights=P, off=P,
             rows=P, slots=P, x=P, out=P, ws=P, nb=need):
        return f(gate, up, down, logits, type, tokens, ld, None, topk, scoring, ids, weights, off, rows, slots, x, out,
                 ws, nb, None)

    for kw in (dict(gate=None), dict(up=None), dict(down=None), dict(logits=None), dict(type=2), dict(tokens=-1),
               dict(ld=3), dict(topk=0), dict(topk=5), dict(scoring=3), dict(ids=None), dict(weights=None),
               dict(off=None), dict(rows=None), dict(slots=None), dict(x=None), dict(out=None), dict(x=P + 8),
               dict(out=P + 2), dict(ws=P + 8)):
        assert call(**kw) == INVALID, kw
    assert call(ws=None) == WORKSPACE
    assert call(nb=need - 1) == WORKSPACE
    assert call(tokens=17) == WORKSPACE                            # the two calls' workspaces
    for h in (gate, up, down, wide, few):
        uw._lib.uw_free_experts(h)


def test_binding_refuses(uw):
    e8, f32 = torch.float8_e4m3fn, torch.float32
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    assert uw.fp8_scale_shape(129, 160, 128) == (2, 2) and uw.fp8_scale_shape(5, 128) == (5, 1)
    for src, elem, scale, br in [
            (x.half(), torch.zeros(4, 64, dtype=e8), torch.zeros(4, 1), 1),
            (x, torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4, 1), 1),
            (x, torch.zeros(4, 32, dtype=e8), torch.zeros(4, 1), 1),
            (x, torch.zeros(4, 64, dtype=e8), torch.zeros(1, 1), 1),
            (x, torch.zeros(4, 64, dtype=e8), torch.zeros(4, 1), 128),
            (x, torch.zeros(4, 64, dtype=e8), torch.zeros(4, 1), 64),
            (x, torch.zeros(4, 64, dtype=e8), torch.zeros(4, 1), 1)]:   # the last: on no device
        with pytest.raises(ValueError):
            uw.uw_quantize_fp8(src, elem, scale, br)
    with pytest.raises(ValueError):
        uw.uw_matmul_fp8(torch.zeros(8, 64, dtype=e8), torch.zeros(1, 1), x, torch.zeros(4, 8, dtype=f32))
    with pytest.raises(ValueError):
        uw.uw_experts_fp8(torch.zeros(8, 64), torch.zeros(1, 1), 1, 8, 64)
    with pytest.raises(ValueError):
        uw.uw_experts_fp8(torch.zeros(8, 64, dtype=e8), torch.zeros(1, 1).half(), 1, 8, 64)
