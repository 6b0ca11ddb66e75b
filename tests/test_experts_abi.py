"""What the expert and MXFP4 calls refuse, on the host alone: no device is touched."""
import ctypes

import pytest
import torch

INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -7
P = 4096   # an aligned address that no refused call reads


@pytest.fixture(scope="module")
def uw():
    from decode_gemm_exp_amd import uw as _uw
    return _uw


def bf16_set(uw, count=4, n=64, k=64, w=P, stride=0):
    h = ctypes.c_void_p()
    return uw._lib.uw_experts_bf16(w, count, n, k, stride, ctypes.byref(h)), h


def test_mx4_conversion_refusals(uw):
    q, d = uw._lib.uw_quantize_mx4, uw._lib.uw_dequantize_mx4
    assert q(None, 1, 4, 64, 64, P, P, None) == INVALID
    assert q(P, 1, 4, 64, 64, None, P, None) == INVALID
    assert q(P, 1, 4, 64, 64, P, None, None) == INVALID
    assert q(P, 2, 4, 64, 64, P, P, None) == INVALID          # type
    assert q(P, 1, -1, 64, 64, P, P, None) == INVALID
    assert q(P, 1, 4, 0, 64, P, P, None) == INVALID
    assert q(P, 1, 4, 48, 64, P, P, None) == UNSUPPORTED      # a block is 32
    assert q(P, 1, 4, 64, 32, P, P, None) == INVALID          # rows overlap
    assert q(P, 1, 4, 64, 68, P, P, None) == UNSUPPORTED      # rows not on 16 bytes
    assert q(P + 2, 1, 4, 64, 64, P, P, None) == INVALID
    assert q(P, 1, 4, 64, 64, P + 4, P, None) == INVALID
    assert q(P, 1, 4, 64, 64, P, P + 1, None) == INVALID
    assert q(P, 1, 0, 64, 64, P, P, None) == 0                # nothing to do
    assert d(None, P, 4, 64, P, 64, None) == INVALID
    assert d(P, P, 4, 64, None, 64, None) == INVALID
    assert d(P, P, 4, 40, P, 64, None) == UNSUPPORTED
    assert d(P, P, 4, 64, P, 60, None) == INVALID
    assert d(P, P, 4, 64, P, 65, None) == UNSUPPORTED
    assert d(P, P, 4, 64, P + 8, 64, None) == INVALID
    assert d(P, P, 0, 64, P, 64, None) == 0


def test_mx4_product_refusals(uw):
    n = ctypes.c_size_t()
    size = uw._lib.uw_workspace_size_mx4
    assert size(64, 64, 4, 0, None) == INVALID
    assert size(64, 64, 4, 2, ctypes.byref(n)) == INVALID
    assert size(64, 64, -1, 0, ctypes.byref(n)) == INVALID
    assert size(0, 64, 4, 0, ctypes.byref(n)) == INVALID
    assert size(64, 65, 4, 0, ctypes.byref(n)) == UNSUPPORTED
    assert size(64, 64, 1 << 31, 0, ctypes.byref(n)) == UNSUPPORTED
    assert size((1 << 20) + 1, 64, 4, 0, ctypes.byref(n)) == UNSUPPORTED
    assert size(64, (1 << 20) + 32, 4, 0, ctypes.byref(n)) == UNSUPPORTED
    m = uw._lib.uw_matmul_mx4
    assert m(None, P, 64, 64, P, 4, P, 0, None, 0, None) == INVALID
    assert m(P, P, 64, 64, P + 2, 4, P, 0, None, 0, None) == INVALID
    assert m(P, P, 64, 64, P, 4, P, 0, P + 8, 0, None) == INVALID
    assert m(P, P, 64, 64, P, 4, P, 1, None, 0, None) == WORKSPACE
    assert m(P, P, 64, 64, P, 4, P, 1, P, 16, None) == WORKSPACE
    assert m(P, P, 64, 64, P, 0, P, 0, None, 0, None) == 0


def test_expert_sets_refuse(uw):
    f = uw._lib.uw_free_experts
    st, h = bf16_set(uw)
    assert st == 0 and h.value
    f(h)
    f(None)
    for kw, want in [(dict(count=0), INVALID), (dict(n=0), INVALID), (dict(k=-32), INVALID), (dict(w=None), INVALID),
                     (dict(w=P + 2), INVALID), (dict(stride=64), INVALID), (dict(stride=64 * 64 + 1), UNSUPPORTED),
                     (dict(k=40), UNSUPPORTED), (dict(count=1025), UNSUPPORTED)]:
        st, h = bf16_set(uw, **kw)
        assert st == want and not h.value, kw
    h = ctypes.c_void_p()
    mk = uw._lib.uw_experts_mx4
    r = ctypes.byref(h)
    assert mk(P, P, 4, 64, 160, 0, 0, r) == 0
    f(h)
    assert mk(None, P, 4, 64, 64, 0, 0, r) == INVALID and not h.value
    assert mk(P, P + 1, 4, 64, 64, 0, 0, r) == INVALID
    assert mk(P, P, 4, 64, 64, 64 * 32 - 16, 0, r) == INVALID
    assert mk(P, P, 4, 64, 64, 64 * 32 + 8, 0, r) == UNSUPPORTED
    assert mk(P, P, 4, 64, 64, 0, 64 * 4 + 2, r) == UNSUPPORTED
    assert uw._lib.uw_experts_uwf1(None, 2, None, r) == INVALID
    assert uw._lib.uw_experts_uwf1((ctypes.c_void_p * 2)(None, None), 2, None, r) == INVALID
    assert uw._lib.uw_experts_bf16(P, 4, 64, 64, 0, None) == INVALID


def test_routing_refusals(uw):
    n = ctypes.c_size_t()
    size = uw._lib.uw_workspace_size_route
    assert size(8, 4, 2, None) == INVALID
    assert size(-1, 4, 2, ctypes.byref(n)) == INVALID
    assert size(8, 4, 5, ctypes.byref(n)) == INVALID
    assert size(8, 1025, 2, ctypes.byref(n)) == UNSUPPORTED
    assert size(8, 64, 17, ctypes.byref(n)) == UNSUPPORTED
    assert size(1 << 30, 64, 2, ctypes.byref(n)) == UNSUPPORTED
    assert size(8, 64, 2, ctypes.byref(n)) == 0 and n.value == 0
    assert size(5000, 64, 2, ctypes.byref(n)) == 0 and n.value > 0
    r = uw._lib.uw_route_experts

    def call(logits=P, type=0, tokens=8, experts=4, ld=4, topk=2, scoring=1, ids=P, weights=P, off=P, rows=P, slots=P,
             ws=None, nb=0):
        return r(logits, type, tokens, experts, ld, None, topk, scoring, ids, weights, off, rows, slots, ws, nb, None)

    for kw in (dict(logits=None), dict(type=5), dict(scoring=3), dict(scoring=-1), dict(ld=3), dict(ids=None),
               dict(weights=None), dict(off=None), dict(rows=None), dict(slots=None), dict(topk=0), dict(tokens=-2)):
        assert call(**kw) == INVALID, kw
    assert call(tokens=5000) == WORKSPACE
    assert call(tokens=5000, ws=P, nb=16) == WORKSPACE
    assert uw._lib.uw_plan_experts(None, 8, 4, 2, P, P, P, None, 0, None) == INVALID
    assert uw._lib.uw_plan_experts(P, 8, 4, 2, P, None, P, None, 0, None) == INVALID
    assert uw._lib.uw_plan_experts(P, 5000, 4, 2, P, P, P, None, 0, None) == WORKSPACE


def test_grouped_product_refusals(uw):
    _, a = bf16_set(uw)
    _, b = bf16_set(uw, n=32)
    m, g = uw._lib.uw_matmul_experts, uw._lib.uw_matmul_experts_gated
    assert m(None, P, P, 8, P, 8, P, None) == INVALID
    assert m(a, None, P, 8, P, 8, P, None) == INVALID
    assert m(a, P, P, 8, None, 8, P, None) == INVALID
    assert m(a, P, P, 8, P, 8, None, None) == INVALID
    assert m(a, P, P, -1, P, 8, P, None) == INVALID
    assert m(a, P, P, 8, P, 0, P, None) == INVALID
    assert m(a, P, None, 8, P, 7, P, None) == INVALID       # slot s is row s: there must be as many
    assert m(a, P, P, 8, P + 2, 8, P, None) == INVALID
    assert m(a, P, P, 1 << 31, P, 8, P, None) == UNSUPPORTED
    assert g(a, None, P, P, 8, P, 8, P, None) == INVALID
    n = ctypes.c_size_t()
    size = uw._lib.uw_workspace_size_expert_mlp
    assert size(a, None, 8, 2, ctypes.byref(n)) == INVALID
    assert size(a, b, 8, 2, ctypes.byref(n)) == INVALID     # down is not [k][n]
    assert size(a, a, 8, 5, ctypes.byref(n)) == INVALID     # topk > experts
    assert size(a, a, 8, 2, ctypes.byref(n)) == 0
    mlp = uw._lib.uw_expert_mlp
    assert mlp(a, None, a, 8, 2, P, P, P, P, P, P, P, n.value, None) == INVALID
    assert mlp(a, a, a, 8, 2, P, P, P, P, P, P, None, 0, None) == WORKSPACE
    assert mlp(a, a, a, 8, 2, P, P, P, P, P, P, P, n.value - 1, None) == WORKSPACE
    assert mlp(a, a, a, 8, 2, P, None, P, P, P, P, P, n.value, None) == INVALID
    assert mlp(a, a, a, 0, 2, P, P, P, P, P, P, None, 0, None) == 0
    for h in (a, b):
        uw._lib.uw_free_experts(h)


def test_binding_refuses_what_pointers_cannot_say(uw):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    e, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 4, dtype=torch.uint8)
    with pytest.raises(ValueError):
        uw.uw_quantize_mx4(x, e, s)                  # host tensors
    with pytest.raises(ValueError):
        uw.uw_quantize_mx4(x.half(), e, s)
    with pytest.raises(ValueError):
        uw.uw_matmul_mx4(e, s, x, torch.zeros(4, 4))
    with pytest.raises(ValueError):
        uw.uw_experts_bf16(x, 4, 1, 64)
    r = uw.Routing(4, 8, 2, device="cpu")
    assert r.rows.shape == (8,) and r.offsets.shape == (9,)
    with pytest.raises(ValueError):
        uw.uw_route_experts(torch.zeros(4, 8), r)
    with pytest.raises(ValueError):
        uw.uw_route_experts(torch.zeros(4, 8), r, "top")
    with pytest.raises(uw.UwError):
        uw.Routing(4, 8, 9, device="cpu")


def test_expert_sets_refuse_views_that_pointers_cannot_say(uw, monkeypatch):
    """A transposed, sliced or expanded stack is no stack of [n][k]; views that are one are taken."""
    monkeypatch.setattr(uw, "_on_device", lambda *a: None)   # host tensors: the sets are never multiplied by
    e, n, k = 3, 8, 64
    w = torch.zeros(e, n, k, dtype=torch.bfloat16)
    both = torch.zeros(e, 2, n, k, dtype=torch.bfloat16)
    fused = both.view(e, 2 * n, k)
    taken = [(w, 0), (w.view(e * n, k), 0), (w.view(-1), 0), (w.view(1, e * n, k), 0), (both, 2 * n * k), (both[:, 1], 2 * n * k),
             (both[:, :1], 2 * n * k), (fused, 2 * n * k), (fused[:, n:], 2 * n * k), (both[0, 1], 2 * n * k),
             (torch.zeros(e + 2, n, k, dtype=torch.bfloat16), 0), (torch.zeros(2 * e, n, k, dtype=torch.bfloat16)[::2], 2 * n * k)]
    for t, stride in taken:
        uw.uw_experts_bf16(t, e, n, k, stride).free()
    square = torch.zeros(e, k, k, dtype=torch.bfloat16)
    refused = [(torch.zeros(e, k, n, dtype=torch.bfloat16).transpose(1, 2), n, 0),       # [K][N], transposed
               (torch.zeros(e, k, n, dtype=torch.bfloat16), n, 0),                       # ... or as it is
               (square.transpose(1, 2), k, 0), (square.permute(1, 0, 2), k, 0),
               (torch.zeros(e, n, 2 * k, dtype=torch.bfloat16)[:, :, :k], n, 0),         # gaps between rows
               (torch.zeros(e, n, 2 * k, dtype=torch.bfloat16)[:, :, ::2], n, 0),        # gaps inside rows
               (torch.zeros(e * n, 2 * k, dtype=torch.bfloat16)[:, :k], n, 0),
               (torch.zeros(2 * e * n * k, dtype=torch.bfloat16)[::2], n, 0),
               (both[:, 1], n, 0),                                                       # experts 2 n k apart
               (both[:, 1], n, 3 * n * k), (both[:2, 1], n, 2 * n * k),                  # not its stride, too few
               (both, n, 0), (fused, n, 0),                                              # which half?
               (w[:2], n, 0), (w[:1].expand(e, n, k), n, 0)]
    for t, rows, stride in refused:
        with pytest.raises(ValueError):
            uw.uw_experts_bf16(t, e, rows, k, stride)
    el, sc = torch.zeros(e, n, k // 2, dtype=torch.uint8), torch.zeros(e, n, 4, dtype=torch.uint8)
    uw.uw_experts_mx4(el, sc, e, n, k).free()
    el2, sc2 = torch.zeros(e, 2, n, k // 2, dtype=torch.uint8), torch.zeros(e, 2, n, 4, dtype=torch.uint8)
    uw.uw_experts_mx4(el2[:, 1], sc2[:, 1], e, n, k, n * k, 2 * n * 4).free()
    for a, b in ((el.transpose(1, 2), sc), (el, sc.transpose(1, 2)), (el2[:, 1], sc), (el, sc2[:, 1]),
                 (torch.zeros(e, k // 2, n, dtype=torch.uint8).transpose(1, 2), sc),
                 (el, torch.zeros(e, n, 8, dtype=torch.uint8)[:, :, :4])):
        with pytest.raises(ValueError):
            uw.uw_experts_mx4(a, b, e, n, k)


def test_calls_of_more_threads_than_a_launch_holds(uw):
    """2^32 threads are refused as unsupported before anything is launched, not as a failure of the device."""
    n = ctypes.c_size_t()
    size = uw._lib.uw_workspace_size_mx4
    for act in (0, 1):
        # 4096 tiles of columns, 512 threads each
        assert size(1 << 20, 32, (1 << 17) - 64, act, ctypes.byref(n)) == 0
        assert size(1 << 20, 32, 1 << 17, act, ctypes.byref(n)) == UNSUPPORTED   # 2^23 tiles
        assert size(1 << 20, 32, 1 << 20, act, ctypes.byref(n)) == UNSUPPORTED
        assert uw._lib.uw_matmul_mx4(P, P, 1 << 20, 32, P, 1 << 20, P, act, P, 1 << 62, None) == UNSUPPORTED
    assert uw._lib.uw_quantize_mx4(P, 1, 1 << 20, 1 << 20, 1 << 20, P, P, None) == UNSUPPORTED
    assert uw._lib.uw_dequantize_mx4(P, P, 1 << 20, 1 << 20, P, 1 << 20, None) == UNSUPPORTED
    _, gate = bf16_set(uw, n=32, k=1 << 20)
    _, down = bf16_set(uw, n=1 << 20, k=32)
    size = uw._lib.uw_workspace_size_expert_mlp
    assert size(gate, down, 1 << 14, 2, ctypes.byref(n)) == 0
    assert size(gate, down, 1 << 15, 2, ctypes.byref(n)) == UNSUPPORTED
    assert uw._lib.uw_expert_mlp(gate, gate, down, 1 << 20, 1, P, P, P, P, P, P, P, 1 << 62, None) == UNSUPPORTED
    for h in (gate, down):
        uw._lib.uw_free_experts(h)
