"""FP8 products and the layer where sizes, addresses and splits are extreme.

Whole numbers: elements and x in -2 .. 2 at scales of one give sums far below 2^24, exact in FP32
whatever their order, so results are equal, not near.
"""
import pytest
import torch

from tests import test_gpu_fp8_blocks as fp8
from tests import test_gpu_layer as layer
from tests.test_gpu_experts import h_ref, route_ref, weights

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def uw():
    from decode_gemm_exp_amd import uw as _uw
    return _uw


def whole_numbers(g, *shape):
    return torch.randint(-2, 3, shape, generator=g).float().to(DEV)


def ones(uw, n, k):
    return torch.ones(uw.fp8_scale_shape(n, k, 128), device=DEV)


# Row tiles of 64 and 128, tiles that all go in slices of K, whole rounds of tiles with a last one in slices (289 and
# 300 tiles of 128 rows), columns that end inside a tile and are no multiple of four, a K tail.
@pytest.mark.parametrize("batch,n,k", [(333, 4096, 14336), (200, 5001, 8224), (2100, 4100, 4096), (1500, 6400, 2080),
                                       (129, 257, 20000), (1100, 300, 9600), (640, 14337, 1056)])
@pytest.mark.parametrize("act", ["bf16", "fp8"])
def test_slices_of_k_exactly(uw, batch, n, k, act):
    g = torch.Generator().manual_seed(n + k)
    w, x = whole_numbers(g, n, k), whole_numbers(g, batch, k)
    a = uw.ACT_BF16
    if act == "fp8":
        a = uw.ACT_FP8
        x[:, ::128] = 448.0           # x's own scales are one
        w[:, ::128] = 0.0
    elem, scale, xb = w.to(torch.float8_e4m3fn), ones(uw, n, k), x.bfloat16()
    nb = uw.uw_workspace_size_fp8(n, k, batch, a)
    assert nb > 0 or batch <= 256 or k < 2000   # (the rows kernel and whole tiles need none)
    y = torch.full((batch + 1, n), 7.0, device=DEV)
    for fill in (0, 255):             # whatever the workspace held
        ws = torch.full((nb + 256,), fill, dtype=torch.uint8, device=DEV)
        uw.uw_matmul_fp8(elem, scale, xb, y[:batch], ws[:nb], a)
        assert torch.equal(y[:batch], x @ w.T)
        assert bool((y[batch] == 7.0).all()) and bool((ws[nb:] == fill).all())


# Blocks of 20, 24, 32, 36 and 44 rows of the matrix, some of which end in the next row of scale blocks, with the last
# block cut off; a number of columns that is no multiple of four; one to three groups of rows of x.
@pytest.mark.parametrize("n,k", [(4500, 160), (5001, 2080), (5900, 1056), (8300, 96), (9000, 544), (17001, 224),
                                 (22400, 128)])
@pytest.mark.parametrize("batch", [1, 7, 13, 16, 20, 33])
@pytest.mark.parametrize("act", ["bf16", "fp8"])
def test_rows_that_straddle_scale_blocks_exactly(uw, n, k, batch, act):
    """Scales are powers of two from 1/4 to 4, every one of a block's neighbours another."""
    g = torch.Generator().manual_seed(n + k + batch)
    w, x = whole_numbers(g, n, k), whole_numbers(g, batch, k)
    a = uw.ACT_BF16
    if act == "fp8":
        a = uw.ACT_FP8
        x[:, ::128] = 448.0           # x's own scales are one
        w[:, ::128] = 0.0
    i, j = (torch.arange(m, device=DEV) for m in uw.fp8_scale_shape(n, k, 128))
    scale = torch.exp2((2.0 * i[:, None] + j) % 5 - 2)
    wide = w * scale.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    y = torch.full((batch + 1, n), 7.0, device=DEV)
    ws = torch.empty(uw.uw_workspace_size_fp8(n, k, batch, a), dtype=torch.uint8, device=DEV)
    uw.uw_matmul_fp8(w.to(torch.float8_e4m3fn), scale, x.bfloat16(), y[:batch], ws, a)
    assert torch.equal(y[:batch].double(), x.double() @ wide.double().T)
    assert bool((y[batch] == 7.0).all())


def test_workspace_too_small_is_refused(uw):
    n, k, batch = 4096, 14336, 333
    elem = torch.zeros(n, k, dtype=torch.uint8, device=DEV)
    x, y = torch.zeros(batch, k, dtype=torch.bfloat16, device=DEV), torch.full((batch, n), 7.0, device=DEV)
    nb = uw.uw_workspace_size_fp8(n, k, batch)
    for ws in (None, torch.empty(nb - 1, dtype=torch.uint8, device=DEV)):
        with pytest.raises(uw.UwError) as err:
            uw.uw_matmul_fp8(elem, ones(uw, n, k), x, y, ws)
        assert err.value.status == -7
    with pytest.raises(ValueError):
        uw.uw_matmul_fp8(elem, ones(uw, n, k), x.T.contiguous().T, y)
    torch.cuda.synchronize()
    assert bool((y == 7.0).all())


@pytest.mark.parametrize("act", ["bf16", "fp8"])
def test_product_of_x_past_two_gib(uw, act):
    g = torch.Generator().manual_seed(2)
    batch, n, k = 140000, 70, 8192    # 2.3 GB of x
    a = uw.ACT_FP8 if act == "fp8" else uw.ACT_BF16
    elem, scale = fp8.fp8_weights(uw, g, n, k)
    part = torch.randn(batch // 1000, k, generator=g).bfloat16().to(DEV)
    x = part.repeat_interleave(1000, 0)   # row r holds part[r // 1000]
    y = torch.empty(batch, n, device=DEV)
    ws = torch.empty(max(16, uw.uw_workspace_size_fp8(n, k, batch, a)), dtype=torch.uint8, device=DEV)
    uw.uw_matmul_fp8(elem, scale, x, y, ws, a)
    xv = fp8.values(*fp8.quantize(uw, part, 1), 1) if act == "fp8" else part.double()
    w = fp8.values(elem, scale, 128).T.contiguous()
    ref, mag = xv @ w, xv.abs() @ w.abs()
    err = (y.view(-1, 1000, n).double() - ref[:, None]).abs()
    assert bool((err <= ((k + 16) * 2.0 ** -23 * mag)[:, None]).all())


@pytest.mark.parametrize("per", [2, 300])
def test_experts_of_x_past_two_gib(uw, per):
    """Row indices whose bytes pass 2^31 and 2^32, plain and gated."""
    g = torch.Generator().manual_seed(per)
    n, k, x_rows = 40, 8192, 270000   # 4.4 GB
    h, wv = fp8.make_set(uw, weights(g, 2, n, k))
    h2, uv = fp8.make_set(uw, weights(g, 2, n, k))
    off = torch.tensor([0, per, 2 * per + 1], dtype=torch.int32)
    rows = torch.randint(0, x_rows, (2 * per + 1,), generator=g, dtype=torch.int32)
    rows[0], rows[1], rows[-1] = x_rows - 1, 131072, 0
    part = torch.randn(x_rows // 1000, k, generator=g).bfloat16()
    x = part.to(DEV).repeat_interleave(1000, 0)
    y = torch.empty(2 * per + 1, n, device=DEV)
    uw.uw_matmul_experts(h, off.to(DEV), rows.to(DEV), x, y)
    f = (k + 16) / k
    ref, mag = fp8.grouped_ref(off, rows // 1000, part, wv)
    assert bool(((y.double().cpu() - ref).abs() <= k * 2.0 ** -23 * mag * f).all())
    hh = torch.empty(2 * per + 1, n, dtype=torch.bfloat16, device=DEV)
    uw.uw_matmul_experts_gated(h2, h, off.to(DEV), rows.to(DEV), x, hh)
    gv, ga = fp8.grouped_ref(off, rows // 1000, part, uv)
    want, tol = h_ref(gv, ga * f, ref, mag * f, k)
    assert bool(((hh.double().cpu() - want).abs() <= tol).all())


@pytest.mark.parametrize("experts,per,n,k", [(2, 40, 20000, 96), (3, 700, 40, 20000), (5, 3, 33, 32768), (4, 300, 5000, 64)])
def test_long_rows_and_columns_exactly(uw, experts, per, n, k):
    g = torch.Generator().manual_seed(per)
    w = whole_numbers(g, experts, n, k)
    h = uw.uw_experts_fp8(w.to(torch.float8_e4m3fn), torch.ones(experts, *uw.fp8_scale_shape(n, k, 128), device=DEV),
                          experts, n, k)
    slots = experts * per
    x = whole_numbers(g, 50, k)
    off = (torch.arange(experts + 1) * per).to(torch.int32).to(DEV)
    rows = torch.randint(0, 50, (slots,), generator=g, dtype=torch.int32).to(DEV)
    y = torch.empty(slots, n, device=DEV)
    uw.uw_matmul_experts(h, off, rows, x.bfloat16(), y)
    for e in range(experts):
        s = slice(e * per, (e + 1) * per)
        assert torch.equal(y[s], x[rows[s].long()] @ w[e].T)


# ---------------------------------------------------------------- layer -----

@pytest.mark.parametrize("form", ["bf16", "mx4", "fp8"])
@pytest.mark.parametrize("tokens,experts,topk,n,k", [(1, 1, 1, 32, 32), (16, 2, 2, 32, 64), (3, 5, 2, 32, 8192),
                                                     (2, 3, 1, 4128, 32), (16, 3, 3, 288, 160), (16, 600, 16, 32, 96),
                                                     (4, 33, 4, 96, 4128)])
def test_layer_sizes(uw, form, tokens, experts, topk, n, k):
    """The smallest, narrow and long ones; every token to every expert (several items an expert), nearly none shared."""
    g = torch.Generator().manual_seed(n + k)
    sets, vals = layer.build(uw, g, form, form, experts, n, k)
    l, x = torch.randn(tokens, experts, generator=g), torch.randn(tokens, k, generator=g).bfloat16()
    _, out = layer.run(uw, sets, l.to(DEV), x.to(DEV), topk, "softmax")
    ids, w = route_ref(l, topk, "softmax")
    ref, tol = layer.layer_ref(ids, w, experts, x, *vals)
    assert bool(((out.double().cpu() - ref).abs() <= tol).all())


def test_layer_without_any_expert(uw):
    """Every token masked: zeros, no slots, whatever the buffers held."""
    g = torch.Generator().manual_seed(1)
    sets, _ = layer.build(uw, g, "fp8", "fp8", 6, 96, 160)
    for tokens in (1, 16, 30):
        l = torch.full((tokens, 6), float("-inf"), device=DEV)
        r, out = layer.run(uw, sets, l, torch.randn(tokens, 160, device=DEV).bfloat16(), 3)
        assert bool((out == 0).all()) and bool((r.ids == -1).all()) and bool((r.slots == -1).all())
        assert bool((r.offsets == 0).all()) and bool((r.weights == 0).all())


def test_layer_writes_its_outputs_alone(uw):
    """Guards around every output, a strided router, and a stream that is not torch's current one."""
    g = torch.Generator().manual_seed(4)
    tokens, experts, topk, n, k = 7, 20, 3, 160, 288
    sets, _ = layer.build(uw, g, "mx4", "fp8", experts, n, k)
    wide = torch.randn(tokens, experts + 9, generator=g).to(DEV)
    l, x = wide[:, 4:4 + experts], torch.randn(tokens, k, generator=g).bfloat16().to(DEV)
    r0, want = layer.run(uw, sets, l, x, topk)
    nb = uw.uw_workspace_size_expert_layer(sets[0], sets[2], tokens, topk)
    ws = torch.full((nb + 512,), 17, dtype=torch.uint8, device=DEV)
    out = torch.full((tokens + 2, k), 7.0, dtype=torch.bfloat16, device=DEV)
    r = uw.Routing(tokens, experts, topk, DEV)
    r.rows.fill_(-7)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    uw.uw_expert_layer(*sets, l, r, x, out[1:-1], ws[256:256 + nb], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(out[1:-1], want) and layer.same_routing(r, r0)
    assert bool((out[0] == 7).all()) and bool((out[-1] == 7).all())
    assert bool((ws[:256] == 17).all()) and bool((ws[256 + nb:] == 17).all())
    with pytest.raises(uw.UwError) as err:
        uw.uw_expert_layer(*sets, l, r, x, out[1:-1], ws[:nb - 1])
    assert err.value.status == -7
    with pytest.raises(ValueError):
        uw.uw_expert_layer(*sets, l, r, x[:, :k - 32], out[1:-1], ws)
    with pytest.raises(ValueError):
        uw.uw_expert_layer(*sets, l[:, 1:], r, x, out[1:-1], ws)
    mixed = layer.any_set(uw, "bf16", weights(g, experts, n, k))[0]
    with pytest.raises(uw.UwError) as err:   # gate and up in different forms
        uw.uw_expert_layer(sets[0], mixed, sets[2], l, r, x, out[1:-1], ws)
    assert err.value.status == -2
