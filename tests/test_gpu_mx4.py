"""MXFP4 conversion and product on the GPU against plain 64-bit implementations.

Tolerance of a product: each of the K products of two BF16 (or MXFP4) values is
exact in FP32, and each of at most K additions is off by at most one unit in
the last place of its result (2^-23 relative; the matrix unit's own adders
included), so |error| <= K 2^-23 sum |x w|.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
GRID = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


@pytest.fixture(scope="module")
def uw():
    from decode_gemm_exp_amd import uw as _uw
    return _uw


def quantize_ref(x: np.ndarray):
    """codes [rows][cols], scale bytes [rows][cols/32] of float64 x, by the definition."""
    b = x.reshape(x.shape[0], -1, 32)
    bad = ~np.isfinite(b).all(2)
    amax = np.abs(np.where(np.isfinite(b), b, 0)).max(2)
    e = np.where(amax > 0, np.frexp(amax)[1] - 3, -127).clip(-127, None)
    q = np.abs(np.where(bad[..., None], 0, b)) * np.exp2(-e.astype(np.float64))[..., None]
    # nearest grid value; of two equally near the one with the even code
    dist = np.abs(q[..., None] - GRID)
    near = dist == dist.min(-1, keepdims=True)
    even = near & (np.arange(8) % 2 == 0)
    code = np.where(even.any(-1), even.argmax(-1), near.argmax(-1))
    code = np.where(bad[..., None], 0, code + 8 * np.signbit(b))
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def unpack(elem: torch.Tensor):
    e = elem.cpu().numpy()
    return np.stack([e & 15, e >> 4], 2).reshape(e.shape[0], -1)


def values(code, byte):
    v = GRID[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(byte == 255, np.nan, np.exp2(byte.astype(np.float64) - 127))
    return (v.reshape(code.shape[0], -1, 32) * s[..., None]).reshape(code.shape)


def quantize(uw, x):
    rows, cols = x.shape
    elem = torch.full((rows, cols // 2), 0xAA, dtype=torch.uint8, device=DEV)
    scale = torch.full((rows, uw.mx4_scale_stride(cols)), 0xAA, dtype=torch.uint8, device=DEV)
    uw.uw_quantize_mx4(x, elem, scale)
    return elem, scale


def check_quantize(uw, x):
    elem, scale = quantize(uw, x)
    code, byte = quantize_ref(x.double().cpu().numpy())
    got = scale.cpu().numpy()
    nb = x.shape[1] // 32
    assert np.array_equal(got[:, :nb], byte)
    assert not got[:, nb:].any()
    assert np.array_equal(unpack(elem), code)
    out = torch.empty(x.shape, dtype=torch.bfloat16, device=DEV)
    uw.uw_dequantize_mx4(elem, scale, out)
    want = values(code, byte)
    o = out.double().cpu().numpy()
    assert np.array_equal(np.isnan(o), np.isnan(want))
    assert np.array_equal(np.nan_to_num(o), np.nan_to_num(want))


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (7, 96), (5, 4128), (64, 1024), (33, 160), (1000, 544)])
@pytest.mark.parametrize("f32", [False, True])
def test_quantize_shapes(uw, rows, cols, f32):
    g = torch.Generator().manual_seed(rows * cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=g).float())
    check_quantize(uw, (x if f32 else x.bfloat16()).to(DEV))


def test_quantize_every_bf16_value(uw):
    """Each 16-bit pattern as its block's largest, beside smaller ones, and in blocks of consecutive patterns."""
    p = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    check_quantize(uw, p.view(2048, 32).contiguous().to(DEV))
    f = p.float().nan_to_num(1.0, 1.0, 1.0)
    fractions = torch.tensor([1, .99, .9, .87, .8, .75, .7, .62, .6, .5, .45, .4, .37, .3, .25, .22, .2, .18, .15, .12,
                              .1, .08, .06, .04, .03, .02, .01, .001, 0, -.5, -.3, -1])
    check_quantize(uw, (f[:, None] * fractions).bfloat16().to(DEV))


def test_quantize_midpoints_and_extremes(uw):
    """Exact ties at every scale a float32 can have, subnormal and largest maxima, infinities and NaN."""
    mid = torch.tensor([4.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.999, -0.25, -0.75, -1.25, -1.75, -2.5,
                        -3.5, -5.0, -7.0, 0.2499, 0.7501, 1.2499, 1.7501, 2.4999, 3.5001, 5.0001, 0.0, -0.0, 0.001,
                        -0.001, 3.0, 1.0])
    e = torch.arange(-149, 126)
    x = torch.ldexp(mid.double()[None, :], e[:, None]).float()
    check_quantize(uw, x.to(DEV))
    odd = torch.zeros(6, 64)
    odd[0, 3] = float("inf")
    odd[1, 40] = float("-inf")
    odd[2, 0] = float("nan")
    odd[3, :] = 3.4e38
    odd[4, 5] = 1e-45
    check_quantize(uw, odd.to(DEV))
    check_quantize(uw, odd.bfloat16().to(DEV))


def test_strided_rows_leave_the_gap(uw):
    big = torch.randn(9, 200, device=DEV)
    src = big[:, 8:8 + 96]      # rows 200 apart, 32 bytes in
    assert src.data_ptr() % 16 == 0
    check_quantize(uw, src)
    elem, scale = quantize(uw, src)
    out = torch.full((9, 104), 7.0, dtype=torch.bfloat16, device=DEV)
    uw.uw_dequantize_mx4(elem, scale, out[:, :96])
    assert bool((out[:, 96:] == 7.0).all())
    want = values(*quantize_ref(src.double().cpu().numpy()))
    assert np.array_equal(out[:, :96].double().cpu().numpy(), want)


def test_dequantize_every_code_and_scale(uw):
    elem = torch.arange(256, dtype=torch.uint8).repeat(256, 1)           # 512 elements a row: every byte
    scale = torch.arange(256, dtype=torch.uint8)[:, None].repeat(1, 16)  # row r: scale r
    out = torch.empty(256, 512, dtype=torch.bfloat16, device=DEV)
    uw.uw_dequantize_mx4(elem.to(DEV), scale.to(DEV), out)
    want = torch.from_numpy(values(unpack(elem), scale.numpy())).to(torch.bfloat16)
    got = out.cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(), want.nan_to_num())


def product_case(uw, batch, n, k, act, seed, x=None):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(n, k, generator=g) * 0.02 * torch.exp2(torch.randn(n, 1, generator=g).round() * 2)
    elem, scale = quantize(uw, w.to(DEV))
    if x is None:
        x = torch.randn(batch, k, generator=g).bfloat16()
    x = x.to(DEV)
    y = torch.full((batch, n), float("nan"), device=DEV)
    ws = torch.empty(max(1, uw.uw_workspace_size_mx4(n, k, batch, act)), dtype=torch.uint8, device=DEV)
    uw.uw_matmul_mx4(elem, scale, x, y, ws, act)
    wv = values(*quantize_ref(w.double().numpy()))
    xv = x.double().cpu().numpy()
    if act:
        xv = values(*quantize_ref(xv))
    return y, xv, wv


def check_product(y, xv, wv):
    ref, mag = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    err = np.abs(y.double().cpu().numpy() - ref)
    tol = xv.shape[1] * 2.0 ** -23 * mag
    assert (err <= tol).all(), f"worst {np.max(err / np.maximum(tol, 1e-300))} of the tolerance"


@pytest.mark.parametrize("batch", [1, 2, 15, 16, 17, 33, 64, 65, 129, 300])
@pytest.mark.parametrize("n,k", [(1, 32), (16, 64), (33, 96), (200, 544), (257, 1024)])
@pytest.mark.parametrize("act", [0, 1])
def test_product(uw, batch, n, k, act):
    check_product(*product_case(uw, batch, n, k, act, batch * 1000 + n))


@pytest.mark.parametrize("batch,n,k,act", [(1, 5000, 4096, 0), (128, 1030, 2080, 0), (515, 770, 1056, 1),
                                           (1024, 512, 4096, 1), (260, 1025, 8192, 1), (2, 40, 28672, 0)])
def test_product_larger(uw, batch, n, k, act):
    check_product(*product_case(uw, batch, n, k, act, 5))


# enough blocks for the tiles of 256 and 128 rows (4-bit x) and of 64 rows (BF16 x)
@pytest.mark.parametrize("batch,n,k,act", [(700, 16500, 160, 1), (300, 23001, 96, 1), (130, 23001, 288, 1),
                                           (300, 16500, 160, 0), (45, 20000, 288, 0), (8, 20000, 544, 0),
                                           (9, 700, 2080, 0), (40, 8000, 1120, 0), (16, 16500, 96, 0)])
def test_product_many_blocks(uw, batch, n, k, act):
    check_product(*product_case(uw, batch, n, k, act, 6))


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("batch", [3, 140])
def test_product_not_finite(uw, act, batch):
    """An infinity or a NaN in a row of x reaches that row's outputs and no other's."""
    k, n = 160, 70
    x = torch.randn(batch, k).bfloat16()
    clean = product_case(uw, batch, n, k, act, 9, x)[0].cpu()
    x2 = x.clone()
    x2[1, 159] = float("nan")
    x2[2, 0] = float("inf")
    y = product_case(uw, batch, n, k, act, 9, x2)[0].cpu()
    keep = [i for i in range(batch) if i not in (1, 2)]
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[1]).all()
    assert not torch.isfinite(y[2]).any()


@pytest.mark.parametrize("batch", [1, 40, 200])
@pytest.mark.parametrize("act", [0, 1])
def test_product_extreme_scales(uw, batch, act):
    """Weights whose values are subnormal in BF16, or near its largest, count in full."""
    k, n = 128, 32
    for e in (0, 1, 2, 127, 250):
        elem = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8)
        scale = torch.full((n, 4), e, dtype=torch.uint8)
        x = torch.ldexp(torch.randint(-3, 4, (batch, k)).float(), torch.tensor(min(127 - e, 120))).bfloat16()
        y = torch.empty(batch, n, device=DEV)
        ws = torch.empty(max(1, uw.uw_workspace_size_mx4(n, k, batch, act)), dtype=torch.uint8, device=DEV)
        uw.uw_matmul_mx4(elem.to(DEV), scale.to(DEV), x.to(DEV), y, ws, act)
        xv = x.double().numpy()
        check_product(y, values(*quantize_ref(xv)) if act else xv, values(unpack(elem), scale.numpy()))


def test_product_nan_scale(uw):
    """A NaN block makes its row's outputs NaN and leaves the others."""
    for batch in (1, 200):
        for act in (0, 1):
            k, n = 256, 48
            elem = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8)
            scale = torch.full((n, 8), 120, dtype=torch.uint8)
            scale[5, 3] = 255
            x = torch.randn(batch, k).bfloat16()
            y = torch.empty(batch, n, device=DEV)
            ws = torch.empty(max(1, uw.uw_workspace_size_mx4(n, k, batch, act)), dtype=torch.uint8, device=DEV)
            uw.uw_matmul_mx4(elem.to(DEV), scale.to(DEV), x.to(DEV), y, ws, act)
            bad = torch.isnan(y.cpu())
            assert bad[:, 5].all() and int(bad.sum()) == batch


def test_repeats_bit_for_bit_and_on_another_stream(uw):
    for act in (0, 1):
        a = product_case(uw, 130, 300, 1024, act, 3)[0]
        b = product_case(uw, 130, 300, 1024, act, 3)[0]
        assert torch.equal(a, b)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            c = product_case(uw, 130, 300, 1024, act, 3)[0]
        s.synchronize()
        assert torch.equal(a, c)


def test_captured(uw):
    """One graph of quantise, product and dequantise, replayed on new data."""
    n, k, batch = 96, 512, 70
    w = torch.randn(n, k, device=DEV)
    x = torch.randn(batch, k, device=DEV).bfloat16()
    elem = torch.empty(n, k // 2, dtype=torch.uint8, device=DEV)
    scale = torch.empty(n, uw.mx4_scale_stride(k), dtype=torch.uint8, device=DEV)
    back = torch.empty(n, k, dtype=torch.bfloat16, device=DEV)
    y = torch.empty(batch, n, device=DEV)
    ws = torch.empty(uw.uw_workspace_size_mx4(n, k, batch, uw.ACT_MX4), dtype=torch.uint8, device=DEV)

    def step():
        uw.uw_quantize_mx4(w, elem, scale)
        uw.uw_matmul_mx4(elem, scale, x, y, ws, uw.ACT_MX4)
        uw.uw_dequantize_mx4(elem, scale, back)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(4):
        w.copy_(torch.randn(n, k, generator=torch.Generator().manual_seed(i)))
        x.copy_(torch.randn(batch, k, generator=torch.Generator().manual_seed(50 + i)))
        g.replay()
        torch.cuda.synchronize()
        got = (y.clone(), back.clone())
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], y) and torch.equal(got[1], back)
        check_product(got[0], values(*quantize_ref(x.double().cpu().numpy())),
                      values(*quantize_ref(w.double().cpu().numpy())))
