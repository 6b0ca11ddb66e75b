"""MXFP4 products at the ends of their range, in each of the kernels, on the GPU against plain implementations."""
import numpy as np
import pytest
import torch

from tests.test_gpu_mx4 import DEV, check_product, quantize_ref, unpack, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def uw():
    from decode_gemm_exp_amd import uw as _uw
    return _uw


def product(uw, elem, scale, x, act):
    n, k = elem.shape[0], 2 * elem.shape[1]
    y = torch.full((len(x), n), 7.0, device=DEV)
    ws = torch.empty(max(1, uw.uw_workspace_size_mx4(n, k, len(x), act)), dtype=torch.uint8, device=DEV)
    uw.uw_matmul_mx4(elem.to(DEV), scale.to(DEV), x.to(DEV), y, ws, act)
    return y


@pytest.mark.parametrize("byte", [252, 253, 254])
@pytest.mark.parametrize("act,batch", [(0, 1), (0, 8), (0, 9), (0, 300), (1, 1), (1, 8), (1, 9), (1, 300)])
@pytest.mark.parametrize("n", [48, 33000])
def test_weights_that_overflow_bf16(uw, n, act, batch, byte):
    """Infinite with x in BF16 and with x in 4 bits up to 8 rows (so x = 0 gives NaN), the value itself beyond."""
    k = 128
    g = torch.Generator().manual_seed(byte)
    elem = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, generator=g)
    elem[1] = 0x33                                   # 1.5: overflows at no scale
    scale = torch.full((n, 4), 100, dtype=torch.uint8)
    scale[: n // 2, 1] = byte                        # one block of the upper rows
    x = torch.randint(-3, 4, (batch, k), generator=g).float()
    x[batch // 2] = 0.0
    x = torch.ldexp(x, torch.tensor(-40)).bfloat16()
    y = product(uw, elem, scale, x, act).double().cpu().numpy()
    xv, wv = x.double().numpy(), values(unpack(elem), scale.numpy())
    if act:
        assert np.array_equal(values(*quantize_ref(xv)), xv)
    if not act or batch <= 8:
        with np.errstate(invalid="ignore"):
            wv = np.where(np.abs(wv) >= 2.0 ** 128, np.copysign(np.inf, wv), wv)
            ref = np.stack([(row * wv).sum(1) for row in xv])
    else:
        ref = xv @ wv.T
    assert np.array_equal(np.isnan(y), np.isnan(ref))
    over = np.isinf(ref)
    assert np.array_equal(y[over], ref[over])
    ok = np.isfinite(ref)
    mag = np.abs(xv) @ np.abs(np.where(np.isinf(wv), 0, wv)).T
    assert (np.abs(y[ok] - ref[ok]) <= k * 2.0 ** -23 * mag[ok]).all()
    if byte == 252 or (act and batch > 8):
        assert ok.all()
    else:
        assert np.isnan(y[batch // 2]).any()


@pytest.mark.parametrize("act,batch", [(0, 1), (0, 8), (0, 9), (1, 1), (1, 8), (1, 9)])
def test_one_weight_that_overflows_bf16(uw, act, batch):
    """6 2^127 alone, x not zero: an infinity of the product's sign, or the product."""
    n, k = 20, 128
    elem = torch.zeros(n, k // 2, dtype=torch.uint8)
    scale = torch.full((n, 4), 254, dtype=torch.uint8)
    for r in range(n):
        elem[r, 3 * r] = 0x07 if r % 2 else 0xF0         # 6 in an even column, -6 in an odd one
    x = torch.ldexp(torch.ones(batch, k) * (1 - 2 * (torch.arange(batch)[:, None] % 2)), torch.tensor(-40)).bfloat16()
    y = product(uw, elem, scale, x, act).cpu().double()
    sign = torch.where(torch.arange(n) % 2 == 1, 1.0, -1.0) * torch.sign(x[:, :1].double())
    assert torch.equal(y, sign * (6 * 2.0 ** 87 if act and batch > 8 else float("inf")))


# Sums of whole numbers below 2^24 are exact in FP32, in any order: one k too few or too many shows.
@pytest.mark.parametrize("batch,n,k", [(1, 40, 1 << 20), (2, 40, 28672), (9, 40, 28640), (16, 5001, 28672), (45, 700, 8224),
                                       (200, 300, 28640), (200, 16500, 8224), (200, 33000, 4192), (300, 33000, 4128),
                                       (130, 16500, 4128), (1, 1 << 20, 32), (300, 1 << 20, 32)])
@pytest.mark.parametrize("act", [0, 1])
def test_long_rows_and_columns_exactly(uw, act, batch, n, k):
    g = torch.Generator(device=DEV).manual_seed(n + k)
    w = torch.randint(1, 4, (n, k), generator=g, device=DEV, dtype=torch.int8)
    w *= 1 - 2 * torch.randint(0, 2, (n, k), generator=g, device=DEV, dtype=torch.int8)
    x = 1 - 2 * torch.randint(0, 2, (batch, k), generator=g, device=DEV).bfloat16()
    elem = torch.empty(n, k // 2, dtype=torch.uint8, device=DEV)
    scale = torch.empty(n, uw.mx4_scale_stride(k), dtype=torch.uint8, device=DEV)
    uw.uw_quantize_mx4(w.bfloat16(), elem, scale)                # (exact, as is x's)
    y = product(uw, elem, scale, x, act)
    for c in range(0, n, 1 << 16):
        want = x.double() @ w[c:c + (1 << 16)].double().T.contiguous()
        assert torch.equal(y[:, c:c + (1 << 16)].double(), want)


@pytest.mark.parametrize("batch,n", [(3, 70), (45, 70), (200, 16500), (200, 33000), (300, 33000)])
@pytest.mark.parametrize("act", [0, 1])
def test_nan_and_extreme_scales_in_every_kernel(uw, act, batch, n):
    """A NaN scale makes its row's outputs NaN and no other's, x of zero included; the smallest and large scales count in full."""
    k = 160
    g = torch.Generator().manual_seed(n + batch)
    elem = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, generator=g)
    for e in (0, 1, 127, 250):
        scale = torch.full((n, 8), e, dtype=torch.uint8)
        scale[:, 5:] = 255                                       # padding is never used
        x = torch.ldexp(torch.randint(-3, 4, (batch, k), generator=g).float(), torch.tensor(min(127 - e, 120))).bfloat16()
        y = product(uw, elem, scale, x, act)
        xv = x.double().numpy()
        check_product(y, values(*quantize_ref(xv)) if act else xv, values(unpack(elem), scale[:, :5].numpy()))
    scale = torch.full((n, 8), 120, dtype=torch.uint8)
    bad = [5, n // 2, n - 1]
    scale[bad[0], 0], scale[bad[1], 4], scale[bad[2], 2] = 255, 255, 255
    x = torch.randn(batch, k, generator=g).bfloat16()
    x[batch // 2] = 0.0
    nan = torch.isnan(product(uw, elem, scale, x, act).cpu())
    want = torch.zeros(n, dtype=torch.bool)
    want[bad] = True
    assert torch.equal(nan, want.expand(batch, n))
