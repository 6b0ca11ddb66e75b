"""MXFP4 products at the ends of their range, on the GPU against plain implementations."""
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
