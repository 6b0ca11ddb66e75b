"""Products grouped by expert where their inputs are odd, in each of the kernels: plans that do not ascend,
gates over the whole range of BF16.

Which kernel runs follows from the average rows an expert (all slots used) and
the blocks that tiles of 256 columns (gated: 128) make, 192 of them at least on
256 CUs: ``KERNELS`` holds rows an expert and columns that lead to each.
Tolerances are those of test_gpu_experts.
"""
import numpy as np
import pytest
import torch

from tests.test_gpu_experts import DEV, FORMS, grouped_ref, h_ref, make_set, weights

pytestmark = pytest.mark.gpu
KERNELS = {"rows": (3, 33), "tile64": (50, 16500), "tile128": (150, 16500), "tile256": (300, 16500)}
GUARD = 8   # rows on either side of an output


@pytest.fixture(scope="module")
def uw():
    from decode_gemm_exp_amd import uw as _uw
    return _uw


def guarded(slots, n, dtype):
    """(the whole array, its middle [slots][n]), 7 everywhere."""
    whole = torch.full((slots + 2 * GUARD, n), 7.0, dtype=dtype, device=DEV)
    return whole, whole[GUARD:GUARD + slots]


def grouped_dev(off, rows, x, w):
    """grouped_ref on the device, one expert at a time."""
    y = torch.zeros(len(rows), w.shape[1], dtype=torch.float64, device=DEV)
    a = torch.zeros_like(y)
    for e in range(w.shape[0]):
        s = slice(int(off[e]), int(off[e + 1]))
        if s.start < s.stop:
            xe, we = x[rows[s].long()].double().to(DEV), w[e].to(DEV).T.contiguous()
            y[s], a[s] = xe @ we, xe.abs() @ we.abs()
    return y, a


def check_plan_products(uw, sets, vals, off, x, rows, n, k):
    """Both products on the offsets ``off`` against the plan they are to be read as."""
    slots = len(rows)
    eff = np.maximum.accumulate(np.clip(np.asarray(off, np.int64), 0, slots))
    lo, hi = int(eff[0]), int(eff[-1])
    dev = torch.tensor(off, dtype=torch.int32, device=DEV), rows.to(DEV), x.to(DEV)
    ref, mag = grouped_dev(eff, rows, x, vals[0])
    up, up_mag = grouped_dev(eff, rows, x, vals[1])
    want, tol = h_ref(ref, mag, up, up_mag, k)
    for gated, dtype, value, bound in ((False, torch.float32, ref, k * 2.0 ** -23 * mag), (True, torch.bfloat16, want, tol)):
        first = None
        for _ in range(2):
            whole, y = guarded(slots, n, dtype)
            if gated:
                uw.uw_matmul_experts_gated(*sets, *dev, y)
            else:
                uw.uw_matmul_experts(sets[0], *dev, y)
            assert bool((whole[:GUARD + lo] == 7.0).all()) and bool((whole[GUARD + hi:] == 7.0).all()), (off, gated)
            assert bool(((y[lo:hi].double() - value[lo:hi]).abs() <= bound[lo:hi]).all()), (off, gated)
            assert first is None or torch.equal(first, y)
            first = y


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("form", FORMS)
def test_offsets_that_descend(uw, form, kernel):
    """An offset below an earlier one counts as that one: no slot has two experts, none is left out."""
    (per, n), e, k = KERNELS[kernel], 4, 64
    g = torch.Generator().manual_seed(per)
    sets, vals = zip(*[make_set(uw, form, weights(g, e, n, k)) for _ in range(2)])
    x = torch.randn(9, k, generator=g).bfloat16()
    s = e * per
    rows = torch.randint(0, 9, (s,), generator=g, dtype=torch.int32)
    for off in ([0, per, 2 * per, 3 * per, s], [0, 2 * per, per, 2 * per, s], [0, s, 0, s, 0], [2, 1, 5 * per, 0, per],
                [-9, per, 1 << 30, 2, s], [3, 1, 0, -1, -2], [(1 << 31) - 1, 0, 0, 0, s],
                [-(1 << 31), (1 << 31) - 1, 0, 0, 0]):
        check_plan_products(uw, sets, vals, off, x, rows, n, k)


@pytest.mark.parametrize("per,n", [(3, 33), (45, 260)])
@pytest.mark.parametrize("form", ["bf16", "mx4"])
def test_offsets_that_descend_among_many_experts(uw, form, per, n):
    """The same where the search takes several rounds of 256 experts."""
    e, k = 700, 64
    g = torch.Generator().manual_seed(per)
    sets, vals = zip(*[make_set(uw, form, weights(g, e, n, k)) for _ in range(2)])
    x = torch.randn(9, k, generator=g).bfloat16()
    rows = torch.randint(0, 9, (e * per,), generator=g, dtype=torch.int32)
    up = torch.sort(torch.randint(0, e * per + 1, (e + 1,), generator=g)).values
    for at in ([255, 256, 257], [3, 4, 255, 300, 511, 512, 513, 699, 700], list(range(250, 530)), [256, 512], [1, 700]):
        off = up.clone()
        off[at] = torch.randint(-5, e * per, (len(at),), generator=g) // 2
        check_plan_products(uw, sets, vals, off.tolist(), x, rows, n, k)


@pytest.mark.parametrize("per,n", [(300, 33), (50, 33000), (150, 33000), (300, 33000)])
@pytest.mark.parametrize("form", FORMS)
def test_gates_over_the_whole_range(uw, form, per, n):
    """silu(g) u where g and u are single elements of x, so that nothing but the epilogue rounds.

    The exponential's argument g log2(e) (or half of it, counted twice) is off by 2^-24 of itself and by its
    constant's 2^-25 of at most 150, 2^-17.2 of the value together; exponential, sum, reciprocal and the
    products add 2^-23 each: 2^-17 in all.  Subnormal FP32 silu (below g = -91) rounds by 2^-150, and so does its
    product with u; BF16 rounds by half a step, 2^-8 of the value or 2^-134.
    """
    k = 64
    pick = torch.zeros(2, 1, n, k)
    pick[0, 0, :, 0] = pick[1, 0, :, 1] = 1.0
    gate, up = (make_set(uw, form, w)[0] for w in pick)
    g = torch.cat([torch.linspace(-104.0, -80.0, per // 2), torch.linspace(-80.0, 90.0, per - per // 2 - 12),
                   torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e-40, -1e-40, 1e30, -1e30, 3e38, -3e38, -110.0, -1000.0])])
    x = torch.zeros(per, k)
    x[:, 0] = g[torch.randperm(per, generator=torch.Generator().manual_seed(1))]
    off = torch.tensor([0, per], dtype=torch.int32, device=DEV)
    for u in (1.0, -3.5, 1e-3):
        x[:, 1] = u
        b = x.bfloat16()
        h = torch.empty(per, n, dtype=torch.bfloat16, device=DEV)
        uw.uw_matmul_experts_gated(gate, up, off, None, b.to(DEV), h)
        assert bool((h == h[:, :1]).all())
        gv, uv = b[:, 0].double(), b[:, 1].double()
        want = gv * torch.sigmoid(gv) * uv
        tol = (2.0 ** -8 + 2.0 ** -17) * want.abs() + 2.0 ** -149 * (uv.abs() + 1) + 2.0 ** -134
        big = want.abs() > torch.finfo(torch.bfloat16).max
        got = h[:, 0].double().cpu()
        assert bool((((got - want).abs() <= tol) | (big & torch.isinf(got))).all())
