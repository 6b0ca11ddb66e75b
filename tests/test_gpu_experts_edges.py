"""Products grouped by expert where their inputs are odd, in each of the kernels: plans that do not ascend,
gates over the whole range of BF16, row indices outside x, infinities and NaN, strided stacks, palettes of
both kinds, extreme MXFP4 scales, x past 2 GiB, the longest rows and columns.

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


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("form", FORMS)
def test_row_indices_outside_x_are_zeros(uw, form, kernel):
    (per, n), e, k = KERNELS[kernel], 4, 192 if form == "uwf1" else 160
    g = torch.Generator().manual_seed(per + 1)
    sets, vals = zip(*[make_set(uw, form, weights(g, e, n, k)) for _ in range(2)])
    x = torch.randn(9, k, generator=g).bfloat16()
    s = e * per
    rows = torch.randint(0, 9, (s,), generator=g, dtype=torch.int32)
    off = torch.tensor([0, per, 2 * per, 3 * per, s], dtype=torch.int32)
    bad = torch.randperm(s, generator=g)[:max(4, s // 5)]
    given = rows.clone()
    given[bad] = torch.tensor([-1, 9, 10, (1 << 31) - 1, -(1 << 31), 1 << 30], dtype=torch.int32).repeat(s)[:len(bad)]
    ref, mag = grouped_dev(off, rows, x, vals[0])
    up, up_mag = grouped_dev(off, rows, x, vals[1])
    for t in (ref, mag, up, up_mag):
        t[bad] = 0
    want, tol = h_ref(ref, mag, up, up_mag, k)
    dev = off.to(DEV), given.to(DEV), x.to(DEV)
    whole, y = guarded(s, n, torch.float32)
    uw.uw_matmul_experts(sets[0], *dev, y)
    assert bool(((y.double() - ref).abs() <= k * 2.0 ** -23 * mag).all()) and bool((y[bad] == 0).all())
    assert bool((whole[:GUARD] == 7.0).all()) and bool((whole[GUARD + s:] == 7.0).all())
    whole, h = guarded(s, n, torch.bfloat16)
    uw.uw_matmul_experts_gated(*sets, *dev, h)
    assert bool(((h.double() - want).abs() <= tol).all()) and bool((h[bad] == 0).all())
    assert bool((whole[:GUARD] == 7.0).all()) and bool((whole[GUARD + s:] == 7.0).all())


@pytest.mark.parametrize("kernel", list(KERNELS))
@pytest.mark.parametrize("form", FORMS)
def test_infinities_and_nan_reach_their_rows_only(uw, form, kernel):
    """In a K tail too, and in x rows that several slots share."""
    (per, n), e, k = KERNELS[kernel], 4, 192 if form == "uwf1" else 160
    g = torch.Generator().manual_seed(per + 2)
    gate, up = (make_set(uw, form, weights(g, e, n, k))[0] for _ in range(2))
    x = torch.randn(9, k, generator=g).bfloat16()
    s = e * per
    rows = torch.randint(0, 9, (s,), generator=g, dtype=torch.int32)
    off = torch.tensor([0, per, 2 * per, 3 * per, s], dtype=torch.int32, device=DEV)
    out = []
    for bad in (False, True):
        if bad:
            x[1, 0], x[2, k - 1], x[3, 70] = float("inf"), float("nan"), float("-inf")
        y, h = torch.empty(s, n, device=DEV), torch.empty(s, n, dtype=torch.bfloat16, device=DEV)
        uw.uw_matmul_experts(gate, off, rows.to(DEV), x.to(DEV), y)
        uw.uw_matmul_experts_gated(gate, up, off, rows.to(DEV), x.to(DEV), h)
        out.append((y, h))
    clean = ((rows < 1) | (rows > 3)).to(DEV)
    (y, h), (y2, h2) = out
    assert torch.equal(y[clean], y2[clean]) and torch.equal(h[clean], h2[clean])
    nan = (rows == 2).to(DEV)
    assert bool(torch.isnan(y2[nan]).all()) and bool(torch.isnan(h2[nan]).all())
    inf = ((rows == 1) | (rows == 3)).to(DEV)
    assert not bool(torch.isfinite(y2[inf]).any())


@pytest.mark.parametrize("kernel", list(KERNELS))
def test_strided_stacks_in_every_kernel(uw, kernel):
    """Gate and up interleaved in one array, [E][2][n][k], BF16 and MXFP4."""
    (per, n), e, k = KERNELS[kernel], 4, 96
    g = torch.Generator().manual_seed(per + 3)
    w = weights(g, 2 * e, n, k).bfloat16().view(e, 2, n, k)
    d = w.to(DEV)
    el = torch.empty(2 * e, n, k // 2, dtype=torch.uint8, device=DEV)
    sc = torch.empty(2 * e, n, 4, dtype=torch.uint8, device=DEV)
    back = torch.empty(2 * e * n, k, dtype=torch.bfloat16, device=DEV)
    uw.uw_quantize_mx4(d.view(-1, k), el.view(-1, k // 2), sc.view(-1, 4))
    uw.uw_dequantize_mx4(el.view(-1, k // 2), sc.view(-1, 4), back)
    el, sc = el.view(e, 2, n, k // 2), sc.view(e, 2, n, 4)
    s = e * per
    off = torch.tensor([0, per + 1, per + 1, 3 * per, s], dtype=torch.int32)
    x = torch.randn(17, k, generator=g).bfloat16()
    rows = torch.randint(0, 17, (s,), generator=g, dtype=torch.int32)
    dev = off.to(DEV), rows.to(DEV), x.to(DEV)
    for make, v in ((lambda i: uw.uw_experts_bf16(d[:, i], e, n, k, 2 * n * k), w),
                    (lambda i: uw.uw_experts_mx4(el[:, i], sc[:, i], e, n, k, n * k, 2 * n * 4), back.view(e, 2, n, k).cpu())):
        gate, up = make(0), make(1)
        gv, uv = grouped_dev(off, rows, x, v[:, 0].double()), grouped_dev(off, rows, x, v[:, 1].double())
        y, h = torch.empty(s, n, device=DEV), torch.empty(s, n, dtype=torch.bfloat16, device=DEV)
        uw.uw_matmul_experts(up, *dev, y)
        assert bool(((y.double() - uv[0]).abs() <= k * 2.0 ** -23 * uv[1]).all())
        uw.uw_matmul_experts_gated(gate, up, *dev, h)
        want, tol = h_ref(*gv, *uv, k)
        assert bool(((h.double() - want).abs() <= tol).all())


def two_bands(g, e, n, k):
    """Magnitudes of two kinds, 2^40 apart: their exponents are no run."""
    w = weights(g, e, n, k)
    return torch.where(torch.rand(w.shape, generator=g) < 0.5, w, w * 2.0 ** -40)


@pytest.mark.parametrize("kernel", list(KERNELS))
def test_palettes_of_both_kinds_in_every_kernel(uw, kernel):
    """K an odd number of groups, so that rows straddle flag words; verbatim groups; gate and up of different kinds."""
    (per, n), e = KERNELS[kernel], 2
    g = torch.Generator().manual_seed(per + 4)
    for k in (64, 320):
        plain, odd = weights(g, e, n, k), torch.cat([weights(g, 1, n, k, outliers=True), two_bands(g, 1, n, k)])
        (a, av), (b, bv) = make_set(uw, "uwf1", plain), make_set(uw, "uwf1", odd)
        s = e * per
        off = torch.tensor([0, s // 2 - 1, s], dtype=torch.int32)
        x = torch.randn(11, k, generator=g).bfloat16()
        rows = torch.randint(0, 11, (s,), generator=g, dtype=torch.int32)
        dev = off.to(DEV), rows.to(DEV), x.to(DEV)
        ra, rb = grouped_dev(off, rows, x, av), grouped_dev(off, rows, x, bv)
        for h, (ref, mag) in ((a, ra), (b, rb)):
            y = torch.empty(s, n, device=DEV)
            uw.uw_matmul_experts(h, *dev, y)
            assert bool(((y.double() - ref).abs() <= k * 2.0 ** -23 * mag).all())
        for gate, up, rg, ru in ((a, b, ra, rb), (b, a, rb, ra)):
            h = torch.empty(s, n, dtype=torch.bfloat16, device=DEV)
            uw.uw_matmul_experts_gated(gate, up, *dev, h)
            want, tol = h_ref(*rg, *ru, k)
            assert bool(((h.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("kernel", list(KERNELS))
def test_extreme_mx4_scales_in_every_kernel(uw, kernel):
    """Subnormal and large weights count in full; a NaN scale makes its row's outputs NaN and no other's, in a K tail too."""
    (per, n), e, k = KERNELS[kernel], 4, 160
    g = torch.Generator().manual_seed(per + 5)
    s = e * per
    off = torch.tensor([0, per, 2 * per, 3 * per, s], dtype=torch.int32)
    rows = torch.randint(0, 5, (s,), generator=g, dtype=torch.int32)
    elem = torch.randint(0, 256, (e * n, k // 2), dtype=torch.uint8, generator=g)
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
    code = torch.stack([elem & 15, elem >> 4], 2).view(e, n, k).long()
    val = grid[code & 7] * torch.where(code > 7, -1.0, 1.0)
    for byte in (0, 1, 127, 250):
        scale = torch.full((e * n, 8), byte, dtype=torch.uint8)
        scale[:, 5:] = 255                       # padding is never used
        h = uw.uw_experts_mx4(elem.to(DEV), scale.to(DEV), e, n, k)
        x = torch.ldexp(torch.randint(-3, 4, (5, k), generator=g).float(), torch.tensor(min(127 - byte, 120))).bfloat16()
        ref, mag = grouped_dev(off, rows, x, torch.ldexp(val, torch.tensor(byte - 127)))
        y = torch.empty(s, n, device=DEV)
        uw.uw_matmul_experts(h, off.to(DEV), rows.to(DEV), x.to(DEV), y)
        assert bool(((y.double() - ref).abs() <= k * 2.0 ** -23 * mag).all()), byte
    scale = torch.full((e * n, 8), 120, dtype=torch.uint8)
    bad = torch.zeros(e, n, dtype=torch.bool)
    for i, (ex, row) in enumerate(((0, 5), (1, 0), (3, n - 1), (2, n // 2))):
        scale[ex * n + row, (0, 4, 3, 1)[i]] = 255
        bad[ex, row] = True
    h = uw.uw_experts_mx4(elem.to(DEV), scale.to(DEV), e, n, k)
    x = torch.randn(5, k, generator=g).bfloat16()
    x[0] = 0.0
    y, hh = torch.empty(s, n, device=DEV), torch.empty(s, n, dtype=torch.bfloat16, device=DEV)
    uw.uw_matmul_experts(h, off.to(DEV), rows.to(DEV), x.to(DEV), y)
    uw.uw_matmul_experts_gated(h, h, off.to(DEV), rows.to(DEV), x.to(DEV), hh)
    want = bad.repeat_interleave(per, 0).to(DEV)
    assert torch.equal(torch.isnan(y), want) and torch.equal(torch.isnan(hh), want)


@pytest.mark.parametrize("form", FORMS + ["two bands"])
@pytest.mark.parametrize("per", [2, 300])
def test_x_past_two_gib_gated(uw, form, per):
    """Rows whose bytes pass 2^31 and 2^32, and row indices outside x, through both products."""
    g = torch.Generator().manual_seed(per)
    n, k, x_rows = 40, 8192, 270000            # 4.4 GB
    make = (lambda: make_set(uw, "uwf1", two_bands(g, 2, n, k))) if form == "two bands" else (
        lambda: make_set(uw, form, weights(g, 2, n, k)))
    sets, vals = zip(*[make() for _ in range(2)])
    s = 2 * per + 1
    off = torch.tensor([0, per, s], dtype=torch.int32)
    rows = torch.randint(0, x_rows, (s,), generator=g, dtype=torch.int32)
    rows[0], rows[1], rows[-1] = x_rows - 1, 131072, 0
    part = torch.randn(x_rows // 1000, k, generator=g).bfloat16()
    x = torch.empty(x_rows // 1000, 1000, k, dtype=torch.bfloat16, device=DEV)
    x.copy_(part.view(-1, 1, k).to(DEV))       # row r holds part[r // 1000]
    x = x.view(x_rows, k)
    (gv, ga), (uv, ua) = (grouped_ref(off, rows // 1000, part, v) for v in vals)
    given = rows.clone()
    given[2], given[3] = x_rows, -1
    for t in (gv, ga, uv, ua):
        t[2:4] = 0
    y, h = torch.empty(s, n, device=DEV), torch.empty(s, n, dtype=torch.bfloat16, device=DEV)
    uw.uw_matmul_experts(sets[0], off.to(DEV), given.to(DEV), x, y)
    assert bool(((y.double().cpu() - gv).abs() <= k * 2.0 ** -23 * ga).all())
    uw.uw_matmul_experts_gated(*sets, off.to(DEV), given.to(DEV), x, h)
    want, tol = h_ref(gv, ga, uv, ua, k)
    assert bool(((h.double().cpu() - want).abs() <= tol).all())


def small_integers(seed, *size):
    """-3 .. 3 without 0, on the device."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    v = torch.randint(1, 4, size, generator=g, device=DEV, dtype=torch.int8)
    return v * (1 - 2 * torch.randint(0, 2, size, generator=g, device=DEV, dtype=torch.int8))


# Sums of whole numbers below 2^24 are exact in FP32, in any order: one k too few or too many shows.
@pytest.mark.parametrize("per,n,k", [(1, 40, 1 << 20), (3, 40, 28672), (20, 40, 28608), (50, 16500, 8256), (150, 16500, 8192),
                                     (300, 16500, 8256), (3, 1 << 20, 64), (40, 1 << 20, 64)])
@pytest.mark.parametrize("form", FORMS)
def test_long_rows_and_columns_exactly(uw, form, per, n, k):
    w = small_integers(n + k, 2, n, k)
    if form == "uwf1":
        ms = []
        for i in range(2):
            m = uw.uw_compress(w[i].bfloat16(), n, k)
            uw.uw_transcode_palette(m, None)
            ms.append(m)
        h = uw.uw_experts_uwf1(ms)
    elif form == "bf16":
        h = uw.uw_experts_bf16(w.bfloat16(), 2, n, k)
    else:
        el = torch.empty(2, n, k // 2, dtype=torch.uint8, device=DEV)
        sc = torch.empty(2, n, uw.mx4_scale_stride(k), dtype=torch.uint8, device=DEV)
        for i in range(2):                                       # (a call takes 2^20 rows; exact)
            uw.uw_quantize_mx4(w[i].bfloat16(), el[i], sc[i])
        h = uw.uw_experts_mx4(el, sc, 2, n, k)
    x = torch.where(small_integers(per, per + 1, k) > 0, 1.0, -1.0)
    off = torch.tensor([0, per, 2 * per], dtype=torch.int32, device=DEV)
    rows = torch.arange(2 * per, dtype=torch.int32, device=DEV) % (per + 1)
    y = torch.empty(2 * per, n, device=DEV)
    uw.uw_matmul_experts(h, off, rows, x.bfloat16(), y)
    for e in range(2):
        for c in range(0, n, 1 << 16):
            want = x[rows[e * per:(e + 1) * per].long()].double() @ w[e, c:c + (1 << 16)].double().T.contiguous()
            assert torch.equal(y[e * per:(e + 1) * per, c:c + (1 << 16)].double(), want)
