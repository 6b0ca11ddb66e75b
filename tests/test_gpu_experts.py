"""Routing, products grouped by expert and the whole layer on the GPU against
plain 64-bit implementations.

Tolerances, derived:
  * a product's K terms are exact in FP32 and each addition is off by at most
    2^-23 relative: e = K 2^-23 sum |x w|;
  * h = silu(g) u: |silu'| <= 1.1, so 1.1 e_g (|u| + e_u) + (|silu(g)| + 1.1 e_g) e_u,
    2^-18 |h| for the FP32 exponential, quotient and product (2^-22 relative each
    at |g| < 16; exp(-g) inherits the rounding of its argument), and BF16's half
    step 2^-8 |h|;
  * the layer: the down product's own e plus sum |h error| |d|, weighted and
    summed (2^-21 relative for the weights and the sum), and 2^-8 |out|.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FORMS = ["bf16", "mx4", "uwf1"]


@pytest.fixture(scope="module")
def uw():
    from decode_gemm_exp_amd import uw as _uw
    return _uw


# ------------------------------------------------------------- routing -----

def route_ref(logits, topk, scoring, bias=None):
    l = logits.double().numpy()
    t, n = l.shape
    key = l if bias is None else (logits.float() + bias).double().numpy()
    live = ~np.isnan(key) & (key != -np.inf)
    ids = np.full((t, topk), -1, np.int32)
    w = np.zeros((t, topk))

    def softmax(v):
        m = v.max()
        e = np.ones_like(v)      # equal to the largest, an infinity too
        e[v != m] = np.exp(v[v != m] - m)
        return e / e.sum()

    for i in range(t):
        order = sorted(np.flatnonzero(live[i]), key=lambda e: (-key[i, e], e))[:topk]
        c = len(order)
        if not c:
            continue
        ids[i, :c] = order
        if scoring == "softmax":
            every = np.flatnonzero(live[i])
            p = dict(zip(every, softmax(l[i, every])))
            w[i, :c] = [p[e] for e in order]
        elif scoring == "softmax_topk":
            w[i, :c] = softmax(l[i, order])
        else:
            v = l[i, order]
            w[i, :c] = softmax(np.minimum(v, 0) - np.log1p(np.exp(-np.abs(v))))
    return ids, w


def plan_ref(ids, experts):
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < experts)
    order = [p for _, p in sorted((int(flat[p]), p) for p in np.flatnonzero(ok))]
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[ok], minlength=experts))])
    slots = np.full(flat.size, -1, np.int32)
    slots[order] = np.arange(len(order))
    return offsets.astype(np.int32), np.array([p // ids.shape[1] for p in order], np.int32), slots.reshape(ids.shape)


def check_plan(r, ids, experts):
    off, rows, slots = plan_ref(ids, experts)
    assert np.array_equal(r.offsets.cpu().numpy(), off)
    got = r.rows.cpu().numpy()
    assert np.array_equal(got[:off[-1]], rows)
    assert (got[off[-1]:] == -7).all(), "rows behind the last pair were written"
    assert np.array_equal(r.slots.cpu().numpy(), slots)


def check_route(uw, logits, topk, scoring, bias=None, ld=None):
    t, n = logits.shape
    r = uw.Routing(t, n, topk, DEV)
    r.rows.fill_(-7)
    dev = logits.to(DEV)
    if ld:
        wide = torch.full((t, ld), float("nan"), dtype=logits.dtype, device=DEV)
        wide[:, :n] = dev
        dev = wide[:, :n]
    uw.uw_route_experts(dev, r, scoring, bias.to(DEV) if bias is not None else None)
    ids, w = route_ref(logits, topk, scoring, bias)
    assert np.array_equal(r.ids.cpu().numpy(), ids)
    got = r.weights.cpu().double().numpy()
    # exp, log1p and the sums of at most 1024 terms in FP32; a log sigmoid keeps |l| 2^-24 absolute
    big = np.abs(logits.double().numpy())
    big = big[np.isfinite(big)].max(initial=0)
    assert np.allclose(got, w, rtol=2.0 ** -16 + 2 * big * 2.0 ** -23, atol=1e-37)
    check_plan(r, ids, n)


@pytest.mark.parametrize("tokens,experts,topk", [(1, 1, 1), (1, 64, 4), (3, 4, 4), (65, 8, 2), (64, 16, 16), (257, 60, 1),
                                                 (300, 128, 8), (513, 129, 6), (90, 256, 8), (70, 257, 3),
                                                 (1100, 1024, 16), (5000, 33, 5)])
@pytest.mark.parametrize("scoring", ["softmax", "softmax_topk", "sigmoid"])
def test_route(uw, tokens, experts, topk, scoring):
    g = torch.Generator().manual_seed(tokens + experts)
    l = torch.randn(tokens, experts, generator=g) * 2
    check_route(uw, l, topk, scoring)
    check_route(uw, l.bfloat16(), topk, scoring, ld=experts + 3)      # BF16: many ties


@pytest.mark.parametrize("scoring", ["softmax", "softmax_topk", "sigmoid"])
@pytest.mark.parametrize("tokens", [40, 2000])
def test_route_masks_and_specials(uw, scoring, tokens):
    g = torch.Generator().manual_seed(1)
    l = torch.randn(tokens, 24, generator=g)
    l[torch.rand(tokens, 24, generator=g) < 0.3] = float("-inf")
    l[1] = float("-inf")                    # nothing left
    l[2] = float("nan")
    l[3, :] = 0.5                           # all equal
    l[4, :23] = float("-inf")               # fewer than topk
    l[5, 7] = float("nan")
    l[6, 3] = l[6, 9] = float("inf")        # share the weight
    l[7] = -300.0                           # far below what exp holds
    l[8] = torch.finfo(torch.float32).min   # a mask of the type's lowest value is a score like any other
    l[9, ::2], l[9, 1::2] = 0.0, -0.0       # equal
    l[10] = 1e-42                           # subnormal and equal
    l[11] = 80.0 * torch.randn(24, generator=g)
    check_route(uw, l, 6, scoring)
    bias = torch.randn(24, generator=g)
    bias[5] = float("-inf")                 # never chosen
    bias[6] = 100.0                         # always, where it can be
    l[6, 3] = l[6, 9] = 0.0
    check_route(uw, l, 6, scoring, bias)


@pytest.mark.parametrize("tokens,experts,topk", [(1, 3, 1), (30, 8, 4), (1024, 40, 1), (3000, 7, 3), (700, 1024, 16)])
def test_plan_of_given_ids(uw, tokens, experts, topk):
    g = torch.Generator().manual_seed(tokens)
    ids = torch.randint(-1, experts + 1, (tokens, topk), generator=g, dtype=torch.int32)   # -1 and E: none
    ids[0] = 0                                            # one expert several times
    ids[-1] = torch.iinfo(torch.int32).min
    r = uw.Routing(tokens, experts, topk, DEV)
    r.rows.fill_(-7)
    uw.uw_plan_experts(ids.to(DEV), r)
    check_plan(r, np.where((ids >= 0) & (ids < experts), ids, -1), experts)


def test_route_of_no_tokens(uw):
    r = uw.Routing(0, 8, 2, DEV)
    r.offsets.fill_(5)
    uw.uw_route_experts(torch.empty(0, 8, device=DEV), r)
    assert r.offsets.cpu().tolist() == [0] * 9


# ------------------------------------------------------------ products -----

def make_set(uw, form, w):
    """w [E][n][k] float32 -> (handle, the float64 values it stands for)."""
    e, n, k = w.shape
    b = w.bfloat16()
    if form == "bf16":
        return uw.uw_experts_bf16(b.to(DEV), e, n, k), b.double()
    if form == "mx4":
        el = torch.empty(e * n, k // 2, dtype=torch.uint8, device=DEV)
        sc = torch.empty(e * n, uw.mx4_scale_stride(k), dtype=torch.uint8, device=DEV)
        out = torch.empty(e * n, k, dtype=torch.bfloat16, device=DEV)
        uw.uw_quantize_mx4(b.view(-1, k).to(DEV), el, sc)
        uw.uw_dequantize_mx4(el, sc, out)      # pinned against the definition in test_gpu_mx4
        return uw.uw_experts_mx4(el, sc, e, n, k), out.view(e, n, k).double().cpu()
    ms = []
    for i in range(e):
        m = uw.uw_compress(b[i].contiguous().to(DEV), n, k)
        uw.uw_transcode_palette(m, None)
        if i % 2:
            uw.uw_drop_stream(m)               # not needed
        ms.append(m)
    return uw.uw_experts_uwf1(ms), b.double()


def weights(g, e, n, k, outliers=False):
    w = torch.randn(e, n, k, generator=g) * 0.05
    if outliers:                               # exponents outside the palette: verbatim groups
        at = torch.rand(w.shape, generator=g) < 0.004
        w = torch.where(at, w * 2.0 ** torch.randint(-60, 30, w.shape, generator=g).float(), w)
    return w


def ragged(g, counts, x_rows):
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32)
    return off, torch.randint(0, x_rows, (int(off[-1]),), generator=g, dtype=torch.int32)


def grouped_ref(off, rows, x, w):
    """(values, magnitudes) of the plain grouped product in 64 bits."""
    y = torch.zeros(len(rows), w.shape[1], dtype=torch.float64)
    a = torch.zeros_like(y)
    for e in range(w.shape[0]):
        s = slice(int(off[e]), int(off[e + 1]))
        xe = x[rows[s].long()].double()
        y[s], a[s] = xe @ w[e].T, xe.abs() @ w[e].abs().T
    return y, a


def h_ref(g, ag, u, au, k):
    """silu(g) u and its tolerance."""
    eg, eu = k * 2.0 ** -23 * ag, k * 2.0 ** -23 * au
    sg = g * torch.sigmoid(g)
    h = sg * u
    return h, 1.1 * eg * (u.abs() + eu) + (sg.abs() + 1.1 * eg) * eu + (2.0 ** -18 + 2.0 ** -8) * h.abs() + 1e-38


COUNTS = [([1], 1), ([0, 1, 0], 1), ([2, 0, 0, 5, 1], 3), ([16, 17, 15, 0], 20), ([0] * 7, 4), ([70, 0, 3, 33], 50),
          ([130, 1, 260, 0, 64], 200), ([1] * 37, 9), ([0] * 300 + [3] + [0] * 20 + [2, 1], 4)]


@pytest.mark.parametrize("counts,x_rows", COUNTS)
@pytest.mark.parametrize("form", FORMS)
def test_grouped_product(uw, form, counts, x_rows):
    g = torch.Generator().manual_seed(len(counts) + x_rows)
    e, (n, k) = len(counts), (37, 192) if form == "uwf1" else (37, 160)
    h, wv = make_set(uw, form, weights(g, e, n, k, outliers=form == "uwf1"))
    h2, uv = make_set(uw, form, weights(g, e, n, k))
    x = torch.randn(x_rows, k, generator=g).bfloat16()
    off, rows = ragged(g, counts, x_rows)
    pad = 5
    rows_p = torch.cat([rows, torch.full((pad,), 1 << 30, dtype=torch.int32)])
    y = torch.full((len(rows) + pad, n), 7.0, device=DEV)
    uw.uw_matmul_experts(h, off.to(DEV), rows_p.to(DEV), x.to(DEV), y)
    ref, mag = grouped_ref(off, rows, x, wv)
    got = y.double().cpu()
    assert bool((got[len(rows):] == 7.0).all()), "rows behind the last slot were written"
    assert bool(((got[:len(rows)] - ref).abs() <= k * 2.0 ** -23 * mag).all())
    hh = torch.full((len(rows) + pad, n), 7.0, dtype=torch.bfloat16, device=DEV)
    uw.uw_matmul_experts_gated(h2, h, off.to(DEV), rows_p.to(DEV), x.to(DEV), hh)
    gv, ga = grouped_ref(off, rows, x, uv)
    want, tol = h_ref(gv, ga, ref, mag, k)
    got = hh.double().cpu()
    assert bool((got[len(rows):] == 7.0).all())
    assert bool(((got[:len(rows)] - want).abs() <= tol).all())


@pytest.mark.parametrize("n,k", [(1, 64), (16, 64), (48, 128), (260, 512), (1000, 1088)])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("per", [1, 24, 150])
def test_grouped_product_shapes(uw, form, n, k, per):
    g = torch.Generator().manual_seed(n + k)
    counts = [per, 0, 2 * per + 1]
    h, wv = make_set(uw, form, weights(g, 3, n, k, outliers=True) if form == "uwf1" else weights(g, 3, n, k))
    off, _ = ragged(g, counts, 1)
    s = int(off[-1])
    x = torch.randn(s, k, generator=g).bfloat16()
    y = torch.empty(s, n, device=DEV)
    uw.uw_matmul_experts(h, off.to(DEV), None, x.to(DEV), y)      # slot s is row s
    ref, mag = grouped_ref(off, torch.arange(s), x, wv)
    assert bool(((y.double().cpu() - ref).abs() <= k * 2.0 ** -23 * mag).all())
    hh = torch.empty(s, n, dtype=torch.bfloat16, device=DEV)
    uw.uw_matmul_experts_gated(h, h, off.to(DEV), None, x.to(DEV), hh)
    want, tol = h_ref(ref, mag, ref, mag, k)
    assert bool(((hh.double().cpu() - want).abs() <= tol).all())


def test_uwf1_rows_cross_flag_words(uw):
    """K an odd number of groups: a row's groups straddle flag words; palettes of both kinds in one set."""
    g = torch.Generator().manual_seed(4)
    for k, outliers in ((320, (False, True, False)), (1984, (True, True, True)), (2112, (False, False, False))):
        w = torch.cat([weights(g, 1, 50, k, o) for o in outliers])
        h, wv = make_set(uw, "uwf1", w)
        for per in (3, 140):
            off, rows = ragged(g, [per] * 3, 11)
            x = torch.randn(11, k, generator=g).bfloat16()
            y = torch.empty(3 * per, 50, device=DEV)
            uw.uw_matmul_experts(h, off.to(DEV), rows.to(DEV), x.to(DEV), y)
            ref, mag = grouped_ref(off, rows, x, wv)
            assert bool(((y.double().cpu() - ref).abs() <= k * 2.0 ** -23 * mag).all())


def test_strided_stacks(uw):
    """Gate and up interleaved in one array, [E][2][n][k], read in place."""
    g = torch.Generator().manual_seed(6)
    e, n, k = 5, 40, 96
    w = weights(g, 2 * e, n, k).bfloat16().view(e, 2, n, k)
    d = w.to(DEV)
    gate = uw.uw_experts_bf16(d, e, n, k, 2 * n * k)
    up = uw.uw_experts_bf16(d[:, 1], e, n, k, 2 * n * k)
    el = torch.empty(2 * e * n, k // 2, dtype=torch.uint8, device=DEV)
    sc = torch.empty(2 * e * n, 4, dtype=torch.uint8, device=DEV)
    uw.uw_quantize_mx4(d.view(-1, k), el, sc)
    back = torch.empty(2 * e * n, k, dtype=torch.bfloat16, device=DEV)
    uw.uw_dequantize_mx4(el, sc, back)
    v4 = back.view(e, 2, n, k).cpu()
    gate4 = uw.uw_experts_mx4(el, sc, e, n, k, n * k, 2 * n * 4)
    up4 = uw.uw_experts_mx4(el[n:], sc[n:], e, n, k, n * k, 2 * n * 4)
    with pytest.raises(ValueError):
        uw.uw_experts_bf16(d[:, 1], e + 1, n, k, 2 * n * k)       # past the storage
    for counts in ([3, 0, 1, 20, 2], [90, 0, 100, 200, 1]):
        off, rows = ragged(g, counts, 17)
        x = torch.randn(17, k, generator=g).bfloat16()
        for a, b, v in ((gate, up, w), (gate4, up4, v4)):
            h = torch.empty(len(rows), n, dtype=torch.bfloat16, device=DEV)
            uw.uw_matmul_experts_gated(a, b, off.to(DEV), rows.to(DEV), x.to(DEV), h)
            want, tol = h_ref(*grouped_ref(off, rows, x, v[:, 0].double()), *grouped_ref(off, rows, x, v[:, 1].double()), k)
            assert bool(((h.double().cpu() - want).abs() <= tol).all())


@pytest.mark.parametrize("per", [3, 140])
@pytest.mark.parametrize("form", FORMS)
def test_bad_plans_stay_inside(uw, form, per):
    """Row indices outside x select zeros; descending, negative and too large offsets are clamped."""
    g = torch.Generator().manual_seed(8)
    k, n, e = 128, 33, 4
    h, wv = make_set(uw, form, weights(g, e, n, k))
    x = torch.randn(6, k, generator=g).bfloat16()
    off, rows = ragged(g, [per] * e, 6)
    rows[1], rows[per + 1] = -1, 6
    y = torch.full((e * per, n), 7.0, device=DEV)
    uw.uw_matmul_experts(h, off.to(DEV), rows.to(DEV), x.to(DEV), y)
    clean = rows.clone()
    clean[1] = clean[per + 1] = 0
    ref, mag = grouped_ref(off, clean, x, wv)
    ref[1] = ref[per + 1] = 0
    mag[1] = mag[per + 1] = 0
    assert bool(((y.double().cpu() - ref).abs() <= k * 2.0 ** -23 * mag).all())
    for bad in ([0, 5 * per, 2, 1, 3], [-9, per, 1 << 30, 2, 4 * per], [3, 1, 0, -1, -2],
                [-(1 << 31), (1 << 31) - 1, 0, 0, 0]):
        y.fill_(7.0)
        uw.uw_matmul_experts(h, torch.tensor(bad, dtype=torch.int32, device=DEV), rows.to(DEV), x.to(DEV), y)
        torch.cuda.synchronize()


@pytest.mark.parametrize("per", [2, 140])
@pytest.mark.parametrize("form", FORMS)
def test_not_finite_rows_stay_alone(uw, form, per):
    """Infinities and NaN in one row of x, in a K tail too, reach no other slot."""
    g = torch.Generator().manual_seed(12)
    k, n = (192, 40) if form == "uwf1" else (160, 40)
    h, _ = make_set(uw, form, weights(g, 2, n, k))
    x = torch.randn(2 * per, k, generator=g).bfloat16()
    off = torch.tensor([0, per, 2 * per], dtype=torch.int32, device=DEV)
    out = []
    for bad in (False, True):
        if bad:
            x[0, 0] = float("inf")
            x[1, k - 1] = float("nan")
        y = torch.empty(2 * per, n, device=DEV)
        uw.uw_matmul_experts(h, off, None, x.to(DEV), y)
        out.append(y.cpu())
    assert torch.equal(out[0][2:], out[1][2:])
    assert torch.isnan(out[1][1]).all() and not torch.isfinite(out[1][0]).any()


def test_gated_extremes(uw):
    """Gates far below zero give zero, far above give gate times up; no NaN from the exponential."""
    k, n = 32, 16
    w = torch.zeros(1, n, k)
    w[0, :, 0] = 1.0
    u = torch.zeros(1, n, k)
    u[0, :, 1] = 1.0
    gate, up = make_set(uw, "bf16", w)[0], make_set(uw, "bf16", u)[0]
    gv = torch.tensor([-1e30, -200.0, -88.0, -20.0, 0.0, 20.0, 200.0, 1e30])
    x = torch.zeros(8, k)
    x[:, 0], x[:, 1] = gv, 2.0
    h = torch.empty(8, n, dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, 8], dtype=torch.int32, device=DEV)
    uw.uw_matmul_experts_gated(gate, up, off, None, x.bfloat16().to(DEV), h)
    b = x.bfloat16().double()[:, 0]
    want = 2.0 * b * torch.sigmoid(b)
    assert torch.allclose(h[:, 0].double().cpu(), want, rtol=2.0 ** -8 + 2.0 ** -16, atol=1e-30)


def test_sets_that_do_not_fit_are_refused(uw):
    g = torch.Generator().manual_seed(2)
    a, _ = make_set(uw, "bf16", weights(g, 2, 64, 64))
    b, _ = make_set(uw, "mx4", weights(g, 2, 64, 64))
    c, _ = make_set(uw, "bf16", weights(g, 3, 64, 64))
    off = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    x = torch.randn(2, 64, device=DEV).bfloat16()
    h = torch.empty(2, 64, dtype=torch.bfloat16, device=DEV)
    for other, status in ((b, -2), (c, -1)):
        with pytest.raises(uw.UwError) as err:
            uw.uw_matmul_experts_gated(a, other, off, None, x, h)
        assert err.value.status == status
    m = uw.uw_compress(torch.randn(64, 64, device=DEV).bfloat16(), 64, 64)
    with pytest.raises(uw.UwError) as err:
        uw.uw_experts_uwf1([m])                       # no resident indices
    assert err.value.status == -6
    uw.uw_transcode_palette(m, None)
    s = uw.uw_experts_uwf1([m])
    y = torch.empty(1, 64, device=DEV)
    one = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    uw.uw_matmul_experts(s, one, None, x[:1], y)
    torch.cuda.synchronize()
    uw.uw_drop_palette(m)
    with pytest.raises(uw.UwError) as err:
        uw.uw_matmul_experts(s, one, None, x[:1], y)
    assert err.value.status == -6
    kn = uw.uw_compress(torch.randn(64, 64, device=DEV).bfloat16(), 64, 64, uw.LAYOUT_KN)
    uw.uw_transcode_palette(kn, None)
    f8 = uw.uw_compress_fp8(torch.randint(0, 255, (64, 64), dtype=torch.uint8, device=DEV), 64, 64)
    for bad in (kn, f8):
        with pytest.raises(uw.UwError) as err:
            uw.uw_experts_uwf1([bad])
        assert err.value.status == -2


# Enough blocks for the LDS tiles of 64, 128 and 256 rows (and, of MXFP4 and UWF1, the
# register-fed kernel's two groups of slots): counts around `per`, none for some
# experts, a K tail, partly filled tiles of rows and of columns.
@pytest.mark.parametrize("experts,per,n,k", [(40, 20, 1290, 192), (300, 20, 260, 64), (30, 150, 1100, 192),
                                             (13, 300, 2500, 64), (4, 1100, 2564, 320), (12, 400, 2052, 1088)])
@pytest.mark.parametrize("form", FORMS)
def test_many_rows(uw, form, experts, per, n, k):
    g = torch.Generator().manual_seed(experts + per)
    counts = torch.randint(per // 2, per + per // 2, (experts,), generator=g).tolist()
    counts[experts // 2] = 0
    counts[1] = 1
    h, wv = make_set(uw, form, weights(g, experts, n, k, outliers=form == "uwf1"))
    h2, uv = make_set(uw, form, weights(g, experts, n, k))
    x_rows = 500
    x = torch.randn(x_rows, k, generator=g).bfloat16()
    off, rows = ragged(g, counts, x_rows)
    s, pad = len(rows), 70                     # capacity beyond the last slot
    rows_p = torch.cat([rows, torch.full((pad,), 1 << 30, dtype=torch.int32)])
    dev = [t.to(DEV) for t in (off, rows_p, x)]
    y = torch.full((s + pad, n), 7.0, device=DEV)
    uw.uw_matmul_experts(h, *dev, y)
    assert bool((y[s:] == 7.0).all()), "rows behind the last slot were written"
    hh = torch.full((s + pad, n), 7.0, dtype=torch.bfloat16, device=DEV)
    uw.uw_matmul_experts_gated(h2, h, *dev, hh)
    assert bool((hh[s:] == 7.0).all())
    for e in range(experts):                   # FP64 on the device, one expert at a time
        sl = slice(int(off[e]), int(off[e + 1]))
        xe = x[rows[sl].long()].double().to(DEV)
        we, ue = wv[e].to(DEV), uv[e].to(DEV)
        ref, mag = xe @ we.T.contiguous(), xe.abs() @ we.abs().T.contiguous()
        assert bool(((y[sl].double() - ref).abs() <= k * 2.0 ** -23 * mag).all()), f"expert {e}"
        gv, ga = xe @ ue.T.contiguous(), xe.abs() @ ue.abs().T.contiguous()
        want, tol = h_ref(gv, ga, ref, mag, k)
        assert bool(((hh[sl].double() - want).abs() <= tol).all()), f"gated, expert {e}"


@pytest.mark.parametrize("form", ["bf16", "mx4"])
@pytest.mark.parametrize("per", [2, 300])
def test_x_past_two_gib(uw, form, per):
    """Row indices whose bytes pass 2^31 and 2^32."""
    g = torch.Generator().manual_seed(per)
    n, k, x_rows = 40, 8192, 270000            # 4.4 GB
    h, wv = make_set(uw, form, weights(g, 2, n, k))
    x = torch.zeros(x_rows, k, dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, per, 2 * per + 1], dtype=torch.int32)
    rows = torch.randint(0, x_rows, (2 * per + 1,), generator=g, dtype=torch.int32)
    rows[0], rows[1], rows[-1] = x_rows - 1, 131072, 0
    part = torch.randn(x_rows // 1000, k, generator=g).bfloat16()
    x.view(x_rows // 1000, 1000, k).copy_(part.view(-1, 1, k).to(DEV))   # row r holds part[r // 1000]
    y = torch.empty(2 * per + 1, n, device=DEV)
    uw.uw_matmul_experts(h, off.to(DEV), rows.to(DEV), x, y)
    ref, mag = grouped_ref(off, rows // 1000, part, wv)
    assert bool(((y.double().cpu() - ref).abs() <= k * 2.0 ** -23 * mag).all())


# ------------------------------------------------------------ the layer -----

def layer_ref(r_ids, r_w, experts, x, gv, uv, dv, topk):
    off, rows, slots = plan_ref(r_ids, experts)
    rows = torch.from_numpy(rows)
    n, k = gv.shape[1:]
    hv, ht = h_ref(*grouped_ref(off, rows, x, gv), *grouped_ref(off, rows, x, uv), k)
    d = torch.zeros(len(rows), k, dtype=torch.float64)
    dt = torch.zeros_like(d)
    for e in range(experts):
        s = slice(off[e], off[e + 1])
        d[s] = hv[s] @ dv[e].T
        dt[s] = (ht[s] + n * 2.0 ** -23 * (hv[s].abs() + ht[s])) @ dv[e].abs().T
    out = torch.zeros(len(x), k, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for t in range(len(x)):
        for j in range(topk):
            if slots[t, j] >= 0:
                w = float(r_w[t, j])
                out[t] += w * d[slots[t, j]]
                tol[t] += w * (dt[slots[t, j]] + (2.0 ** -16) * d[slots[t, j]].abs())
    return out, tol + 2.0 ** -8 * (out.abs() + tol)


@pytest.mark.parametrize("form", FORMS + ["mixed"])
@pytest.mark.parametrize("tokens,experts,topk,n,k", [(1, 4, 2, 64, 128), (9, 8, 3, 128, 192), (70, 5, 2, 192, 64),
                                                     (400, 6, 4, 64, 320)])
def test_layer(uw, form, tokens, experts, topk, n, k):
    g = torch.Generator().manual_seed(tokens)
    gf, df = ("bf16", "mx4") if form == "mixed" else (form, form)
    gate, gv = make_set(uw, gf, weights(g, experts, n, k))
    up, uv = make_set(uw, gf, weights(g, experts, n, k, outliers=False))
    down, dv = make_set(uw, df, weights(g, experts, k, n))
    l = torch.randn(tokens, experts, generator=g)
    if tokens > 4:
        l[2:4] = float("-inf")                 # padded tokens
        l[4, 1:] = float("-inf")               # one expert left
    x = torch.randn(tokens, k, generator=g).bfloat16()
    r = uw.Routing(tokens, experts, topk, DEV)
    uw.uw_route_experts(l.to(DEV), r)
    out = torch.full((tokens, k), float("nan"), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(uw.uw_workspace_size_expert_mlp(gate, down, tokens, topk), dtype=torch.uint8, device=DEV)
    ws.fill_(255)                              # NaN wherever nothing is written
    uw.uw_expert_mlp(gate, up, down, r, x.to(DEV), out, ws)
    ids, w = route_ref(l, topk, "softmax_topk")
    ref, tol = layer_ref(ids, w, experts, x, gv, uv, dv, topk)
    got = out.double().cpu()
    assert bool(((got - ref).abs() <= tol).all())
    if tokens > 4:
        assert bool((got[2:4] == 0).all())


@pytest.mark.parametrize("tokens", [6, 600])
def test_layer_captured(uw, tokens):
    """Route and layer in one graph, replayed with other tokens and other routings, eager work between."""
    g = torch.Generator().manual_seed(3)
    experts, topk, n, k = 6, 2, 96, 160
    sets = [make_set(uw, "bf16", weights(g, experts, *s))[0] for s in ((n, k), (n, k), (k, n))]
    l, x = torch.zeros(tokens, experts, device=DEV), torch.zeros(tokens, k, dtype=torch.bfloat16, device=DEV)
    r = uw.Routing(tokens, experts, topk, DEV)
    out = torch.empty(tokens, k, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(uw.uw_workspace_size_expert_mlp(sets[0], sets[2], tokens, topk), dtype=torch.uint8, device=DEV)

    def step():
        uw.uw_route_experts(l, r)
        uw.uw_expert_mlp(*sets, r, x, out, ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    seen = []
    for i in range(4):
        l.copy_(torch.randn(tokens, experts, generator=g))
        x.copy_(torch.randn(tokens, k, generator=g))
        if i == 2:
            l[:, 1:] = float("-inf")           # every token to one expert
        graph.replay()
        torch.cuda.synchronize()
        replayed = out.clone()
        out.fill_(0)
        step()
        torch.cuda.synchronize()
        assert torch.equal(replayed, out)
        seen.append(replayed)
    assert not torch.equal(seen[0], seen[1])


def test_two_graphs_share_a_workspace(uw):
    """Two captured layers of different sizes with one workspace, replayed in turn on one stream."""
    g = torch.Generator().manual_seed(17)
    experts, topk, n, k = 5, 2, 96, 160
    sets = [make_set(uw, "mx4", weights(g, experts, *s))[0] for s in ((n, k), (n, k), (k, n))]
    nb = uw.uw_workspace_size_expert_mlp(sets[0], sets[2], 500, topk)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)
    jobs = []
    for tokens in (3, 500):
        l, x = torch.randn(tokens, experts, generator=g).to(DEV), torch.randn(tokens, k, generator=g).bfloat16().to(DEV)
        r, out = uw.Routing(tokens, experts, topk, DEV), torch.empty(tokens, k, dtype=torch.bfloat16, device=DEV)

        def step(l=l, x=x, r=r, out=out):
            uw.uw_route_experts(l, r)
            uw.uw_expert_mlp(*sets, r, x, out, ws)

        step()
        torch.cuda.synchronize()
        want = out.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        jobs.append((graph, out, want, step))  # (step holds what the graph reads)
    for _ in range(3):
        for graph, out, _, _ in jobs:
            out.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for _, out, want, _ in jobs:
            assert torch.equal(out, want)


def test_two_streams_at_once(uw):
    """The layer on two streams with their own workspaces gives what it gives alone."""
    g = torch.Generator().manual_seed(5)
    tokens, experts, topk, n, k = 300, 8, 2, 128, 256
    sets = [make_set(uw, "mx4", weights(g, experts, *s))[0] for s in ((n, k), (n, k), (k, n))]
    nb = uw.uw_workspace_size_expert_mlp(sets[0], sets[2], tokens, topk)
    jobs = []
    for _ in range(2):
        jobs.append((torch.randn(tokens, experts, generator=g).to(DEV), torch.randn(tokens, k, generator=g).bfloat16().to(DEV),
                     uw.Routing(tokens, experts, topk, DEV), torch.empty(tokens, k, dtype=torch.bfloat16, device=DEV),
                     torch.empty(nb, dtype=torch.uint8, device=DEV), torch.cuda.Stream()))
    alone = []
    for l, x, r, out, ws, _ in jobs:
        uw.uw_route_experts(l, r)
        uw.uw_expert_mlp(*sets, r, x, out, ws)
        torch.cuda.synchronize()
        alone.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for l, x, r, out, ws, s in jobs:
            with torch.cuda.stream(s):
                uw.uw_route_experts(l, r)
                uw.uw_expert_mlp(*sets, r, x, out, ws)
    torch.cuda.synchronize()
    for (_, _, _, out, _, _), a in zip(jobs, alone):
        assert torch.equal(out, a)


def test_layer_matches_the_single_matrix_product(uw):
    """One expert, every token to it: the grouped product of a UWF1 set is the matrix's own product."""
    g = torch.Generator().manual_seed(7)
    n, k = 320, 256
    w = weights(g, 1, n, k, outliers=True).bfloat16()
    m = uw.uw_compress(w[0].to(DEV), n, k)
    uw.uw_transcode_palette(m, None)
    s = uw.uw_experts_uwf1([m])
    for batch in (1, 20, 150):
        x = torch.randn(batch, k, generator=g).bfloat16().to(DEV)
        off = torch.tensor([0, batch], dtype=torch.int32, device=DEV)
        y, z = torch.empty(batch, n, device=DEV), torch.empty(batch, n, device=DEV)
        uw.uw_matmul_experts(s, off, None, x, y)
        ws = torch.empty(max(16, uw.uw_workspace_size(m, 3, batch)), dtype=torch.uint8, device=DEV)
        uw.uw_matmul_reconstruct(m, uw.PIPE_PALETTE_DIRECT, x, z, ws)
        mag = x.double().abs() @ w[0].double().abs().T.to(DEV)
        assert bool(((y - z).abs().double() <= 2 * k * 2.0 ** -23 * mag).all())
