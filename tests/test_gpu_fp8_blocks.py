"""FP8 with a scale per block of 128: conversion, products and grouped products on the
GPU against plain 64-bit implementations.

Tolerances, derived:
  * conversion: scales, elements and BF16 values are equal, by the definition's own
    FP32 steps;
  * a product: elements' products are exact in FP32.  A block's sum of up to 128 of
    them is off by at most 2^-23 relative per addition, its scaling by two roundings
    (the scales' product, the fused multiply-add), and the blocks' sums are added
    one by one, those of the waves (eight at most) after them:
    min(k, 128) + k / 128 + 10 <= k + 16 steps of 2^-23 of sum |s_x s_w xe we|;
  * the gated form as in tests/test_gpu_experts.py, with these products.
"""
import numpy as np
import pytest
import torch

from tests.test_gpu_experts import grouped_ref, h_ref, ragged, weights

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# the finite E4M3 magnitudes, by code
GRID = np.array([m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127])
MIDS = (GRID[1:] + GRID[:-1]) / 2


@pytest.fixture(scope="module")
def uw():
    from decode_gemm_exp_amd import uw as _uw
    return _uw


def quantize_ref(x: np.ndarray, block_rows: int):
    """codes [rows][cols], scales, by the definition; x float64 holding FP32 numbers."""
    rows, cols = x.shape
    nr, nc = -(-rows // block_rows), -(-cols // 128)
    code, scale = np.zeros(x.shape, np.uint8), np.zeros((nr, nc), np.float32)
    for i in range(nr):
        for j in range(nc):
            b = x[i * block_rows:(i + 1) * block_rows, 128 * j:128 * j + 128]
            if not np.isfinite(b).all():
                scale[i, j] = np.nan
                continue
            m = np.float32(max(np.abs(b).max(), 2.0 ** -110))
            scale[i, j] = m / np.float32(448)
            q = b.astype(np.float32) * (np.float32(448) / m)          # FP32 arithmetic
            a = np.abs(q).astype(np.float64)
            lo = np.searchsorted(MIDS, a, side="left")                # a tie: the code below it
            tie = (lo < 126) & (a == MIDS[np.minimum(lo, 125)])
            c = np.where(tie & (lo % 2 == 1), lo + 1, lo)
            code[i * block_rows:(i + 1) * block_rows, 128 * j:128 * j + 128] = c + 128 * np.signbit(q)
    return code, scale


def code_values(code):
    return np.where(code & 127 == 127, np.nan, GRID[np.minimum(code & 127, 126)]) * np.where(code & 128, -1.0, 1.0)


def expand(scale, shape, block_rows):
    return np.repeat(np.repeat(scale.astype(np.float64), block_rows, 0), 128, 1)[:shape[0], :shape[1]]


def quantize(uw, x, block_rows, dtype=torch.float8_e4m3fn):
    elem = torch.full(x.shape, 0xAA, dtype=torch.uint8, device=DEV).view(dtype)
    scale = torch.full(uw.fp8_scale_shape(*x.shape, block_rows), 7.0, device=DEV)
    uw.uw_quantize_fp8(x, elem, scale, block_rows)
    return elem, scale


def check_quantize(uw, x, block_rows):
    elem, scale = quantize(uw, x, block_rows)
    code, want = quantize_ref(x.double().cpu().numpy(), block_rows)
    assert np.array_equal(scale.cpu().numpy(), want, equal_nan=True)
    got = elem.view(torch.uint8).cpu().numpy()
    live = ~np.isnan(expand(want, x.shape, block_rows))
    assert np.array_equal(got[live], code[live]) and not got[~live].any()
    out = torch.empty(x.shape, dtype=torch.bfloat16, device=DEV)
    uw.uw_dequantize_fp8(elem, scale, out, block_rows)
    with np.errstate(over="ignore", invalid="ignore"):
        v = code_values(got).astype(np.float32) * expand(want, x.shape, block_rows).astype(np.float32)
    back = torch.from_numpy(v).bfloat16()
    o = out.cpu()
    assert torch.equal(o.isnan(), back.isnan()) and torch.equal(o.nan_to_num(), back.nan_to_num())


SHAPES = [(1, 32), (3, 64), (7, 96), (128, 128), (129, 160), (5, 4128), (64, 1024), (33, 224), (1000, 544), (300, 8224)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_shapes(uw, rows, cols, f32, block_rows):
    g = torch.Generator().manual_seed(rows * cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(torch.randint(-20, 20, (rows, 1), generator=g).float())
    check_quantize(uw, (x if f32 else x.bfloat16()).to(DEV), block_rows)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_values(uw, f32, block_rows):
    """Every code and every tie between two codes, at scales of 1 and of other powers of two; zeros, subnormal
    and extreme blocks; infinities and NaN."""
    every = np.concatenate([GRID, MIDS, np.nextafter(np.float32(MIDS), np.float32(0)) if f32 else MIDS])
    every = np.concatenate([every, -every])
    every = np.concatenate([every, np.zeros(-every.size % 127)]).reshape(-1, 127)
    rows = [np.concatenate([r, [448.0]]) * 2.0 ** e for r in every for e in (0, -30, 17)]
    tiny = 2.0 ** -149 if f32 else 2.0 ** -133
    rows += [np.zeros(128), np.full(128, -0.0), np.full(128, tiny), np.full(128, 2.0 ** -110), np.full(128, 2.0 ** -109),
             np.full(128, 2.0 ** -120), np.linspace(-3e38, 3e38, 128), np.linspace(-1, 1, 128) * 2.0 ** -126]
    for bad in (np.inf, -np.inf, np.nan):
        rows.append(np.where(np.arange(128) == 77, bad, 1.0))
    x = torch.from_numpy(np.stack(rows)).float()
    x = (x if f32 else x.bfloat16()).to(DEV)
    if block_rows == 1:
        check_quantize(uw, x, 1)
        check_quantize(uw, x.reshape(2, -1) if x.shape[0] % 2 == 0 else x.reshape(1, -1), 1)   # blocks beside each other
    else:
        for r in x:
            check_quantize(uw, r.view(8, 16).repeat(1, 2).contiguous(), 128)


@pytest.mark.parametrize("f32", [False, True])
def test_quantize_strided(uw, f32):
    """Rows further apart than they are long, read and written in place; elements as bytes."""
    g = torch.Generator().manual_seed(5)
    dt = torch.float32 if f32 else torch.bfloat16
    wide = torch.full((40, 264), float("nan"), dtype=dt, device=DEV)
    x = torch.randn(40, 160, generator=g).to(dt).to(DEV)
    wide[:, 8:168] = x
    for br in (1, 128):
        a, sa = quantize(uw, x, br)
        b, sb = quantize(uw, wide[:, 8:168], br, torch.uint8)
        assert torch.equal(a.view(torch.uint8), b) and torch.equal(sa, sb)
        out = torch.full((40, 264), 7.0, dtype=torch.bfloat16, device=DEV)
        uw.uw_dequantize_fp8(b, sb, out[:, 8:168], br)
        flat = torch.empty(40, 160, dtype=torch.bfloat16, device=DEV)
        uw.uw_dequantize_fp8(a, sa, flat, br)
        assert torch.equal(out[:, 8:168], flat)
        assert bool((out[:, :8] == 7).all()) and bool((out[:, 168:] == 7).all())


def test_no_rows(uw):
    for br in (1, 128):
        uw.uw_quantize_fp8(torch.empty(0, 64, device=DEV), torch.empty(0, 64, dtype=torch.uint8, device=DEV),
                           torch.empty(0, 1, device=DEV), br)
        uw.uw_dequantize_fp8(torch.empty(0, 64, dtype=torch.uint8, device=DEV), torch.empty(0, 1, device=DEV),
                             torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), br)
    elem, scale = quantize(uw, torch.ones(32, 64, device=DEV), 128)
    uw.uw_matmul_fp8(elem, scale, torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), torch.empty(0, 32, device=DEV))


# ------------------------------------------------------------- product -----

def values(elem, scale, block_rows):
    """FP64 values of the library's arrays, on the device."""
    v = torch.from_numpy(code_values(np.arange(256))).to(DEV)[elem.view(torch.uint8).long()]
    s = scale.double().repeat_interleave(block_rows, 0)[:elem.shape[0]].repeat_interleave(128, 1)[:, :elem.shape[1]]
    return v * s


def fp8_weights(uw, g, n, k):
    """Scales that differ from block to block, by powers of two and otherwise."""
    w = torch.randn(n, k, generator=g)
    w *= torch.exp2(torch.randint(-3, 4, (1, k), generator=g).float()) * (1 + torch.rand(n, 1, generator=g))
    elem, scale = quantize(uw, w.to(DEV), 128)
    scale *= torch.exp2(torch.randint(-6, 6, scale.shape, generator=g).float()).to(DEV)
    return elem, scale


def product(uw, elem, scale, x, act):
    n, k = elem.shape
    y = torch.full((len(x), n), float("nan"), device=DEV)
    ws = torch.full((uw.uw_workspace_size_fp8(n, k, len(x), act),), 255, dtype=torch.uint8, device=DEV)
    uw.uw_matmul_fp8(elem, scale, x, y, ws, act)
    return y


def check_product(uw, elem, scale, x, act):
    n, k = elem.shape
    y = product(uw, elem, scale, x, act)
    xv = x.double()
    if act == uw.ACT_FP8:
        xv = values(*quantize(uw, x, 1), 1)
    w = values(elem, scale, 128).T.contiguous()
    ref, mag = xv @ w, xv.abs() @ w.abs()
    assert bool(((y.double() - ref).abs() <= (k + 16) * 2.0 ** -23 * mag).all())
    assert torch.equal(y, product(uw, elem, scale, x, act)), "two calls differ"


SIZES = [(1, 1, 32), (1, 16, 64), (2, 37, 160), (1, 300, 1056), (3, 1000, 128), (7, 129, 4128), (16, 260, 288),
         (17, 64, 96), (31, 1001, 1184), (33, 130, 2048), (64, 5001, 544), (65, 256, 256), (100, 2500, 320),
         (128, 4096, 512), (129, 700, 1088), (200, 33, 2080), (256, 1537, 224), (300, 8200, 160), (513, 2052, 416),
         (1025, 4100, 1056)]


@pytest.mark.parametrize("batch,n,k", SIZES)
@pytest.mark.parametrize("act", ["bf16", "fp8"])
def test_product(uw, batch, n, k, act):
    g = torch.Generator().manual_seed(batch + n + k)
    elem, scale = fp8_weights(uw, g, n, k)
    x = (torch.randn(batch, k, generator=g) * torch.exp2(torch.randint(-4, 5, (1, k), generator=g).float())).bfloat16()
    check_product(uw, elem, scale, x.to(DEV), uw.ACT_FP8 if act == "fp8" else uw.ACT_BF16)


@pytest.mark.parametrize("batch", [1, 12, 40, 200, 1000])
@pytest.mark.parametrize("act", ["bf16", "fp8"])
def test_product_of_special_values(uw, batch, act):
    """A NaN element or scale reaches its row of W alone (its block of rows), an infinity or a NaN in x its
    row of y alone, a scale of zero and a block of zeros give zeros."""
    g = torch.Generator().manual_seed(batch)
    n, k = 1300, 544
    a = uw.ACT_FP8 if act == "fp8" else uw.ACT_BF16
    elem, scale = fp8_weights(uw, g, n, k)
    x = torch.randn(batch, k, generator=g).bfloat16().to(DEV)
    clean = product(uw, elem, scale, x, a)
    e2, s2, x2 = elem.clone(), scale.clone(), x.clone()
    e2.view(torch.uint8)[5, k - 1] = 0x7F
    e2.view(torch.uint8)[700, 3] = 0xFF
    s2[3, 4] = float("nan")           # rows 384 .. 511, the block the K tail is in
    s2[1] = 0.0                       # rows 128 .. 255
    x2[batch - 1, k - 1] = float("inf")
    y = product(uw, e2, s2, x2, a)
    if batch > 1:
        x2[0, 0] = float("nan")
        z = product(uw, e2, s2, x2, a)
        assert z[0, 700:].isnan().all() and torch.equal(z[1:].nan_to_num(), y[1:].nan_to_num())
    assert y[:, 5].isnan().all() and y[:, 700].isnan().all() and y[:, 384:512].isnan().all()
    assert not y[batch - 1, 600:].isfinite().any()
    rest = torch.ones(n, dtype=torch.bool, device=DEV)
    rest[5] = rest[700] = False
    rest[384:512] = False
    if batch > 1:
        assert bool((y[:batch - 1, 128:256] == 0).all())
        rest[128:256] = False
        assert torch.equal(y[:batch - 1][:, rest], clean[:batch - 1][:, rest])
    x3 = torch.zeros_like(x)
    assert bool((product(uw, elem, scale, x3, a) == 0).all())


@pytest.mark.parametrize("act", ["bf16", "fp8"])
def test_product_exactly(uw, act):
    """Small whole numbers at scales of one: every sum is exact whatever its order; long rows, many columns."""
    for batch, n, k in [(2, 40, 32768), (300, 3000, 64), (70, 20000, 96), (513, 600, 6400)]:
        g = torch.Generator().manual_seed(n)
        w = torch.randint(-2, 3, (n, k), generator=g).float().to(DEV)
        x = torch.randint(-2, 3, (batch, k), generator=g).float().to(DEV)
        scale = torch.ones(uw.fp8_scale_shape(n, k, 128), device=DEV)
        if act == "fp8":
            x[:, ::128] = 448.0       # x's own scales are one
            w[:, ::128] = 0.0
        y = product(uw, w.to(torch.float8_e4m3fn), scale, x.bfloat16(), uw.ACT_FP8 if act == "fp8" else uw.ACT_BF16)
        assert torch.equal(y, x @ w.T)


def test_product_of_compressed_fp8_weights(uw):
    """Elements that were stored without loss and decoded serve the product."""
    g = torch.Generator().manual_seed(9)
    n, k = 256, 512
    elem, scale = fp8_weights(uw, g, n, k)
    m = uw.uw_compress_fp8(elem.view(torch.uint8), n, k)
    back = torch.empty(n, k, dtype=torch.uint8, device=DEV)
    uw.uw_decode_fp8(m, back)
    assert uw.uw_sync_status(m) == 0 and torch.equal(back, elem.view(torch.uint8))
    for batch in (1, 200):
        x = torch.randn(batch, k, generator=g).bfloat16().to(DEV)
        for a in (uw.ACT_BF16, uw.ACT_FP8):
            assert torch.equal(product(uw, back, scale, x, a), product(uw, elem, scale, x, a))


@pytest.mark.parametrize("batch", [5, 600])
def test_captured_on_two_streams(uw, batch):
    """Conversion and product in two graphs that share a workspace, replayed in turn with other inputs, eager work
    between; and the product on another stream than torch's current one."""
    g = torch.Generator().manual_seed(3)
    n, k = 300, 288
    w, x = torch.zeros(n, k, dtype=torch.bfloat16, device=DEV), torch.zeros(batch, k, dtype=torch.bfloat16, device=DEV)
    elem = torch.empty(n, k, dtype=torch.uint8, device=DEV)
    scale = torch.empty(uw.fp8_scale_shape(n, k, 128), device=DEV)
    ys = [torch.empty(batch - i, n, device=DEV) for i in range(2)]
    ws = torch.empty(max(16, uw.uw_workspace_size_fp8(n, k, batch, uw.ACT_FP8)), dtype=torch.uint8, device=DEV)

    def step(i):
        uw.uw_quantize_fp8(w, elem, scale, 128)
        uw.uw_matmul_fp8(elem, scale, x[i:], ys[i], ws, uw.ACT_FP8)

    step(0), step(1)
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            step(i)
    seen = []
    for _ in range(3):
        w.copy_(torch.randn(n, k, generator=g))
        x.copy_(torch.randn(batch, k, generator=g))
        for i in range(2):
            ys[i].zero_()
            graphs[i].replay()
        torch.cuda.synchronize()
        got = [y.clone() for y in ys]
        for i in range(2):
            ys[i].zero_()
            step(i)
        torch.cuda.synchronize()
        assert torch.equal(got[0], ys[0]) and torch.equal(got[1], ys[1])
        seen.append(got[0])
    assert not torch.equal(seen[0], seen[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other, ws2 = torch.empty_like(ys[0]), torch.empty_like(ws)
    torch.cuda.synchronize()
    uw.uw_matmul_fp8(elem, scale, x, other, ws2, uw.ACT_FP8, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(other, ys[0])


# ------------------------------------------------------------- experts -----

def make_set(uw, w):
    """FP8 set of w [e][n][k] (floats), and the values it stands for in FP64 on the host."""
    e, n, k = w.shape
    elem = torch.empty(e, n, k, dtype=torch.float8_e4m3fn, device=DEV)
    scale = torch.empty(e, *uw.fp8_scale_shape(n, k, 128), device=DEV)
    vals = []
    for i in range(e):
        uw.uw_quantize_fp8(w[i].to(DEV), elem[i], scale[i], 128)
        vals.append(values(elem[i], scale[i], 128).cpu())
    return uw.uw_experts_fp8(elem, scale, e, n, k), torch.stack(vals)


COUNTS = [([1], 1), ([0, 1, 0], 1), ([2, 0, 0, 5, 1], 3), ([16, 17, 15, 0], 20), ([0] * 7, 4), ([70, 0, 3, 33], 50),
          ([130, 1, 260, 0, 64], 200), ([1] * 37, 9), ([0] * 300 + [3] + [0] * 20 + [2, 1], 4), ([600, 1100], 77)]


@pytest.mark.parametrize("counts,x_rows", COUNTS)
@pytest.mark.parametrize("n,k", [(37, 160), (300, 288)])
def test_grouped_product(uw, counts, x_rows, n, k):
    g = torch.Generator().manual_seed(len(counts) + x_rows)
    e = len(counts)
    h, wv = make_set(uw, weights(g, e, n, k))
    h2, uv = make_set(uw, weights(g, e, n, k))
    x = torch.randn(x_rows, k, generator=g).bfloat16()
    off, rows = ragged(g, counts, x_rows)
    pad = 70
    rows_p = torch.cat([rows, torch.full((pad,), 1 << 30, dtype=torch.int32)])
    y = torch.full((len(rows) + pad, n), 7.0, device=DEV)
    uw.uw_matmul_experts(h, off.to(DEV), rows_p.to(DEV), x.to(DEV), y)
    ref, mag = grouped_ref(off, rows, x, wv)
    mag *= (k + 16) / k
    got = y.double().cpu()
    assert bool((got[len(rows):] == 7.0).all()), "rows behind the last slot were written"
    assert bool(((got[:len(rows)] - ref).abs() <= k * 2.0 ** -23 * mag).all())
    hh = torch.full((len(rows) + pad, n), 7.0, dtype=torch.bfloat16, device=DEV)
    uw.uw_matmul_experts_gated(h2, h, off.to(DEV), rows_p.to(DEV), x.to(DEV), hh)
    gv, ga = grouped_ref(off, rows, x, uv)
    want, tol = h_ref(gv, ga * (k + 16) / k, ref, mag, k)
    got = hh.double().cpu()
    assert bool((got[len(rows):] == 7.0).all())
    assert bool(((got[:len(rows)] - want).abs() <= tol).all())


@pytest.mark.parametrize("experts,per,n,k", [(40, 20, 1290, 192), (300, 20, 260, 64), (30, 150, 1100, 192),
                                             (13, 300, 2500, 96), (4, 1100, 2564, 320), (12, 400, 2052, 1088)])
def test_many_rows(uw, experts, per, n, k):
    g = torch.Generator().manual_seed(experts + per)
    counts = torch.randint(per // 2, per + per // 2, (experts,), generator=g).tolist()
    counts[experts // 2] = 0
    counts[1] = 1
    h, wv = make_set(uw, weights(g, experts, n, k))
    h2, uv = make_set(uw, weights(g, experts, n, k))
    x = torch.randn(500, k, generator=g).bfloat16()
    off, rows = ragged(g, counts, 500)
    s, pad = len(rows), 70
    rows_p = torch.cat([rows, torch.full((pad,), 1 << 30, dtype=torch.int32)])
    dev = [t.to(DEV) for t in (off, rows_p, x)]
    y = torch.full((s + pad, n), 7.0, device=DEV)
    uw.uw_matmul_experts(h, *dev, y)
    assert bool((y[s:] == 7.0).all())
    hh = torch.full((s + pad, n), 7.0, dtype=torch.bfloat16, device=DEV)
    uw.uw_matmul_experts_gated(h2, h, *dev, hh)
    assert bool((hh[s:] == 7.0).all())
    for e in range(experts):
        sl = slice(int(off[e]), int(off[e + 1]))
        xe = x[rows[sl].long()].double().to(DEV)
        we, ue = wv[e].to(DEV), uv[e].to(DEV)
        ref, mag = xe @ we.T.contiguous(), xe.abs() @ we.abs().T.contiguous() * ((k + 16) / k)
        assert bool(((y[sl].double() - ref).abs() <= k * 2.0 ** -23 * mag).all()), f"expert {e}"
        gv, ga = xe @ ue.T.contiguous(), xe.abs() @ ue.abs().T.contiguous() * ((k + 16) / k)
        want, tol = h_ref(gv, ga, ref, mag, k)
        assert bool(((hh[sl].double() - want).abs() <= tol).all()), f"gated, expert {e}"


@pytest.mark.parametrize("per", [3, 140, 400])
def test_bad_plans_stay_inside(uw, per):
    """Row indices outside x select zeros; descending, negative and too large offsets are clamped."""
    g = torch.Generator().manual_seed(8)
    k, n, e = 160, 33, 4
    h, wv = make_set(uw, weights(g, e, n, k))
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
    assert bool(((y.double().cpu() - ref).abs() <= (k + 16) * 2.0 ** -23 * mag).all())
    for bad in ([0, 5 * per, 2, 1, 3], [-9, per, 1 << 30, 2, 4 * per], [-(1 << 31), (1 << 31) - 1, 0, 0, 0]):
        uw.uw_matmul_experts(h, torch.tensor(bad, dtype=torch.int32, device=DEV), rows.to(DEV), x.to(DEV), y)
        torch.cuda.synchronize()


def test_strided_stacks(uw):
    """Gate and up in one array, [E][2][n][k] and its scales, read in place."""
    g = torch.Generator().manual_seed(6)
    e, n, k = 5, 130, 160
    elem = torch.empty(e, 2, n, k, dtype=torch.float8_e4m3fn, device=DEV)
    scale = torch.empty(e, 2, 2, 2, device=DEV)
    vals = torch.empty(e, 2, n, k, dtype=torch.float64)
    for i in range(e):
        for j in range(2):
            uw.uw_quantize_fp8(weights(g, 1, n, k)[0].to(DEV), elem[i, j], scale[i, j], 128)
            vals[i, j] = values(elem[i, j], scale[i, j], 128).cpu()
    gate = uw.uw_experts_fp8(elem, scale, e, n, k, 2 * n * k, 8)
    up = uw.uw_experts_fp8(elem[:, 1], scale[:, 1], e, n, k, 2 * n * k, 8)
    with pytest.raises(ValueError):
        uw.uw_experts_fp8(elem[:, 1], scale[:, 1], e + 1, n, k, 2 * n * k, 8)
    with pytest.raises(ValueError):
        uw.uw_experts_fp8(elem, scale[:, 1, :1], e, n, k, 2 * n * k, 8)
    for counts in ([3, 0, 1, 20, 2], [90, 0, 100, 300, 1]):
        off, rows = ragged(g, counts, 17)
        x = torch.randn(17, k, generator=g).bfloat16()
        h = torch.empty(len(rows), n, dtype=torch.bfloat16, device=DEV)
        uw.uw_matmul_experts_gated(gate, up, off.to(DEV), rows.to(DEV), x.to(DEV), h)
        f = (k + 16) / k
        (a, am), (b, bm) = grouped_ref(off, rows, x, vals[:, 0]), grouped_ref(off, rows, x, vals[:, 1])
        want, tol = h_ref(a, am * f, b, bm * f, k)
        assert bool(((h.double().cpu() - want).abs() <= tol).all())
