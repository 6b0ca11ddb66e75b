"""FP8 products through kernels and splits that a call's sizes choose, exactly.

Whole numbers: elements and x in -2 .. 2 at scales that are powers of two give sums far below 2^24
steps, exact in FP32 whatever their order, so results are equal, not near.  With x in 8 bits a 448 at
the head of each of its blocks, beside a zero weight, makes its scales one.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(scope="module")
def uw():
    from decode_gemm_exp_amd import uw as _uw
    return _uw


def whole_numbers(g, *shape):
    return torch.randint(-2, 3, shape, generator=g).float().to(DEV)


def problem(uw, batch, n, k, act, seed=0):
    """elem, scale, x, activation type and the product."""
    g = torch.Generator().manual_seed(batch + n + k + seed)
    w, x = whole_numbers(g, n, k), whole_numbers(g, batch, k)
    if act == "fp8":
        x[:, ::128] = 448.0
        w[:, ::128] = 0.0
    i, j = (torch.arange(m, device=DEV) for m in uw.fp8_scale_shape(n, k, 128))
    scale = torch.exp2((2.0 * i[:, None] + j) % 5 - 2)   # 1/4 .. 4, every one of a block's neighbours another
    wide = w * scale.repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    return (w.to(torch.float8_e4m3fn), scale, x.bfloat16(), uw.ACT_FP8 if act == "fp8" else uw.ACT_BF16,
            (x.double() @ wide.double().T).float())


def workspace(uw, batch, n, k, a, fill=0xA5):
    return torch.full((uw.uw_workspace_size_fp8(n, k, batch, a) + 256,), fill, dtype=torch.uint8, device=DEV)


def check(uw, batch, n, k, act):
    """The product is exact, twice, whatever the workspace held, and nothing beside y and the workspace is written;
    returns the workspace's bytes afterwards, filled with 0xA5 before."""
    elem, scale, x, a, want = problem(uw, batch, n, k, act)
    y = torch.full((batch + 1, n), 7.0, device=DEV)
    for fill in (0xFF, 0xA5):
        ws = workspace(uw, batch, n, k, a, fill)
        y[:batch] = float("nan")
        uw.uw_matmul_fp8(elem, scale, x, y[:batch], ws[:-256], a)
        assert torch.equal(y[:batch], want)
        assert bool((y[batch] == 7.0).all()) and bool((ws[-256:] == fill).all())
    return ws[:-256]


@pytest.mark.parametrize("batch,n,k", [(300, 300, 20000), (700, 130, 32768), (1100, 520, 16544)])
def test_scales_of_long_rows_of_x(uw, batch, n, k):
    """Tiles whose rows' scales of x lie far apart: with more than 129 blocks a row, offsets of rows behind the last
    block of k pass 2^31."""
    ws = check(uw, batch, n, k, "fp8")
    assert bool((ws != 0xA5).any())   # the tiles' x was laid out there


@pytest.mark.parametrize("n,k,batches", [(4096, 14336, (2048, 1024, 333, 200, 48, 13, 1)),
                                         (14336, 4096, (2048, 640, 129, 100, 96, 5)),
                                         (5960, 8736, (96, 80, 64, 30)), (2532, 5152, (256, 208, 192, 100, 16))])
@pytest.mark.parametrize("act", ["bf16", "fp8"])
def test_workspace_of_the_largest_batch_serves_the_smaller(uw, n, k, batches, act):
    a = uw.ACT_FP8 if act == "fp8" else uw.ACT_BF16
    ws = workspace(uw, batches[0], n, k, a)
    for batch in batches:
        elem, scale, x, _, want = problem(uw, batch, n, k, act)
        y = torch.full((batch, n), float("nan"), device=DEV)
        uw.uw_matmul_fp8(elem, scale, x, y, ws[:-256], a)
        assert torch.equal(y, want), batch
    assert bool((ws[-256:] == 0xA5).all())


# 192 to 255 blocks of 64 rows of the matrix and two groups of sixteen rows of x: the last block and the last group cut off.
@pytest.mark.parametrize("batch,n,k", [(17, 12288, 160), (32, 12229, 1056), (25, 16331, 96), (31, 14337, 2080),
                                       (33, 6145, 288), (64, 7001, 416), (50, 8129, 544), (96, 4100, 224)])
@pytest.mark.parametrize("act", ["bf16", "fp8"])
def test_two_groups_of_rows(uw, batch, n, k, act):
    ws = check(uw, batch, n, k, act)
    assert bool((ws == 0xA5).all())   # the rows kernel uses none


def check_slices(uw, ws, batch, n, k, act, rows, count):
    """`count` slices of tiles of `rows` rows by 256 sums, from the workspace's bytes after x's share, and nothing
    else, were written (each tile's rows up to the batch's last)."""
    at = 0
    if act == "fp8":
        at = sum(-(-b // 256) * 256 for b in (2 * batch * k, 4 * batch * (-(-k // 128))))
        assert bool((ws[:at].view(-1, 256) != 0xA5).any(1).all())
    part = ws[at:]
    wrote = (part[:len(part) // 1024 * 1024].view(-1, 1024) != 0xA5).any(1)
    assert bool(wrote[0:count * rows:rows].all()) and not bool(wrote[count * rows:].any()), "other slices than expected"


# Up to 96 rows blocks start along K at different places, each inside its own slice: 64-row and 128-row tiles, all of
# them in slices or the last round's alone, or none; then more rows, as in tests/test_gpu_fp8_edges.py.  The last two
# numbers: rows of a tile, tiles in slices times slices, on 256 CUs.
TILES = [(57, 4096, 8192, 64, 16 * 13), (33, 4096, 16384, 64, 16 * 13), (65, 4096, 8224, 64, 32 * 8),
         (96, 5001, 8224, 64, 40 * 6), (72, 33838, 5056, 64, 10 * 7), (79, 5931, 18400, 128, 24 * 10),
         (76, 8101, 14144, 128, 32 * 8), (45, 49228, 416, 64, 0), (68, 22654, 2560, 64, 0), (66, 33000, 1024, 128, 0),
         (80, 43410, 1184, 128, 0), (333, 4096, 14336, 128, 48 * 5), (200, 5001, 8224, 128, 40 * 6),
         (2100, 4100, 4096, 128, 33 * 4), (1500, 6400, 2080, 128, 44 * 3), (1100, 300, 9600, 64, 36 * 7),
         (300, 300, 20000, 64, 10 * 16), (640, 14337, 1056, 128, 0)]


@pytest.mark.parametrize("batch,n,k,rows,slices", TILES)
@pytest.mark.parametrize("act", ["bf16", "fp8"])
def test_tiles_and_slices(uw, batch, n, k, rows, slices, act):
    check_slices(uw, check(uw, batch, n, k, act), batch, n, k, act, rows, slices)


@pytest.mark.parametrize("per,n", [(3, 33), (3, 5000), (20, 4160), (140, 33), (400, 33), (400, 2600)])
@pytest.mark.parametrize("gated", [False, True])
def test_plans_that_descend_or_leave_the_rows(uw, per, n, gated):
    """Offsets count as clamped to the slots and to those before them, row indices outside x as rows of zeros;
    slots that no expert has, and what lies behind the last, keep what they held."""
    g = torch.Generator().manual_seed(per + n)
    e, k = 4, 160
    slots = e * per
    w = whole_numbers(g, 2, e, n, k)
    scale = torch.ones(e, *uw.fp8_scale_shape(n, k, 128), device=DEV)
    gate, up = (uw.uw_experts_fp8(v.to(torch.float8_e4m3fn), scale, e, n, k) for v in w)
    x = whole_numbers(g, 6, k)
    rows = torch.randint(0, 6, (slots,), generator=g, dtype=torch.int32)
    rows[1], rows[per + 1], rows[-1] = -1, 6, -(1 << 31)
    xs = x[rows.clamp(0, 5).long()] * ((rows >= 0) & (rows < 6)).to(DEV)[:, None]
    for off in ([per * i for i in range(e + 1)], [0, 3 * per, 2, 1, 3], [-9, per, 1 << 30, 2, slots],
                [-(1 << 31), (1 << 31) - 1, 0, 0, 0], [2, 1, per, per, slots - 1], [slots + 5] * 5, [0] * 5):
        at, bounds = 0, []
        for o in off:
            at = max(at, min(max(o, 0), slots))
            bounds.append(at)
        want = torch.full((slots + 3, n), 7.0, device=DEV)
        for i in range(e):
            s = slice(bounds[i], bounds[i + 1])
            a = xs[s] @ w[0][i].T
            if gated:   # (whole numbers: the sums are exact; silu, the product and BF16's rounding are not)
                b = xs[s] @ w[1][i].T
                a = (a.double() * torch.sigmoid(a.double()) * b.double()).float()
            want[s] = a
        got = torch.full((slots + 3, n), 7.0, device=DEV, dtype=torch.bfloat16 if gated else torch.float32)
        dev = torch.tensor(off, dtype=torch.int32, device=DEV), rows.to(DEV), x.bfloat16()
        if gated:
            uw.uw_matmul_experts_gated(gate, up, *dev, got[:slots])
            # the exponential of up to 150 and what follows it 2^-17 (tests/test_gpu_experts_edges.py, gates over the
            # whole range), BF16 2^-8, and one more FP32 step of `want`; 1e-38 covers subnormals
            near = (got.float() - want).abs() <= (2.0 ** -8 + 2.0 ** -17 + 2.0 ** -23) * want.abs() + 1e-38
            assert bool(near.all()), off
            kept = torch.ones(slots + 3, dtype=torch.bool, device=DEV)
            kept[bounds[0]:bounds[-1]] = False
            assert bool((got[kept] == 7.0).all()), off
        else:
            uw.uw_matmul_experts(gate, *dev, got[:slots])
            assert torch.equal(got, want), off
