"""Workspace sizes as batches grow, on the host alone."""
import ctypes
import random

import pytest

SHAPES = [(4096, 14336), (14336, 4096), (5001, 8224), (28672, 8192), (257, 20000), (1, 32), (16987, 192), (2532, 5152),
          (4450, 29920), (5960, 8736)]


@pytest.fixture(scope="module")
def uw():
    from decode_gemm_exp_amd import uw as _uw
    return _uw


def batches(rng):
    return sorted(set(range(1, 300)) | {512, 640, 1000, 1024, 2047, 2048, 2049, 4096, 8192, 20000}
                  | {rng.randint(300, 30000) for _ in range(40)})


@pytest.mark.parametrize("act", ["bf16", "fp8"])
def test_fp8_size_never_falls_with_more_rows(uw, act):
    """A server that sizes once for its largest batch has enough for every smaller one."""
    rng = random.Random(7)
    a = uw.ACT_FP8 if act == "fp8" else uw.ACT_BF16
    for n, k in SHAPES + [(rng.randint(1, 40000), 32 * rng.randint(1, 900)) for _ in range(60)]:
        sizes = [uw.uw_workspace_size_fp8(n, k, b, a) for b in batches(rng)]
        assert sizes == sorted(sizes), (n, k)


@pytest.mark.parametrize("act", ["bf16", "fp8"])
def test_fp8_size_is_bounded(uw, act):
    """None for a few rows; beyond x's elements and scales at most 512 rows of 256 sums for each of 256 CUs."""
    a = uw.ACT_FP8 if act == "fp8" else uw.ACT_BF16
    for n, k in SHAPES:
        assert uw.uw_workspace_size_fp8(n, k, 0, a) == uw.uw_workspace_size_fp8(n, k, 1, a) == 0
        for b in (200, 1024, 20000):
            x = (2 * k + 4 * (-(-k // 128))) * b + 512 if act == "fp8" else 0
            assert uw.uw_workspace_size_fp8(n, k, b, a) <= x + (128 << 20)


def test_mx4_size_never_falls_with_more_rows(uw):
    rng = random.Random(8)
    for n, k in SHAPES:
        for a in (uw.ACT_BF16, uw.ACT_MX4):
            sizes = [uw.uw_workspace_size_mx4(n, k, b, a) for b in batches(rng)]
            assert sizes == sorted(sizes), (n, k)


def test_router_and_layer_sizes_never_fall_with_more_tokens(uw):
    """16385 tokens make fewer, larger blocks than 16384."""
    tokens = list(range(0, 1200, 7)) + list(range(16300, 17000)) + [32768, 32769, 33000, 65536, 65537]
    n = ctypes.c_size_t()
    sets = []
    for n_, k in ((32, 32), (1408, 2048)):
        for shape in ((n_, k), (k, n_)):
            h = ctypes.c_void_p()
            assert uw._lib.uw_experts_bf16(4096, 1024, *shape, 0, ctypes.byref(h)) == 0
            sets.append(h)

    def sizes(f, *args):
        out = []
        for t in tokens:
            assert f(*args[0], t, *args[1], ctypes.byref(n)) == 0
            out.append(n.value)
        return out

    for topk in (1, 3, 16):
        for experts in [e for e in (1, 60, 1024) if e >= topk]:
            got = sizes(uw._lib.uw_workspace_size_route, (), (experts, topk))
            assert got == sorted(got)
        for i in (0, 2):
            for f in (uw._lib.uw_workspace_size_expert_mlp, uw._lib.uw_workspace_size_expert_layer):
                got = sizes(f, (sets[i], sets[i + 1]), (topk,))
                assert got == sorted(got)
    for h in sets:
        uw._lib.uw_free_experts(h)
