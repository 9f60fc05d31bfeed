"""The plans of rdg_linear on the host: what workspaces they ask for, and that the GPU tests take each."""
import ctypes
import itertools
import random

import pytest


def _rdg():
    import routing_dispatch_grouped_amd as rdg
    return rdg


DTYPES = [0, 1, 2, 3]   # RDG_F32, RDG_BF16, RDG_FP8_E4M3, RDG_FP8_E4M3_UE8M0
TOKENS = sorted({1, 2, 7, 8, 15, 16, 17, 24, 31, 32, 33, 48, 63, 64, 65, 96, 100, 128, 129, 160, 161, 200, 255, 256, 257, 300, 384, 500, 512,
                 513, 700, 900, 1000, 1023, 1024, 1025, 1216, 1500, 2000, 2048, 2049, 2300, 3000, 4001, 4096, 5000, 8191, 8192, 10000,
                 16384, 30000, 65536, 1 << 20, (1 << 31) - 1})
SIZES = list(itertools.product([16, 48, 256, 272, 784, 1040, 2064, 4112, 7168, 9216, 18432, 31312],
                               [128, 384, 640, 1152, 2048, 3968, 7168, 8192, 14336, 18432]))


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_workspace_for_the_most_tokens_does_for_fewer(dtype):
    """The size for a number of tokens is no bound for smaller ones; rdg_linear_workspace_bound is, and grows with the tokens."""
    rdg = _rdg()
    falls = 0
    for N, K in SIZES:
        most = bound = 0
        for T in TOKENS:
            need, last = rdg.rdg_linear_workspace_bytes(T, N, K, dtype), bound
            bound = rdg.rdg_linear_workspace_bound(T, N, K, dtype)
            falls += need < most
            most = max(most, need)
            assert max(most, last) <= bound <= 256 << 20, (T, N, K)
            assert bound <= 64 * T * N
    assert falls > 0


def test_bound_of_what_no_call_takes():
    rdg = _rdg()
    bound = rdg.rdg_linear_workspace_bound
    assert bound(0, 256, 256, rdg.RDG_BF16) == 0 and bound(-1, 256, 7168, rdg.RDG_BF16) == 0
    assert bound(8, 250, 256, rdg.RDG_BF16) == 0 and bound(8, 256, 100, rdg.RDG_BF16) == 0 and bound(8, 256, 256, 4) == 0
    assert bound(8, 256, 128, rdg.RDG_BF16) == 0                      # one block of the reduction: nothing to split


@pytest.mark.parametrize("dtype", DTYPES)
def test_small_products_over_long_reductions_have_splits(dtype):
    """Where the work has to be shared along the reduction a workspace is asked for, and a smaller one refused."""
    rdg = _rdg()
    a = 0x100000   # a stand-in address: the call fails its checks first
    for T, N, K in ((64, 256, 7168), (128, 256, 16384), (37, 528, 7168)):
        need = rdg.rdg_linear_workspace_bytes(T, N, K, dtype)
        assert 0 < need <= 256 << 20 and need % (T * N * 4) == 0
        for work, size in ((a, need - 1), (None, need), (a + 8, need), (a, 0)):
            assert rdg._lib.rdg_linear(a, a, dtype, K, T, N, K, a, a, None, 0, None, 0, 2 * a, rdg.RDG_F32, N, work, size, None) == \
                rdg.RDG_EINVAL


KERNELS = ["rows", "256 x 256", "128 x 128", "128 x 64", "64 x 32", "96 x 64", "80 x 64", "64 x 64"]   # features x tokens
TILE_TOKENS = [16, 256, 128, 64, 32, 64, 64, 64]


def _forms(T, N, K, dtype):
    """The forms of the kernels that a call takes: which part, kernel, splits, and whether its weights pass the caches (one tile of tokens
    of at most 64)."""
    parts = (ctypes.c_int * 6)()
    _rdg()._lib.rdg_linear_plan_of(T, N, K, dtype, parts)
    return {(i, KERNELS[k], splits, k >= 3 and T <= TILE_TOKENS[k])
            for i, (k, splits, features) in enumerate((parts[:3], parts[3:])) if features}


@pytest.mark.parametrize("kind,dtype", [("f32", 0), ("bf16", 1), ("fp8", 2), ("fp8", 3)])
def test_the_gpu_tests_take_every_form_that_a_plan_gives(kind, dtype):
    from test_gpu_joins import LARGE, SHAPES
    from test_gpu_joins_edges import PLANS
    tested = set().union(*(_forms(*size, dtype) for size in SHAPES + LARGE + PLANS[kind]))
    assert {"rows", "128 x 128", "128 x 64", "64 x 32"} <= {f[1] for f in tested}
    rng = random.Random(3)
    for _ in range(40000):
        T, N, K = int(2 ** rng.uniform(0, 13)), 16 * int(2 ** rng.uniform(0, 11)), 128 * int(2 ** rng.uniform(0, 7.1))
        if T * N * K < 1.5e12:
            assert _forms(T, N, K, dtype) <= tested, (T, N, K)
