"""The feed-forward products' choice of tile and parts, on the host."""
import ctypes

import pytest

from test_gpu_gated_ff import MANY, SHAPES

NONE, FULL, EIGHT = 0, 1, 2
FORWARD, INPUT, WEIGHTS = 0, 1, 2


def choice(lib, M, N, K, keep, product):
    columns, parts = ctypes.c_int(), ctypes.c_int()
    st = lib.sgemm_gated_ff_choose_check(M, N, K, keep, product, ctypes.byref(columns),
                                         ctypes.byref(parts))
    return (columns.value, parts.value) if st == 0 else st


def test_choices_fit(lib):
    """Few tokens have their own kernel unless blocks of 64 have to be whole, parts keep eight
    stages, and the workspace holds every part's sums."""
    need = ctypes.c_size_t()
    sizes = (1, 16, 17, 100, 257, 1000, 4096, 16384)
    for M in sizes:
        for N in sizes:
            for K in sizes:
                for keep in (NONE, FULL, EIGHT):
                    columns, parts = choice(lib, M, N, K, keep, FORWARD)
                    assert parts == 1
                    assert columns == 256 if keep == EIGHT else (columns == 0) == (M <= 16)
                sums = 0
                for product, stages, result in ((INPUT, 2 * -(-N // 64), M * -(-K // 64) * 64),
                                                (WEIGHTS, -(-M // 64), 2 * N * -(-K // 64) * 64)):
                    columns, parts = choice(lib, M, N, K, FULL, product)
                    assert columns in (128, 256) and 1 <= parts <= 16
                    assert parts == 1 or stages // parts >= 8
                    sums += parts * 4 * result if parts > 1 else 0
                assert lib.sgemm_gated_ff_workspace(M, N, K, 1, 0, ctypes.byref(need)) == 0
                assert need.value == 4 * M * -(-N // 64) * 64 + sums


def test_every_kind_is_run_by_the_gpu_tests(lib):
    """The shapes of the GPU tests take every kernel, with and without parts."""
    kinds = {FORWARD: set(), INPUT: set(), WEIGHTS: set()}
    for s in SHAPES + MANY:
        kinds[FORWARD] |= {choice(lib, *s, k, FORWARD)[0] for k in (NONE, EIGHT)}
        for product in (INPUT, WEIGHTS):
            columns, parts = choice(lib, *s, FULL, product)
            kinds[product].add((columns, parts > 1))
    assert kinds[FORWARD] == {0, 128, 160, 224, 256}
    assert kinds[INPUT] == kinds[WEIGHTS] == {(c, p) for c in (128, 256) for p in (False, True)}


@pytest.mark.parametrize("args", [(0, 8, 8, 0, 0), (8, 0, 8, 0, 0), (8, 8, 0, 0, 0), (8, 8, 8, 3, 0),
                                  (8, 8, 8, 0, 3), (8, 8, 8, 0, -1), (-1, 8, 8, 0, 0)])
def test_refusals(lib, args):
    assert choice(lib, *args) == -1
    n = ctypes.c_int()
    assert lib.sgemm_gated_ff_choose_check(8, 8, 8, 0, 0, None, ctypes.byref(n)) == -1
    assert choice(lib, 2**30 + 1, 8, 8, 0, 0) == -4
