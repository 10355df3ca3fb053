"""The workspace of the feed-forward block's fp16 gradient, on the host."""
import ctypes

import pytest


def ask(lib, M, N, K, backward, packed):
    n = ctypes.c_size_t(0)
    st = lib.sgemm_gated_ff_workspace(M, N, K, backward, packed, ctypes.byref(n))
    return n.value if st == 0 else st


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (3, 65, 7), (500, 4096, 1024), (2**20, 2**20, 64), (2**30, 2**30, 1)])
def test_size(lib, M, N, K):
    """dg and du twice, and fp32 numbers for each token and each output of dg and of du."""
    up = lambda n: -(-n // 64) * 64
    for packed in range(8):
        more = ask(lib, M, N, K, 1, packed | 8) - ask(lib, M, N, K, 1, packed)
        assert more == 2 * 2 * M * up(N) + 4 * up(M + 2 * N)
    assert ask(lib, 0, N, K, 1, 8) == 0


def test_refusals(lib):
    """It is a matter of the gradient only."""
    for args in ((8, 8, 8, 0, 8), (8, 8, 8, 0, 15), (8, 8, 8, 1, 16), (8, 8, 8, 1, -1)):
        assert ask(lib, *args) == -1
