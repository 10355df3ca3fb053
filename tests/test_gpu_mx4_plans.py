"""Each kernel and plan that the product's rules choose (152 SMs), on sizes that take it.

As in test_gpu_mx4.py, scales of 1/2, 1 and 2 make every partial sum a multiple of 1/16; the
sums of these sizes stay below 2^20 (asserted), so any order of summation is exact."""
import numpy as np
import pytest
import torch

from test_gpu_mx4 import random_stored, sg  # noqa: F401  (sg: fixture)

pytestmark = pytest.mark.gpu


def exact(va, vb):
    """A . B^T in 64 bits, and proof that fp32 sums in any order have the same bits."""
    a, b = torch.from_numpy(va).cuda(), torch.from_numpy(vb).cuda()
    assert float((a.abs() @ b.abs().t()).max()) < 2.0 ** 20
    return a @ b.t()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,N,K", [(2100, 1900, 9000), (8192, 520, 4096), (1100, 4200, 1500)])
def test_pairs_hand_over_whole_stages(sg, M, N, K, fmt):  # noqa: F811
    """Products of many stages and of several tiles a pair, many times over: a stage that is
    multiplied before it has arrived in both of the pair's CTAs would leave the sums of
    the stage before it."""
    a, va = random_stored(sg, M, K, fmt, 5 * M + K, True)
    b, vb = random_stored(sg, N, K, fmt, 7 * N + K, True)
    want = exact(va, vb).float()
    for _ in range(40):
        assert torch.equal(sg.mx4_matmul(a, b), want)
