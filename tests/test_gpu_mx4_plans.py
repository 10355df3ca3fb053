"""Each kernel and plan that the product's rules choose (152 SMs), on sizes that take it.

As in test_gpu_mx4.py, scales of 1/2, 1 and 2 make every partial sum a multiple of 1/16; the
sums of these sizes stay below 2^20 (asserted), so any order of summation is exact."""
import ctypes

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


# (M, N, K): (rows of A a tile, parts of its K range)
PLANS = [((3, 2500, 700), (16, 1)), ((16, 700, 2300), (16, 2)), ((9, 2500, 4100), (16, 4)),
         ((5, 64, 9000), (16, 8)), ((16, 2300, 8100), (16, 8)), ((15, 129, 7937), (16, 8)),
         ((30, 4500, 2100), (32, 2)), ((17, 3000, 5000), (32, 4)), ((20, 100, 9000), (32, 8)),
         ((32, 1025, 8193), (32, 8)), ((33, 200, 3000), (64, 1)), ((64, 6000, 8200), (64, 2)),
         ((100, 2000, 5000), (64, 4)), ((64, 1000, 9000), (64, 8)), ((70, 1000, 8000), (64, 8)),
         ((512, 4096, 512), (128, 1)), ((1280, 1280, 200), (128, 1)), ((20000, 100, 96), (128, 1)),
         ((127, 20001, 64), (128, 1)), ((16385, 64, 300), (128, 1)), ((2100, 1900, 900), (256, 1))]
IDS = ["x".join(map(str, s)) for s, _ in PLANS]


def plan(sg, M, N, K):  # noqa: F811
    tile, split = ctypes.c_int(), ctypes.c_int()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert sg.load().sgemm_mx4_choose_check(M, N, K, sms, ctypes.byref(tile), ctypes.byref(split)) == 0
    return tile.value, split.value


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("size,expect", PLANS, ids=IDS)
def test_each_plan_is_exact(sg, size, expect, fmt):  # noqa: F811
    M, N, K = size
    assert plan(sg, M, N, K) == expect
    a, va = random_stored(sg, M, K, fmt, 2 * M + K, True)
    b, vb = random_stored(sg, N, K, fmt, 3 * N + K, True)
    assert torch.equal(sg.mx4_matmul(a, b), exact(va, vb).float())


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("pad,off", [(0, 0), (5, 1)])
@pytest.mark.parametrize("size,expect", PLANS, ids=IDS)
def test_each_plan_scaled_into_views(sg, size, expect, pad, off, out):  # noqa: F811
    """alpha / 16 and beta = -2 of small whole numbers are exact in fp32: one rounding."""
    M, N, K = size
    fmt = "mxfp4" if pad else "nvfp4"
    a, va = random_stored(sg, M, K, fmt, M + K, True)
    b, vb = random_stored(sg, N, K, fmt, N + K, True)
    ld = N + pad
    buf = torch.randint(-8, 9, (off + M * ld,), device="cuda").to(out)
    before, c = buf.clone(), buf[off:].view(M, ld)[:, :N]
    want = (exact(va, vb) / 16 - 2 * c.double()).float().to(out)
    assert sg.mx4_matmul(a, b, c, alpha=1 / 16, beta=-2.0) is c
    assert torch.equal(c, want)
    if pad:
        assert torch.equal(buf[off:].view(M, ld)[:, N:], before[off:].view(M, ld)[:, N:])
        assert torch.equal(buf[:off], before[:off])
