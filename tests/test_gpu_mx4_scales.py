"""Tensor scales at the ends of their range, and those whose quotients are hardest."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
from test_gpu_mx4 import DTYPES, check_stored, sample, sg  # noqa: F401  (sg: fixture)

pytestmark = pytest.mark.gpu


def held(q):
    return q.dequantize().double().cpu()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 40), (130, 200), (64, 1024)])
def test_zeros_with_their_own_scale(sg, rows, cols, dtype):  # noqa: F811
    """amax(x) / 2688 of zeros is 0: zeros are held, and products with them are 0."""
    x = torch.zeros(rows, cols, dtype=DTYPES[dtype], device="cuda")
    ts = (x.abs().amax().float() / (6 * 448)).view(1)
    w = sg.mx4_quantize(sample(70, cols, "bf16", 3).cuda())
    for q in (sg.mx4_quantize(x, tensor_scale=ts),
              sg.mx4_quantize(x.t().contiguous().t(), tensor_scale=ts)):
        assert not bool(held(q).any())
        rows_of = lambda b, order, n: b.permute(order).reshape(-1, n)[:rows]
        assert not bool(rows_of(q.codes, (0, 2, 1, 3), q.codes.shape[1] * 16).any())
        assert not bool(rows_of(q.scales, (0, 3, 2, 1, 4), q.scales.shape[1] * 4).any())
        c = sg.mx4_matmul(q, w)
        assert c.shape == (rows, 70) and not bool(c.any())
        assert not bool(sg.mx4_matmul(w, q).any())


@pytest.mark.parametrize("ts", [0.0, -0.0])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_scale_of_zero_holds_zeros(sg, dtype, ts):  # noqa: F811
    """Whatever the numbers; a block with a NaN or an infinity is NaN as always."""
    x = sample(70, 200, dtype, 5)
    x[3, 20], x[5, 199] = float("nan"), float("inf")
    t = torch.tensor([ts], device="cuda")
    for v in (x.cuda(), x.t().contiguous().cuda().t()):
        got = held(sg.mx4_quantize(v, tensor_scale=t))
        want = torch.zeros(70, 200, dtype=torch.float64)
        want[3, 16:32], want[5, 192:] = float("nan"), float("nan")
        assert torch.equal(got.isnan(), want.isnan()) and not bool(got.nan_to_num().any())


@pytest.mark.parametrize("ts", [0.0, 3e-39, 1e-45, float("inf")])
def test_zero_blocks_stay_zero(sg, ts):  # noqa: F811
    """Blocks of zeros have scale 0 under any tensor scale."""
    x = torch.zeros(40, 96)
    x[::2, 32:48] = torch.randn(20, 16) * 1e-37
    q = sg.mx4_quantize(x.cuda(), tensor_scale=torch.tensor([ts], device="cuda"))
    s = q.scales.permute(0, 3, 2, 1, 4).reshape(-1, q.scales.shape[1] * 4)[:40].cpu()
    assert not bool(s[:, [0, 1, 3, 4, 5, 6, 7]].any()) and not bool(s[1::2].any())


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", [(5, 512), (400, 512), (400, 264), (6, 9001), (3, 20001), (400, 77)])
def test_norms_of_zero_scale(sg, rows, cols, dtype):  # noqa: F811
    """The norms quantise by the same rule in each of their kernels."""
    x = torch.randn(rows, cols).to(DTYPES[dtype]).cuda()
    x[1] = 0
    t = torch.zeros(1, device="cuda")
    h, _ = sg.norm_before(x, quantize="nvfp4", tensor_scale=t)
    _, _, h2, _ = sg.norm_after(x, torch.zeros_like(x), quantize="nvfp4", tensor_scale=t)
    for q in (h, h2):
        assert not bool(held(q).any())
    y = sg.mx4_matmul(h, sg.mx4_quantize(torch.ones(33, cols, device="cuda")))
    assert np.array_equal(y.cpu().numpy(), np.zeros((rows, 33)))


def around(v, steps=4):
    """fp32 numbers next to each of v."""
    out, lo, hi = [v], v, v
    for _ in range(steps):
        lo, hi = np.nextafter(lo, np.float32(0)), np.nextafter(hi, np.float32(1e30))
        out += [lo, hi]
    return np.concatenate(out)


@pytest.mark.parametrize("base", [1 << 23, 3 << 22, 1 << 24])
def test_quotients_of_the_hardest_divisors(sg, base):  # noqa: F811
    """Scales next to the significands where a quotient is nearest to a tie without being one."""
    mids = ((ref.E2M1[1:] + ref.E2M1[:-1]) / 2).astype(np.float32)
    for j in [j for j in range(-34, 35) if 1 << 23 <= base + j < 1 << 24]:
        ts = np.float32((base + j) * 2.0 ** -23)
        v = around(mids * ts)
        v = np.concatenate([v, -v, v])[:126 // 15 * 15]
        x = np.concatenate([np.full((len(v) // 15, 1), 6 * ts, np.float32), v.reshape(-1, 15)], 1)
        check_stored(sg.mx4_quantize(torch.from_numpy(x).cuda(),
                                     tensor_scale=torch.tensor([ts], device="cuda")),
                     torch.from_numpy(x), "nvfp4", ts)


@pytest.mark.parametrize("base", [i << 20 for i in range(8, 17)])
def test_block_scales_of_the_hardest_divisors(sg, base):  # noqa: F811
    """The same for the block's scale, amax / (6 ts)."""
    mids = ((ref.E4M3[1:] + ref.E4M3[:-1]) / 2).astype(np.float32)
    for j in [j for j in range(-34, 35, 3) if 1 << 23 <= base + j < 1 << 24]:
        six = np.float32((base + j) * 2.0 ** -23)
        ts = np.float32(six / np.float32(6))
        for t in (np.nextafter(ts, np.float32(0)), ts, np.nextafter(ts, np.float32(9))):
            x = np.zeros((len(mids) * 9, 16), np.float32)
            x[:, 5] = around(mids * (np.float32(6) * t))
            x[:, 9] = -x[:, 5] / 3
            check_stored(sg.mx4_quantize(torch.from_numpy(x).cuda(),
                                         tensor_scale=torch.tensor([t], device="cuda")),
                         torch.from_numpy(x), "nvfp4", t)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 77), (130, 200), (64, 1025), (34, 130)])
def test_padding_after_what_is_not_a_number(sg, rows, cols, dtype, fmt):  # noqa: F811
    """Codes past the row's end are zeros also in a block whose scale is NaN, and that block
    makes its row of a product NaN."""
    x = sample(rows, cols, dtype, 2)
    x[0, cols - 1] = float("nan")
    x[rows - 1, cols - 1] = float("inf")
    for v in (x.cuda(), x.t().contiguous().cuda().t()):
        q = sg.mx4_quantize(v, fmt)
        check_stored(q, x, fmt)
        byte = q.codes.transpose(1, 2).reshape(-1, q.codes.shape[1] * 16)[:rows]
        code = torch.stack((byte & 15, byte >> 4), 2).view(rows, -1)
        assert not bool(code[:, cols:].any())
        c = sg.mx4_matmul(q, sg.mx4_quantize(torch.ones(20, cols, device="cuda"), fmt))
        bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
        bad[0] = bad[rows - 1] = True
        assert torch.equal(c.isnan(), bad[:, None].expand(rows, 20))
