"""8-bit activation checkpoints against the definition, bit by bit: every quotient, product and
rounding of the definition is one fp32 operation, which numpy does the same way."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SHAPES = [(1, 1), (1, 64), (1, 4096), (3, 7), (5, 65), (33, 257), (130, 1000), (7, 4100), (2, 40001),
          (700, 96), (1001, 8), (64, 64)]


@pytest.fixture()
def sg(cuda):
    import dense_fp32_gemm_09_gb300 as sg
    return sg


def reference(x):
    """(codes, scales) of a CPU tensor."""
    x = x.float().numpy()
    rows, cols = x.shape
    v = np.zeros((rows, -(-cols // 64) * 64), np.float32)
    v[:, :cols] = x
    v = v.reshape(rows, -1, 64)
    amax = np.abs(v).max(axis=2, keepdims=True)
    amax = np.where(np.isnan(v).any(axis=2, keepdims=True), np.float32(np.nan), amax)
    bad, low = ~np.isfinite(amax), amax < np.float32(2.0 ** -100)
    with np.errstate(all="ignore"):
        inv = np.where(bad | low, np.float32(0), np.float32(127) / amax).astype(np.float32)
        scale = np.where(low, np.float32(0), amax / np.float32(127)).astype(np.float32)
        over = np.isfinite(amax) & ~np.isfinite(scale * np.float32(127))
        scale = np.where(over, np.nextafter(scale, np.float32(0)), scale)
        scale = np.where(bad, np.float32(np.nan), scale)
        code = np.rint(np.where(bad, np.float32(0), v) * inv)
    return code.astype(np.int8).reshape(rows, -1), scale.reshape(rows, -1)


def check(sg, x, view=None):
    q = sg.act8_quantize(x.cuda() if view is None else view)
    codes, scales = reference(x)
    assert q.shape == tuple(x.shape)
    np.testing.assert_array_equal(q.codes.cpu().numpy(), codes)
    np.testing.assert_array_equal(q.scales.cpu().numpy(), scales)
    values = torch.from_numpy(codes.astype(np.float32) * np.repeat(scales, 64, axis=1))[:, :x.shape[1]]
    for dt in DTYPES.values():
        got, want = q.dequantize(dt).cpu(), values.to(dt)
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(torch.nan_to_num(got, 0, torch.inf, -torch.inf),
                           torch.nan_to_num(want, 0, torch.inf, -torch.inf))
    return q


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_codes_and_values(sg, rows, cols, dtype):
    g = torch.Generator().manual_seed(rows * 31 + cols)
    x = torch.randn(rows, cols, generator=g) * torch.randn(cols, generator=g).exp()
    check(sg, x.to(DTYPES[dtype]))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 0), (1, 3), (3, 5), (2, 6), (8, 0)])
def test_strides_and_alignment(sg, dtype, offset, pad):
    rows, cols = 37, 200
    g = torch.Generator().manual_seed(offset * 10 + pad)
    x = torch.randn(rows, cols, generator=g).to(DTYPES[dtype])
    flat = torch.full((offset + rows * (cols + pad) + 8,), float("nan"), dtype=x.dtype, device="cuda")
    view = flat[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    view.copy_(x)
    q = check(sg, x, view)
    out = torch.full_like(flat, 3.0)
    to = out[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
    sg.act8_dequantize(q, out=to)
    assert torch.equal(to, q.dequantize(x.dtype))
    rest = out.clone()
    rest[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols] = 3.0
    assert bool((rest == 3.0).all())


def test_ends_of_the_range(sg):
    """Infinities, NaN, zeros, subnormals, both sides of 2^-100, the largest numbers, ties."""
    x = torch.zeros(13, 130)
    x[0, 3], x[1, 70], x[2, 129] = float("inf"), float("nan"), float("-inf")
    x[3, :] = 1e-40
    x[4, 0], x[4, 64] = 2.0 ** -100, float(np.nextafter(np.float32(2.0 ** -100), np.float32(0)))
    x[5, :] = torch.linspace(-3.4028234e38, 3.4028234e38, 130)     # overflows itself: NaN
    x[6, :64] = torch.arange(64) * 2 + 1.0     # halves of steps: 127 / 127 = 1
    x[6, :64] /= 2
    x[6, 63] = 127.0
    x[7, :64] = -x[6, :64]
    x[8, 5] = -0.0
    x[9, :] = torch.randn(130, generator=torch.Generator().manual_seed(1)) * 2.0 ** -99
    x[10, 0], x[10, 1] = 3.4028234e38, 1e-45
    x[11, :] = 1.1754944e-38
    x[12, :] = torch.linspace(-1, 1, 130) * 3.4028234e38
    q = check(sg, x)
    assert bool(q.dequantize()[[3, 10, 12]].isfinite().all())
    check(sg, x.bfloat16())


def test_empty_and_refusals(sg):
    for shape in ((0, 5), (5, 0), (0, 0)):
        q = sg.act8_quantize(torch.empty(shape, device="cuda"))
        assert q.dequantize().shape == shape
    x = torch.randn(8, 70, device="cuda")
    q = sg.act8_quantize(x)
    for bad in (x.t(), x[:, ::2], x.double(), x.expand(2, 8, 70), x[:1].expand(8, 70), x.cpu(), 3):
        with pytest.raises((TypeError, ValueError)):
            sg.act8_quantize(bad)
    with pytest.raises(TypeError):
        sg.act8_dequantize(x)
    with pytest.raises(TypeError):
        sg.act8_dequantize(q, torch.float64)
    with pytest.raises(ValueError):
        sg.act8_dequantize(q, out=torch.empty(8, 71, device="cuda"))
    with pytest.raises(ValueError):
        sg.Act8(q.codes, q.scales, 8, 200)
    with pytest.raises(ValueError):
        sg.Act8(q.codes.float(), q.scales, 8, 70)
    again = sg.Act8(q.codes, q.scales, 8, 70)
    assert torch.equal(again.dequantize(), q.dequantize())


def test_long_offsets(sg):
    """More than 2^32 codes: rows past that offset are their own."""
    rows, cols = 70000, 65536
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(5, cols, generator=torch.Generator().manual_seed(2)).bfloat16()
    x[-5:] = tail.cuda()
    q = sg.act8_quantize(x)
    codes, scales = reference(tail)
    np.testing.assert_array_equal(q.codes[-5:].cpu().numpy(), codes)
    assert not bool(q.codes[-6].any()) and not bool(q.codes[0].any())
    y = q.dequantize(torch.bfloat16)
    want = torch.from_numpy(codes.astype(np.float32) * np.repeat(scales, 64, axis=1)).bfloat16()
    assert torch.equal(y[-5:].cpu(), want) and not bool(y[:7].any())
