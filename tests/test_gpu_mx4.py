"""4-bit quantisation and products on the GPU against the formats restated in numpy.

Quantisation is exact: every code and scale byte has to be the reference's.  A product's
sum has at most K / 8 sequential additions (the tensor core adds several products at a
time), each off by at most one fp32 ulp (2^-23, truncation) of the running sum, so
|error| <= (K / 8 + 8) 2^-23 sum |a b|, plus the rounding to C's type."""
import numpy as np
import pytest
import torch

import mx4_reference as ref

pytestmark = pytest.mark.gpu

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
HALF_ULP = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


@pytest.fixture()
def sg(cuda):
    import dense_fp32_gemm_09_gb300 as sg
    return sg


def sample(rows, cols, dtype, seed):
    """Numbers of many magnitudes, with zeros, exact ties and whole zero blocks."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g) * torch.exp2(
        torch.randint(-6, 7, (rows, cols), generator=g).float())
    tie = torch.tensor([.25, .75, 1.25, 1.75, 2.5, 3.5, 5., 6., -0.0, 0.0])
    pick = torch.randint(0, 10, (rows, cols), generator=g)
    x = torch.where(torch.rand((rows, cols), generator=g) < 0.3, tie[pick], x)
    x[torch.rand((rows,), generator=g) < 0.1] = 0
    return x.to(DTYPES[dtype])


def check_stored(q, x, fmt, ts=None):
    code, sb = ref.quantize(x.float().cpu().numpy(), fmt, ts)
    codes, scales = ref.store(code, sb, fmt)
    rows = x.shape[0]
    for got, want, what in ((q.codes, codes, "codes"), (q.scales, scales, "scales")):
        got = got.cpu().numpy()
        if what == "codes":     # by row, padded rows left out
            got, want = (v.transpose(0, 2, 1, 3).reshape(-1, v.shape[1] * 16)[:rows]
                         for v in (got, want))
        else:
            got, want = (v.transpose(0, 3, 2, 1, 4).reshape(-1, v.shape[1] * 4)[:rows]
                         for v in (got, want))
        if what == "codes":     # a NaN block's codes say nothing
            keep = np.repeat(np.pad(sb != (0x7F if fmt == "nvfp4" else 255),
                                    ((0, 0), (0, want.shape[1] * 2 // ref.BLOCK[fmt] - sb.shape[1])),
                                    constant_values=True), ref.BLOCK[fmt] // 2, axis=1)
            got, want = np.where(keep, got, 0), np.where(keep, want, 0)
        assert np.array_equal(got, want), what
    return code, sb


SIZES = [(1, 1), (1, 4096), (3, 31), (5, 32), (127, 33), (128, 128), (129, 257), (300, 1000),
         (2, 4097), (515, 64), (34, 130), (130, 2056), (64, 999), (257, 96), (1000, 130)]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", SIZES)
def test_quantize_matches_the_format(sg, rows, cols, dtype, fmt):
    x = sample(rows, cols, dtype, rows + cols)
    q = sg.mx4_quantize(x.cuda(), fmt)
    check_stored(q, x, fmt)
    xt = x.t().contiguous().t()          # the same matrix, stored transposed
    check_stored(sg.mx4_quantize(xt.cuda(), fmt), x, fmt)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("ts", [1.0, 2.0 ** -7, 0.0123, 3e5, 1e-30])
def test_tensor_scale(sg, dtype, ts):
    x = sample(70, 200, dtype, 5)
    t = torch.tensor([ts], device="cuda")
    q = sg.mx4_quantize(x.cuda(), "nvfp4", tensor_scale=t)
    code, sb = check_stored(q, x, "nvfp4", np.float32(ts))
    # Read back: (code * s) * ts in fp32; code * s is exact.
    want = (ref.values(code, sb, "nvfp4", 200).astype(np.float32) * np.float32(ts))
    assert np.array_equal(q.dequantize().cpu().numpy(), want)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("offset,pad", [(0, 0), (1, 0), (0, 3), (8, 8), (3, 16)])
def test_strided_and_misaligned_views(sg, dtype, fmt, offset, pad):
    rows, cols = 150, 96 + 40
    x = sample(rows, cols, dtype, 9)
    for stored in (x, x.t()):
        r, c = stored.shape
        buf = torch.full((offset + r * (c + pad) + 8,), float("nan"), dtype=x.dtype, device="cuda")
        view = buf[offset:offset + r * (c + pad)].view(r, c + pad)[:, :c]
        view.copy_(stored)
        check_stored(sg.mx4_quantize(view if stored is x else view.t(), fmt), x, fmt)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_specials(sg, fmt):
    x = torch.zeros((12, 64))
    x[0, 3], x[1, 3], x[2, 3] = float("inf"), float("-inf"), float("nan")
    x[3, :] = 1e-45                       # the least subnormal
    x[4, 5] = 1e-40
    x[5, :] = 3.4028234663852886e38
    x[6, :] = -0.0
    x[7, :] = 2.0 ** -126
    x[8, 0], x[8, 1] = 1e30, 1e-30
    x[9, 16:32] = -448 * 6.0
    x[10, 0] = 448 * 6.0 * 1.04           # past the largest scale
    x[11, 40] = 2.0 ** -10 * 6            # half the least scale: rounds to 0
    q = sg.mx4_quantize(x.cuda(), fmt)
    code, sb = check_stored(q, x, fmt)
    with np.errstate(all="ignore"):
        want = ref.values(code, sb, fmt, 64).astype(np.float32)
    assert np.array_equal(q.dequantize().cpu().numpy(), want, equal_nan=True)
    y = q.dequantize(torch.bfloat16).float().cpu().numpy()
    assert np.isnan(y[0:3, :16]).all() and np.isfinite(y[0:3, 32:]).all()


def test_quotients_near_every_tie(sg):
    """x = t s (1 + j ulp) around each rounding boundary t, for every e4m3 scale: the code
    has to follow the fp32 quotient, also for scales that are not powers of two."""
    mids = (ref.E2M1[1:] + ref.E2M1[:-1]) / 2
    rows = []
    for s in ref.E4M3[1:]:
        top = np.float32(6 * s)
        t = (mids * s).astype(np.float32)
        near = [t]
        lo, hi = t, t
        for _ in range(2):
            lo, hi = np.nextafter(lo, np.float32(0)), np.nextafter(hi, np.float32(1e9))
            near += [lo, hi]
        v = np.concatenate(near)
        v = np.concatenate([v, -v, v[:5]])
        for i in range(0, len(v), 15):
            rows.append(np.concatenate([[top], v[i:i + 15]]))
    x = torch.from_numpy(np.stack(rows).astype(np.float32))
    check_stored(sg.mx4_quantize(x.cuda(), "nvfp4"), x, "nvfp4")
    for ts in (0.37, 1.0 + 2.0 ** -23, 7.7e-5):
        y = x * ts
        check_stored(sg.mx4_quantize(y.cuda(), "nvfp4", tensor_scale=torch.tensor([ts]).cuda()),
                     y, "nvfp4", np.float32(ts))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_dequantize_into_views(sg, dtype, fmt):
    x = sample(131, 77, "fp32", 3)
    q = sg.mx4_quantize(x.cuda(), fmt)
    code, sb = ref.quantize(x.numpy(), fmt)
    want = torch.from_numpy(ref.values(code, sb, fmt, 77)).to(DTYPES[dtype]).cuda()
    for ld, off in ((77, 0), (80, 0), (96, 1)):
        buf = torch.full((off + 131 * ld,), 7.0, dtype=DTYPES[dtype], device="cuda")
        out = buf[off:].view(131, ld)[:, :77]
        assert sg.mx4_dequantize(q, out=out) is out
        assert torch.equal(out, want)
        assert bool((buf[off:].view(131, ld)[:, 77:] == 7).all())


def random_stored(sg, rows, cols, fmt, seed, exact):
    """A quantised matrix of random codes; padded rows hold bytes that would show."""
    rng = np.random.default_rng(seed)
    nb = -(-cols // ref.BLOCK[fmt])
    code = rng.integers(0, 16, (rows, nb * ref.BLOCK[fmt])).astype(np.uint8)
    code[:, cols:] = 0
    if fmt == "nvfp4":   # 2^-1 .. 2, or any scale up to 4
        sb = rng.choice([48, 56, 64], (rows, nb)) if exact else rng.integers(0, 72, (rows, nb))
    else:
        sb = rng.integers(126, 129, (rows, nb)) if exact else rng.integers(118, 130, (rows, nb))
    sb = sb.astype(np.uint8)
    codes, scales = ref.store(code, sb, fmt, fill=0x7F)
    ts = None
    if fmt == "nvfp4" and not exact:
        ts = torch.tensor([0.37 + seed % 5], device="cuda")
    q = sg.Mx4(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), rows, cols, fmt, ts)
    return q, ref.values(code, sb, fmt, cols, None if ts is None else ts.item())


MNK = [(1, 1, 1), (1, 16, 16), (1, 300, 100), (2, 128, 64), (7, 129, 257), (16, 256, 128),
       (17, 100, 4096), (33, 384, 95), (64, 64, 1000), (100, 257, 33), (128, 128, 128),
       (129, 130, 160), (200, 333, 511), (256, 512, 768), (300, 1000, 97), (513, 255, 640),
       (1, 5000, 2048), (5, 64, 7000), (1000, 40, 200), (700, 900, 384),
       (1537, 1793, 640), (2049, 2047, 1111), (1300, 3000, 64), (4100, 1000, 1920)]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("M,N,K", MNK)
def test_product_is_exact_where_fp32_is(sg, M, N, K, fmt):
    """Scales of 1/2, 1 and 2: every partial sum is a multiple of 1/16 below 2^20, so any
    order of summation gives the exact product."""
    a, va = random_stored(sg, M, K, fmt, 2 * M + K, True)
    b, vb = random_stored(sg, N, K, fmt, 3 * N + K, True)
    want = va @ vb.T
    got = sg.mx4_matmul(a, b)
    assert np.array_equal(got.cpu().numpy().astype(np.float64), want)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("out", list(DTYPES))
@pytest.mark.parametrize("M,N,K", [(1, 700, 1000), (40, 300, 4100), (300, 260, 2000)])
def test_product_within_bound(sg, M, N, K, out, fmt):
    a, va = random_stored(sg, M, K, fmt, 11, False)
    b, vb = random_stored(sg, N, K, fmt, 12, False)
    scale = 2.0 ** -8 if out == "fp16" else 1.0    # keeps fp16 in range
    want = scale * (va @ vb.T)
    mag = scale * (np.abs(va) @ np.abs(vb).T)
    got = sg.mx4_matmul(a, b, dtype=DTYPES[out], alpha=scale).double().cpu().numpy()
    tol = (K / 8 + 8) * 2.0 ** -23 * mag + HALF_ULP[out] * np.abs(want) * 1.01 + 2.0 ** -24
    assert (np.abs(got - want) <= tol).all(), float((np.abs(got - want) - tol).max())


@pytest.mark.parametrize("out", list(DTYPES))
@pytest.mark.parametrize("alpha,beta", [(1.0, 1.0), (0.5, -2.0), (2.0, 0.0)])
@pytest.mark.parametrize("M,N,K,pad,off", [(3, 50, 64, 0, 0), (37, 133, 200, 5, 1), (300, 300, 96, 4, 0)])
def test_scaled_product_into_views(sg, M, N, K, pad, off, alpha, beta, out):
    a, va = random_stored(sg, M, K, "mxfp4", 1, True)
    b, vb = random_stored(sg, N, K, "mxfp4", 2, True)
    ld = N + pad
    buf = torch.randint(-8, 9, (off + M * ld,), device="cuda").to(DTYPES[out])
    if beta == 0:
        buf.fill_(float("nan"))
    before = buf.clone()
    c = buf[off:].view(M, ld)[:, :N]
    start = c.double().cpu().numpy()
    sg.mx4_matmul(a, b, c, alpha=alpha, beta=beta)
    want = alpha * (va @ vb.T) + (beta * start if beta else 0)     # exact in fp32
    assert torch.equal(c.cpu(), torch.from_numpy(want).to(DTYPES[out]))
    if pad:
        gap, was = buf[off:].view(M, ld)[:, N:], before[off:].view(M, ld)[:, N:]
        assert torch.equal(gap.nan_to_num(9), was.nan_to_num(9))


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_nan_stays_in_its_row_and_column(sg, fmt):
    x, w = torch.randn(20, 256), torch.randn(150, 256)
    x[4, 100] = float("inf")
    w[140, 7] = float("nan")
    c = sg.mx4_matmul(sg.mx4_quantize(x.cuda(), fmt), sg.mx4_quantize(w.cuda(), fmt)).cpu()
    bad = torch.zeros(20, 150, dtype=torch.bool)
    bad[4], bad[:, 140] = True, True
    assert torch.equal(torch.isnan(c), bad)


def test_empty_and_degenerate(sg):
    one = torch.ones((3, 0), device="cuda")
    a = sg.mx4_quantize(one, "nvfp4")
    b = sg.mx4_quantize(torch.ones((5, 0), device="cuda"), "nvfp4")
    assert torch.equal(sg.mx4_matmul(a, b), torch.zeros(3, 5, device="cuda"))
    c = torch.ones((3, 5), device="cuda")
    assert bool((sg.mx4_matmul(a, b, c, beta=3.0) == 3).all())
    e = sg.mx4_quantize(torch.ones((0, 64), device="cuda"), "nvfp4")
    w = sg.mx4_quantize(torch.ones((5, 64), device="cuda"), "nvfp4")
    assert sg.mx4_matmul(e, w).shape == (0, 5) and e.dequantize().shape == (0, 64)
    assert sg.mx4_matmul(w, e).shape == (5, 0)
    x = sg.mx4_quantize(torch.full((2, 64), float("nan"), device="cuda"), "nvfp4")
    c = torch.ones((2, 5), device="cuda")
    assert bool((sg.mx4_matmul(x, w, c, alpha=0.0, beta=2.0) == 2).all())   # x is not read


def test_rows_far_into_a_large_matrix(sg):
    """More than 2^31 elements of X: offsets pass 32 bits."""
    rows, cols = 33008, 65536 + 64
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    tail = sample(1, cols, "bf16", 2)
    x[-1] = tail[0].cuda()
    q = sg.mx4_quantize(x, "nvfp4")
    code, sb = ref.quantize(tail.float().numpy(), "nvfp4")
    want = torch.from_numpy(ref.values(code, sb, "nvfp4", cols)).float()
    y = sg.mx4_dequantize(q, torch.bfloat16)
    assert torch.equal(y[-1].float().cpu(), want[0]) and not bool(y[:-1].any())
    qt = sg.mx4_quantize(x.t(), "nvfp4")
    code, sb = ref.quantize(np.pad(tail.float().numpy().T, ((0, 0), (15, 0))), "nvfp4")
    del y, x
    at = (rows - 1) // 32
    assert (rows - 1) % 16 == 15
    got = qt.codes[:, at].reshape(-1, 16)[:cols, ((rows - 1) % 32) // 2].cpu().numpy() >> 4
    assert np.array_equal(got, code[:, 15])


def test_other_stream_and_graph(sg):
    x = sample(64, 256, "bf16", 1).cuda()
    w = sg.mx4_quantize(sample(96, 256, "bf16", 2).cuda())
    want = sg.mx4_matmul(sg.mx4_quantize(x), w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        own = sg.mx4_matmul(sg.mx4_quantize(x), w)
    given = sg.mx4_matmul(sg.mx4_quantize(x, stream=s), w, stream=s)
    s.synchronize()
    assert torch.equal(own, want) and torch.equal(given, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = sg.mx4_matmul(sg.mx4_quantize(x), w)
    x.mul_(2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want * 2)


def test_refusals(sg):
    x = torch.randn(8, 64, device="cuda")
    q = sg.mx4_quantize(x)
    with pytest.raises(ValueError, match="fmt"):
        sg.mx4_quantize(x, "fp4")
    with pytest.raises(TypeError):
        sg.mx4_quantize(x.double())
    with pytest.raises(ValueError, match="CUDA"):
        sg.mx4_quantize(x.cpu())
    with pytest.raises(ValueError, match="2-D"):
        sg.mx4_quantize(x[0])
    with pytest.raises(ValueError, match="unit stride"):
        sg.mx4_quantize(torch.randn(8, 8, 8, device="cuda")[:, ::2, ::2][0])
    with pytest.raises(ValueError, match="overlap"):
        sg.mx4_quantize(x[:1].expand(4, 64))
    with pytest.raises(ValueError, match="nvfp4"):
        sg.mx4_quantize(x, "mxfp4", tensor_scale=torch.ones(1, device="cuda"))
    with pytest.raises(TypeError, match="one float32"):
        sg.mx4_quantize(x, tensor_scale=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError, match="inner"):
        sg.mx4_matmul(q, sg.mx4_quantize(x[:, :32].contiguous()))
    with pytest.raises(ValueError, match="formats"):
        sg.mx4_matmul(q, sg.mx4_quantize(x, "mxfp4"))
    with pytest.raises(TypeError, match="Mx4"):
        sg.mx4_matmul(x, q)
    with pytest.raises(ValueError, match="beta"):
        sg.mx4_matmul(q, q, beta=1.0)
    with pytest.raises(ValueError, match="out must be"):
        sg.mx4_matmul(q, q, torch.empty(8, 9, device="cuda"))
    with pytest.raises(sg.SgemmError, match="NaN"):
        sg.mx4_matmul(q, q, alpha=float("nan"))
    with pytest.raises(ValueError, match="contiguous uint8"):
        sg.Mx4(q.codes[:, :2], q.scales, 8, 64, "nvfp4")
    with pytest.raises(ValueError, match="contiguous uint8"):
        sg.Mx4(q.codes, q.scales, 300, 64, "nvfp4")
