"""Layer norm and its gradient against their formulas in 64 bits.

Tolerances.  u is half an ulp of the output's type (2^-24, 2^-8, 2^-11).  A row's sum of D
terms is at most D / 128 + 32 sequential fp32 additions deep, so it is off by at most
e = (D / 128 + 32) 2^-24 of the sum of its terms' magnitudes.  With A = mean |x| the mean is off by
em = e A; the variance by its own sum's error and by em (squared, as differences to the true
mean add to 0, and once through their own rounding); rstd by half the variance's relative error
and 2^-22 for the root.  Column sums over R rows are R / 64 + 40 deep."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
HALF_ULP = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
EPS, E24 = 1e-5, 2.0 ** -24
SHAPES = [(1, 1), (1, 2), (1, 4096), (3, 7), (5, 64), (33, 257), (130, 1000), (2, 2048), (4, 8200),
          (2, 40001), (700, 96), (2, 70000), (330, 4096), (3, 5000), (2, 4100), (5, 12000),
          (2, 16384), (9, 8192), (300, 128), (3, 16392), (2, 32768), (40, 2047)]


@pytest.fixture()
def sg(cuda):
    import dense_fp32_gemm_09_gb300 as sg
    return sg


def f64(t):
    return t.double().cpu()


def near(got, want, tol, what):
    got = f64(got)
    bad = (got - want).abs() - tol
    assert torch.isfinite(got).all() and bool((bad <= 0).all()), (what, float(bad.max()))


class Case:
    def __init__(self, rows, cols, dtype, weights="fp32", seed=0, mean=0.7):
        g = torch.Generator().manual_seed(rows * 7 + cols + seed)
        r = lambda *s: torch.randn(s, generator=g)
        dt = DTYPES[dtype]
        self.rows, self.cols, self.u = rows, cols, HALF_ULP[dtype]
        self.x = (r(rows, cols) * 2 + mean).to(dt)
        self.dh, self.dy = r(rows, cols).to(dt), r(rows, cols).to(dt)
        wt = dt if weights == "own" else torch.float32
        self.w = None if weights == "none" else (1 + 0.3 * r(cols)).to(wt)
        self.b = None if weights == "none" else (0.3 * r(cols)).to(wt)
        self.e = (cols / 128 + 32) * E24
        self.ec = (rows / 64 + 40) * E24


def cuda(t):
    return None if t is None else t.cuda()


def vec(t, cols, none):
    return torch.full((cols,), none, dtype=torch.float64) if t is None else f64(t)


def moments(c, eps=EPS):
    """m, r and how far a computed pair may be off."""
    x = f64(c.x)
    m = x.mean(1)
    d = x - m[:, None]
    v = (d * d).mean(1)
    em = c.e * x.abs().mean(1) + E24 * m.abs()
    ed = em + E24 * (d.abs().amax(1) + em)
    ev = v * (c.e + 4 * E24) + em * em + 2 * ed * E24 * d.abs().mean(1) + 2 * em * c.e * d.abs().mean(1)
    r = (v + eps) ** -0.5
    return m, r, em, 0.5 * ev / (v + eps) + 2.0 ** -22


def check_forward(sg, c, view=None, eps=EPS):
    got = sg.layer_norm(cuda(c.x) if view is None else view, cuda(c.w), cuda(c.b), eps=eps)
    m, r, em, er = moments(c, eps)
    near(got[1], m, em, "mean")
    near(got[2], r, er * r, "rstd")
    n = (f64(c.x) - m[:, None]) * r[:, None]
    w, b = vec(c.w, c.cols, 1.0), vec(c.b, c.cols, 0.0)
    y = n * w + b
    tol = (em * r)[:, None] * w.abs() * 1.01 + (n * w).abs() * (er[:, None] + 4 * E24) + \
        E24 * (y.abs() + b.abs()) + c.u * y.abs() * 1.01 + 1e-7
    near(got[0], y, tol, "y")
    return got


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(sg, rows, cols, dtype):
    for weights in ("fp32", "none", "own"):
        check_forward(sg, Case(rows, cols, dtype, weights))


def test_only_one_of_weight_and_bias(sg):
    c = Case(9, 333, "bf16")
    b, c.b = c.b, None
    check_forward(sg, c)
    c.w, c.b = None, b
    check_forward(sg, c)


@pytest.mark.parametrize("cols", [2, 63, 1024, 2047, 4096, 8192, 20000])
def test_rows_without_spread(sg, cols):
    """Rows of one number: the variance is 0 up to rounding, not a difference of large squares;
    rows whose mean is far from 0 beside their spread."""
    c = Case(6, cols, "fp32")
    c.x[0], c.x[1], c.x[2] = 0.0, 1000.0, -3e4 / 7
    c.x[3] = 4096 + torch.randn(cols, generator=torch.Generator().manual_seed(3)) / 8
    c.x[4] *= 1e-12
    check_forward(sg, c)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 64), (33, 257), (130, 1000), (3, 4096), (9, 8192),
                                       (40, 2047), (4, 20000), (2, 40001), (3, 4100)])
def test_kept_input_is_the_checkpoint(sg, rows, cols, dtype):
    c = Case(rows, cols, dtype)
    y, mean, rstd, kept = sg.layer_norm(cuda(c.x), cuda(c.w), cuda(c.b), keep="8bit")
    for got, want in zip((y, mean, rstd), sg.layer_norm(cuda(c.x), cuda(c.w), cuda(c.b))):
        assert torch.equal(got, want)
    q = sg.act8_quantize(cuda(c.x))
    assert torch.equal(kept.codes, q.codes) and torch.equal(kept.scales, q.scales)


def check_backward(sg, c, x, x64, dy=True, views=None):
    dh, dyv = (cuda(c.dh), cuda(c.dy)) if views is None else views
    m, r = (t.float() for t in moments(c)[:2])
    dx, dw, db = sg.layer_norm_backward(dh, x, m.cuda(), r.cuda(), cuda(c.w), dy=dyv if dy else None)
    m, r = f64(m)[:, None], f64(r)[:, None]
    n, w, h = (x64 - m) * r, vec(c.w, c.cols, 1.0), f64(c.dh)
    en = 3 * E24 * (n.abs() + (m * r).abs() + (x64 * r).abs())       # of n, element by element
    g = w * h
    mean = lambda t: t.mean(1, keepdim=True)
    want = r * (g - mean(g) - n * mean(g * n))
    gn, gna = mean(g * n).abs(), mean((g * n).abs())
    tol = r * ((c.e + 8 * E24) * (g.abs() + mean(g.abs()) + n.abs() * gna) + en * gn +
               n.abs() * mean(g.abs() * en)) * 1.01
    if dy:
        want, tol = want + f64(c.dy), tol + 2 * E24 * f64(c.dy).abs()
    near(dx, want, tol + c.u * want.abs() * 1.01 + 1e-7, "dx")
    near(db, h.sum(0), (c.ec + E24) * h.abs().sum(0) + 1e-30, "dbias")
    if c.w is None:
        assert dw is None
    else:
        near(dw, (h * n).sum(0), (c.ec + 2 * E24) * (h * n).abs().sum(0) + (h.abs() * en).sum(0) + 1e-30,
             "dweight")
    return dx, dw, db


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(sg, rows, cols, dtype):
    c = Case(rows, cols, dtype)
    first = check_backward(sg, c, cuda(c.x), f64(c.x))
    again = check_backward(sg, c, cuda(c.x), f64(c.x))
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    for weights in ("none", "own"):
        c = Case(rows, cols, dtype, weights)
        check_backward(sg, c, cuda(c.x), f64(c.x), dy=False)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward_from_a_checkpoint(sg, rows, cols, dtype):
    c = Case(rows, cols, dtype)
    q = sg.act8_quantize(cuda(c.x))
    check_backward(sg, c, q, f64(q.dequantize()))
    c = Case(rows, cols, dtype, "none")
    q = sg.act8_quantize(cuda(c.x))
    check_backward(sg, c, q, f64(q.dequantize()), dy=False)


@pytest.mark.parametrize("rows", [1000, 3001, 20000])
@pytest.mark.parametrize("cols,dtype", [(64, "bf16"), (1000, "fp32"), (2047, "bf16"), (1024, "fp16")])
def test_sums_over_many_rows(sg, rows, cols, dtype):
    c = Case(rows, cols, dtype)
    check_backward(sg, c, cuda(c.x), f64(c.x))


def test_gradient_against_differences(sg):
    """The formula's gradient is the forward pass's: central differences in 64 bits of the
    reference, which the forward test ties to the kernels."""
    c = Case(4, 96, "fp32")
    x, w, b, h = f64(c.x), f64(c.w), f64(c.b), f64(c.dh)

    def loss(x, w, b):
        m = x.mean(1, keepdim=True)
        d = x - m
        return ((d * ((d * d).mean(1, keepdim=True) + EPS) ** -0.5 * w + b) * h).sum()

    y, mean, rstd = sg.layer_norm(cuda(c.x), cuda(c.w), cuda(c.b), eps=EPS)
    dx, dw, db = sg.layer_norm_backward(cuda(c.dh), cuda(c.x), mean, rstd, cuda(c.w))
    for which, got in ((0, dx), (1, dw), (2, db)):
        at = [x, w, b]
        for i in range(0, at[which].numel(), 7):
            step = torch.zeros_like(at[which])
            step.view(-1)[i] = 1e-5
            up, down = list(at), list(at)
            up[which], down[which] = at[which] + step, at[which] - step
            want = float(loss(*up) - loss(*down)) / 2e-5
            # 1e-10 (step squared) of third derivatives, and fp32 sums of about 100 terms.
            assert abs(float(got.view(-1)[i]) - want) < 2e-5 * (1 + abs(want))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 0), (1, 3), (3, 5), (2, 6), (8, 0)])
def test_strides_and_alignment(sg, dtype, offset, pad):
    c = Case(37, 200, dtype)

    def strided(t):
        flat = torch.full((offset + 37 * (200 + pad) + 8,), float("nan"), dtype=t.dtype, device="cuda")
        view = flat[offset:offset + 37 * (200 + pad)].view(37, 200 + pad)[:, :200]
        view.copy_(t)
        return view

    check_forward(sg, c, strided(c.x))
    check_backward(sg, c, strided(c.x), f64(c.x), views=(strided(c.dh), strided(c.dy)))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_rows_at_different_places(sg, rows, cols, dtype):
    """Matrices that begin at different places of a 16-byte group, and all at the same one past its
    start: as contiguous ones."""
    c = Case(rows, cols, dtype)

    def at(t, offset):
        flat = torch.full((t.numel() + 16,), float("nan"), dtype=t.dtype, device="cuda")
        view = flat[offset:offset + t.numel()].view(t.shape)
        view.copy_(t)
        return view

    x = cuda(c.x)
    want = sg.layer_norm(x, cuda(c.w), cuda(c.b), keep="8bit")
    for offset in (1, 3):
        got = check_forward(sg, c, at(c.x, offset))
        kept = sg.layer_norm(at(c.x, offset), cuda(c.w), cuda(c.b), keep="8bit")[3]
        assert torch.equal(kept.codes, want[3].codes) and torch.equal(kept.scales, want[3].scales)
        check_backward(sg, c, at(c.x, offset), f64(c.x), views=(at(c.dh, 2 * offset), at(c.dy, 1)))
        check_backward(sg, c, kept, f64(kept.dequantize()), views=(at(c.dh, offset), at(c.dy, 2)))


@pytest.mark.parametrize("rows,cols,pad", [(700, 2047, 0), (700, 2047, 2), (41, 1001, 7), (700, 1022, 0), (9, 6, 0),
                                           (310, 4097, 0), (1000, 5001, 0), (400, 4100, 1), (320, 8185, 2),
                                           (500, 8191, 0), (400, 9001, 0), (350, 20003, 0), (310, 33000, 1)])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_rows_at_one_place(sg, rows, cols, pad, dtype):
    """Every matrix of the C call begins at the same place of a 16-byte group, which is not its start,
    and nothing outside the outputs is written."""
    import ctypes
    c, lib, s = Case(rows, cols, dtype), sg.load(), torch.cuda.current_stream().cuda_stream
    ld, code = cols + pad, {"fp32": 0, "bf16": 1, "fp16": 2}[dtype]

    def buffer(t=None):
        flat = torch.full((1 + rows * ld + 16,), 7.0, dtype=DTYPES[dtype], device="cuda")
        view = flat[1:1 + rows * ld].view(rows, ld)[:, :cols]
        if t is not None:
            view.copy_(t)
        return flat, view

    (_, x), (_, dh), (_, dy), (y_all, y), (dx_all, dx) = buffer(c.x), buffer(c.dh), buffer(c.dy), buffer(), buffer()
    w, b = cuda(c.w), cuda(c.b)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    assert lib.sgemm_layer_norm_forward(rows, cols, code, x.data_ptr(), ld, w.data_ptr(), b.data_ptr(), 0, EPS,
                                        y.data_ptr(), ld, mean.data_ptr(), rstd.data_ptr(), None, None, s) == 0
    m, r, em, er = moments(c)
    near(mean, m, em, "mean")
    near(rstd, r, er * r, "rstd")
    n = (f64(c.x) - m[:, None]) * r[:, None]
    want = n * f64(c.w) + f64(c.b)
    near(y, want, (em * r)[:, None] * f64(c.w).abs() * 1.01 + (n * f64(c.w)).abs() * (er[:, None] + 4 * E24) +
         E24 * (want.abs() + f64(c.b).abs()) + c.u * want.abs() * 1.01 + 1e-7, "y")
    q = sg.act8_quantize(cuda(c.x))
    size = ctypes.c_size_t(0)
    assert lib.sgemm_layer_norm_backward_workspace(rows, cols, ctypes.byref(size)) == 0
    ws = torch.full((size.value + 256,), 9, dtype=torch.uint8, device="cuda")
    for kept in (False, True):
        dw, db = torch.full((cols,), 7.0, device="cuda"), torch.full((cols,), 7.0, device="cuda")
        of = (None, 0, q.codes.data_ptr(), q.scales.data_ptr()) if kept else (x.data_ptr(), ld, None, None)
        assert lib.sgemm_layer_norm_backward(
            rows, cols, code, dh.data_ptr(), ld, dy.data_ptr(), ld, *of, mean.data_ptr(), rstd.data_ptr(),
            w.data_ptr(), 0, dx.data_ptr(), ld, dw.data_ptr(), db.data_ptr(), ws.data_ptr(), size.value, s) == 0
        # Against the call on matrices at their groups' starts, of padded rows: the terms are the same,
        # their sums' orders are not.  c.e and c.ec bound one side's sums of magnitudes.
        width = -(-cols // 8) * 8

        def padded(t):
            return torch.zeros(rows, width, dtype=DTYPES[dtype], device="cuda")[:, :cols].copy_(t)

        ref = sg.layer_norm_backward(padded(c.dh), q if kept else padded(c.x), mean, rstd, w, dy=padded(c.dy))
        v = f64(q.dequantize()) if kept else f64(c.x)
        n, dh64 = (v - f64(mean)[:, None]) * f64(rstd)[:, None], f64(c.dh)
        g, r64 = dh64 * f64(c.w), f64(rstd)[:, None]
        ga, na = g.abs().mean(1, keepdim=True), (g * n).abs().mean(1, keepdim=True)
        off = 2 * r64 * (c.e * ga + n.abs() * c.e * na + 6 * E24 * (g.abs() + ga + n.abs() * na)) + \
            4 * E24 * f64(c.dy).abs()
        near(dx, f64(ref[0]), off + 2 * c.u * 1.01 * (f64(ref[0]).abs() + off), "dx")
        near(dw, f64(ref[1]), 2 * (c.ec + 4 * E24) * (dh64 * n).abs().sum(0) + 1e-30, "dweight")
        near(db, f64(ref[2]), 2 * (c.ec + 4 * E24) * dh64.abs().sum(0) + 1e-30, "dbias")
        assert bool((ws[size.value:] == 9).all())
    for flat, view in ((y_all, y), (dx_all, dx)):
        rest = flat.clone()
        rest[1:1 + rows * ld].view(rows, ld)[:, :cols] = 7.0
        assert bool((rest == 7.0).all())


@pytest.mark.parametrize("cols", [64, 1000, 4096, 8192, 40001])
def test_odd_numbers_stay_in_their_row(sg, cols):
    """Infinities and NaN make their own row NaN and no other; the columns' sums get them."""
    c = Case(7, cols, "fp32")
    clean = sg.layer_norm(cuda(c.x), cuda(c.w), cuda(c.b))
    x = cuda(c.x)
    x[2, cols - 1], x[5, 0] = float("inf"), float("nan")
    y, mean, rstd = sg.layer_norm(x, cuda(c.w), cuda(c.b))
    good = [0, 1, 3, 4, 6]
    for got, want in zip((y, mean, rstd), clean):
        assert torch.equal(got[good], want[good])
    assert bool(y[2].isnan().all()) and bool(y[5].isnan().all())
    dx, dw, db = sg.layer_norm_backward(cuda(c.dh), x, mean, rstd, cuda(c.w))
    ref = sg.layer_norm_backward(cuda(c.dh), cuda(c.x), clean[1], clean[2], cuda(c.w))
    assert torch.equal(dx[good], ref[0][good]) and bool(dw.isnan().all())
    assert bool(dx[2].isnan().all()) and torch.equal(db, ref[2])


def test_no_rows(sg):
    x, w = torch.empty(0, 48, device="cuda"), torch.ones(48, device="cuda")
    y, mean, rstd, kept = sg.layer_norm(x, w, w, keep="8bit")
    assert y.shape == (0, 48) and mean.shape == (0,) and kept.shape == (0, 48)
    dx, dw, db = sg.layer_norm_backward(x, kept, mean, rstd, w)
    assert dx.shape == (0, 48) and not bool(dw.any()) and not bool(db.any())


def test_long_offsets(sg):
    """More than 2^31 elements: the last rows are their own."""
    rows, cols = 300000, 8192
    c = Case(64, cols, "bf16")
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    x[-64:] = cuda(c.x)
    y, mean, rstd = sg.layer_norm(x, cuda(c.w), cuda(c.b))
    # (A call of 64 rows may sum a row in another order.)
    for got, want, rel in zip((y, mean, rstd), check_forward(sg, c), (2 * c.u, 2 * c.e, 2 * c.e)):
        assert torch.allclose(got[-64:].float(), want.float(), rtol=rel, atol=4 * c.e)
    assert torch.equal(y[0].float(), cuda(c.b).bfloat16().float())


def test_refusals(sg):
    x, w = torch.randn(8, 64, device="cuda"), torch.ones(64, device="cuda")
    y, mean, rstd = sg.layer_norm(x, w)
    for args in ((x.t(),), (x.double(),), (x.cpu(),), (x[:, ::2],), (x, w[:63]), (x, w.double()),
                 (x, w, w.bfloat16()), (x, w.cpu()), (x[:, :0],), (x[0],), (3,), (x, torch.ones(128, device="cuda")[::2])):
        with pytest.raises((TypeError, ValueError)):
            sg.layer_norm(*args)
    for kw in (dict(keep="full"), dict(keep=8)):
        with pytest.raises(ValueError):
            sg.layer_norm(x, w, **kw)
    with pytest.raises(sg.SgemmError):
        sg.layer_norm(x, w, eps=-1.0)
    q = sg.act8_quantize(x)
    for args in ((x, x[:7], mean, rstd, w), (x, x.bfloat16(), mean, rstd, w), (x, x, mean[:7], rstd, w),
                 (x, x, mean, rstd.double(), w), (x, x, mean, rstd, w[:5]), (x.t(), x, mean, rstd, w),
                 (x[:7], q, mean[:7], rstd[:7], w), (x, sg.act8_quantize(x[:, :63]), mean, rstd, w), (x, x, mean.cpu(), rstd, w), (x, None, mean, rstd, w)):
        with pytest.raises((TypeError, ValueError)):
            sg.layer_norm_backward(*args)
    with pytest.raises(ValueError):
        sg.layer_norm_backward(x, x, mean, rstd, w, dy=x[:, :63])


@pytest.mark.parametrize("cols", [64, 1000, 2047, 4096, 9000, 20001])
def test_without_sums_the_workspace_stays(sg, cols):
    """The C entry without dweight and dbias takes any workspace, of no bytes too, and leaves it."""
    import ctypes
    c, lib, s = Case(37, cols, "fp32"), sg.load(), torch.cuda.current_stream().cuda_stream
    x, dh, w = cuda(c.x), cuda(c.dh), cuda(c.w)
    _, mean, rstd = sg.layer_norm(x, w)
    want = sg.layer_norm_backward(dh, x, mean, rstd, w)[0]
    n = ctypes.c_size_t(0)
    assert lib.sgemm_layer_norm_backward_workspace(37, cols, ctypes.byref(n)) == 0
    ws = torch.full((n.value,), 9, dtype=torch.uint8, device="cuda")
    dx = torch.zeros_like(x)
    assert lib.sgemm_layer_norm_backward(
        37, cols, 0, dh.data_ptr(), cols, None, 0, x.data_ptr(), cols, None, None, mean.data_ptr(),
        rstd.data_ptr(), w.data_ptr(), 0, dx.data_ptr(), cols, None, None, ws.data_ptr(), 0, s) == 0
    torch.cuda.synchronize()
    assert torch.equal(dx, want) and bool((ws == 9).all())


@pytest.mark.parametrize("cols", [8192, 8191])
def test_gradient_of_long_offsets(sg, cols):
    """More than 2^31 elements, from a matrix and from a checkpoint: the last rows are their own."""
    rows, few = 270000, 400
    c = Case(64, cols, "bf16")
    x, dh, dy = (torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    for big, small in ((x, c.x), (dh, c.dh), (dy, c.dy)):
        big[-64:] = cuda(small)
    _, mean, rstd, kept = sg.layer_norm(x, cuda(c.w), cuda(c.b), keep="8bit")
    x_few, dh_few, dy_few = (t[-few:].clone() for t in (x, dh, dy))
    for of, rows_of in ((x, x_few), (kept, sg.act8_quantize(x_few))):
        got = sg.layer_norm_backward(dh, of, mean, rstd, cuda(c.w), dy=dy)
        want = sg.layer_norm_backward(dh_few, rows_of, mean[-few:], rstd[-few:], cuda(c.w), dy=dy_few)
        # The same kernel and the same statistics: the same rows.  The other rows' dh are 0, but sums are
        # added in another order: 64 terms of fp32, twice, of at most 64 times the largest |dh| |n|.
        assert torch.equal(got[0][-few:], want[0]) and not bool(got[0][:-64].any())
        most = 64 * float(c.dh.abs().max()) * max(1.0, float(((c.x.float() - 0.7) / 2).abs().max()) * 1.5)
        for a, b in zip(got[1:], want[1:]):
            assert bool(((a - b).abs() <= 2 * 64 * E24 * most).all())
