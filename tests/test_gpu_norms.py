"""Norms around a block and their gradients against their formulas in 64 bits.

Tolerances.  u is half an ulp of the output's type (2^-24, 2^-8, 2^-11).  A row's sum of D
terms is at most D / 128 + 32 sequential fp32 additions deep, so the sum, and with it rstd
and every mean, is off by at most e = (D / 128 + 32) 2^-24 of the sum of its terms'
magnitudes; a result is off by e times the magnitudes it is made of, and by its rounding u.
Column sums are R / 64 + 40 deep."""
import numpy as np
import pytest
import torch

import mx4_reference as ref

pytestmark = pytest.mark.gpu

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
HALF_ULP = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
EPS = 1e-5
SHAPES = [(1, 1), (1, 4096), (3, 7), (5, 64), (33, 257), (130, 1000), (2, 2048), (4, 8200),
          (2, 40001), (700, 96), (2, 70000), (330, 4096), (3, 5000), (2, 4100), (5, 12000), (2, 16384)]


@pytest.fixture()
def sg(cuda):
    import dense_fp32_gemm_09_gb300 as sg
    return sg


class Case:
    def __init__(self, rows, cols, dtype, gate, weighted=True, wdtype=torch.float32, seed=0):
        g = torch.Generator().manual_seed(rows * 7 + cols + seed)
        r = lambda *s: torch.randn(s, generator=g)
        dt = DTYPES[dtype]
        self.rows, self.cols, self.u = rows, cols, HALF_ULP[dtype]
        self.block, self.residual = (r(rows, cols) * 3).to(dt), r(rows, cols).to(dt)
        self.dy, self.dh, self.y = r(rows, cols).to(dt), r(rows, cols).to(dt), r(rows, cols).to(dt)
        self.w = (1 + 0.3 * r(cols)).to(wdtype) if weighted else None
        self.nw = (1 + 0.3 * r(cols)).to(wdtype) if weighted else None
        self.gate = None if gate == "none" else torch.sigmoid(
            r(rows, cols) if gate == "rows" else r(cols)).to(dt)
        self.scale = 0.7
        self.e = (cols / 128 + 32) * 2.0 ** -24
        self.ec = (rows / 64 + 40) * 2.0 ** -24 + self.e


def f64(t):
    return t.double().cpu()


def ones(c, w):
    return torch.ones(c.cols, dtype=torch.float64) if w is None else f64(w)


def forward(c):
    b, res = f64(c.block), f64(c.residual)
    gate = 1.0 if c.gate is None else f64(c.gate)
    r = ((b * b).mean(1) + EPS) ** -0.5
    add = c.scale * gate * b * r[:, None] * ones(c, c.w)
    y = res + add
    rn = ((y * y).mean(1) + EPS) ** -0.5
    return y, r, y * rn[:, None] * ones(c, c.nw), rn, res.abs() + add.abs()


def near(got, want, tol, what):
    got = f64(got)
    bad = (got - want).abs() - tol
    assert torch.isfinite(got).all() and bool((bad <= 0).all()), (what, float(bad.max()))


def cuda(t):
    return None if t is None else t.cuda()


@pytest.mark.parametrize("gate", ["none", "rows", "shared"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(sg, rows, cols, dtype, gate):
    c = Case(rows, cols, dtype, gate)
    y, r, h, rn, mag = forward(c)
    got = sg.norm_after(cuda(c.block), cuda(c.residual), cuda(c.w), gate=cuda(c.gate),
                        scale=c.scale, eps=EPS, next_weight=cuda(c.nw))
    # y: 8 roundings and rstd's error; h: y's error relative to u, its own and rstd's.
    ey = (c.e + 8 * 2.0 ** -24) * mag
    near(got[0], y, ey + c.u * y.abs() * 1.01 + 1e-7, "y")
    near(got[1], r, (c.e + 2.0 ** -22) * r, "rstd")
    # rn moves by at most its sum's error and the relative error of u in norm.
    shift = (ey.norm(dim=1) / y.norm(dim=1).clamp(min=1e-30)).clamp(max=1)
    ern = (c.e + 2.0 ** -22 + shift) * rn
    near(got[3], rn, ern, "next_rstd")
    w = ones(c, c.nw).abs()
    eh = (ey * rn[:, None] + y.abs() * ern[:, None]) * w + 4 * 2.0 ** -24 * h.abs()
    near(got[2], h, eh + c.u * h.abs() * 1.01 + 1e-7, "h")
    two = sg.norm_after(cuda(c.block), cuda(c.residual), cuda(c.w), gate=cuda(c.gate),
                        scale=c.scale, eps=EPS)
    assert len(two) == 2 and torch.equal(two[0], got[0]) and torch.equal(two[1], got[1])
    h1, r1 = sg.norm_before(cuda(c.block), cuda(c.w), eps=EPS)
    n = f64(c.block) * r[:, None] * ones(c, c.w)
    near(r1, r, (c.e + 2.0 ** -22) * r, "before rstd")
    near(h1, n, (c.e + 2.0 ** -21) * n.abs() + c.u * n.abs() * 1.01 + 1e-7, "before h")


def norm_grad(g, x, r):
    """Gradient of sum(g * x r(x)) over x, r the saved rstd, and its magnitude."""
    n = x * r[:, None]
    m, ma = (g * n).mean(1, keepdim=True), (g * n).abs().mean(1, keepdim=True)
    return r[:, None] * (g - n * m), r[:, None] * (g.abs() + n.abs() * ma)


def saved(c):
    r = (f64(c.block).square().mean(1) + EPS) ** -0.5
    rn = (f64(c.y).square().mean(1) + EPS) ** -0.5
    return r.float(), rn.float()


@pytest.mark.parametrize("gate", ["none", "rows", "shared"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(sg, rows, cols, dtype, gate):
    c = Case(rows, cols, dtype, gate)
    r, rn = saved(c)
    got = sg.norm_after_backward(cuda(c.dy), cuda(c.block), cuda(r), cuda(c.w), gate=cuda(c.gate),
                                 scale=c.scale, dh=cuda(c.dh), y=cuda(c.y), next_rstd=cuda(rn),
                                 next_weight=cuda(c.nw))
    e, small = c.e + 12 * 2.0 ** -24, 1e-6
    y, b, dh, w, nw = f64(c.y), f64(c.block), f64(c.dh), f64(c.w), f64(c.nw)
    gv = c.scale * (torch.ones(cols, dtype=torch.float64) if c.gate is None else f64(c.gate))
    t, tm = norm_grad(nw * dh, y, f64(rn))
    t, tm = t + f64(c.dy), tm + f64(c.dy).abs()
    near(got[0], t, e * tm + c.u * t.abs() * 1.01 + small, "dresidual")
    g, gm = gv * t, gv.abs() * tm
    db, _ = norm_grad(w * g, b, f64(r))
    _, dbm = norm_grad(w * gm, b, f64(r))
    near(got[1], db, 2 * e * dbm + c.u * db.abs() * 1.01 + small, "dblock")
    n, ec = b * f64(r)[:, None], c.ec + 24 * 2.0 ** -24
    near(got[2], (g * n).sum(0), 2 * ec * (gm * n.abs()).sum(0) + small, "dweight")
    if c.gate is not None:
        dg, dgm = c.scale * t * n * w, c.scale * tm * (n * w).abs()
        if gate == "rows":
            near(got[3], dg, 2 * e * dgm + c.u * dg.abs() * 1.01 + small, "dgate")
        else:
            near(got[3], dg.sum(0), 2 * ec * dgm.sum(0) + small, "dgate")
            assert got[3].dtype == torch.float32
    else:
        assert got[3] is None
    nn = y * f64(rn)[:, None]
    near(got[4], (dh * nn).sum(0), 2 * ec * (dh * nn).abs().sum(0) + small, "dnext_weight")
    again = sg.norm_after_backward(cuda(c.dy), cuda(c.block), cuda(r), cuda(c.w),
                                   gate=cuda(c.gate), scale=c.scale, dh=cuda(c.dh), y=cuda(c.y),
                                   next_rstd=cuda(rn), next_weight=cuda(c.nw))
    for a, z in zip(got, again):
        assert (a is None and z is None) or torch.equal(a, z)    # a fixed order of sums


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", [(1, 40), (6, 513), (140, 2048)])
def test_backward_of_each_half(sg, rows, cols, dtype):
    c = Case(rows, cols, dtype, "rows")
    r, rn = saved(c)
    e, small = c.e + 12 * 2.0 ** -24, 1e-6
    dy = cuda(c.dy)
    got = sg.norm_after_backward(dy, cuda(c.block), cuda(r), cuda(c.w), gate=cuda(c.gate),
                                 scale=c.scale)
    assert got[0] is dy and got[4] is None
    g = c.scale * f64(c.gate) * f64(c.dy)
    db, dbm = norm_grad(f64(c.w) * g, f64(c.block), f64(r))
    near(got[1], db, e * dbm + c.u * db.abs() * 1.01 + small, "dblock")
    for extra in (None, c.dy):
        dx, dw = sg.norm_before_backward(cuda(c.dh), cuda(c.y), cuda(rn), cuda(c.nw),
                                         dy=cuda(extra))
        t, tm = norm_grad(f64(c.nw) * f64(c.dh), f64(c.y), f64(rn))
        if extra is not None:
            t, tm = t + f64(extra), tm + f64(extra).abs()
        near(dx, t, e * tm + c.u * t.abs() * 1.01 + small, "dx")
        nn = f64(c.dh) * f64(c.y) * f64(rn)[:, None]
        near(dw, nn.sum(0), 2 * (c.ec + e) * nn.abs().sum(0) + small, "dw")


def test_gradient_against_differences(sg):
    """The fp32 gradient along random directions against central differences of the
    formula in 64 bits (step 1e-4: truncation below 1e-6 of the scale)."""
    c = Case(9, 130, "fp32", "rows", seed=4)
    g = torch.Generator().manual_seed(1)
    cy, ch = (torch.randn((9, 130), generator=g).double() for _ in range(2))
    y, r, h, rn, _ = forward(c)
    got = sg.norm_after_backward(cy.float().cuda(), cuda(c.block), r.float().cuda(), cuda(c.w),
                                 gate=cuda(c.gate), scale=c.scale, dh=ch.float().cuda(),
                                 y=y.float().cuda(), next_rstd=rn.float().cuda(),
                                 next_weight=cuda(c.nw))
    cy, ch = cy.float().double(), ch.float().double()
    names = ["residual", "block", "w", "gate", "nw"]
    for name, grad in zip(names, got):
        base = f64(getattr(c, name))
        v = torch.randn(base.shape, generator=g, dtype=torch.float64)
        step, val = 1e-4, []
        for sign in (1, -1):
            setattr(c, name, base + sign * step * v)
            out = forward(c)
            val.append(float((cy * out[0]).sum() + (ch * out[2]).sum()))
        setattr(c, name, base.float())
        diff = (val[0] - val[1]) / (2 * step)
        mine = float((f64(grad) * v).sum())
        assert abs(diff - mine) <= 2e-5 * (f64(grad) * v).abs().sum(), (name, diff, mine)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", [(1, 4096), (3, 17), (130, 200), (5, 1056), (2, 9000), (2, 70000), (3, 9001), (3, 2056), (400, 512)])
def test_quantized_output(sg, rows, cols, dtype, fmt):
    """Numbers whose 64-bit quotient is not within 1e-4 of a rounding boundary have the
    reference's value; near one either neighbour is right."""
    c = Case(rows, cols, dtype, "shared")
    ts = 0.03 if fmt == "nvfp4" else None
    t = None if ts is None else torch.tensor([ts], device="cuda")
    y, r, h, rn, _ = forward(c)
    got = sg.norm_after(cuda(c.block), cuda(c.residual), cuda(c.w), gate=cuda(c.gate),
                        scale=c.scale, eps=EPS, next_weight=cuda(c.nw), quantize=fmt,
                        tensor_scale=t)
    plain = sg.norm_after(cuda(c.block), cuda(c.residual), cuda(c.w), gate=cuda(c.gate),
                          scale=c.scale, eps=EPS, next_weight=cuda(c.nw))
    for i in (0, 1, 3):
        assert torch.equal(got[i], plain[i])
    lo, hi = ((h * (1 + s * 1e-5)).float().numpy() for s in (-1, 1))
    v = [ref.values(*ref.quantize(x, fmt, ts), fmt, cols, ts) for x in (lo, hi)]
    q = got[2].dequantize().double().cpu().numpy()
    low, high = np.minimum(*v), np.maximum(*v)
    slack = 1e-6 * np.abs(high) + 1e-30
    assert ((q >= low - slack) & (q <= high + slack)).all()
    assert (low == high).mean() > 0.9 or cols < 100
    # Padded columns are zero.
    pad = got[2].codes.transpose(1, 2).reshape(-1, got[2].codes.shape[1] * 16)[:rows]
    assert not bool(pad[:, (cols + 1) // 2:].any())
    hb, rb = sg.norm_before(cuda(c.block), cuda(c.w), eps=EPS, quantize=fmt)
    assert hb.shape == (rows, cols) and rb.shape == (rows,)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols,pad", [(400, 512, 0), (700, 96, 0), (333, 4096, 8), (5, 16384, 0),
                                           (3, 8200, 0), (400, 264, 16), (1, 4096, 0), (400, 520, 1)])
def test_before_quantized(sg, rows, cols, pad, dtype, fmt):
    """Codes and scales against the 64-bit norm; the statistics' fp32 rounding may move a number
    by 1e-5 of itself, and with it to the next code where it was that near a boundary.  A
    row of zeros, one with an infinity and one with a NaN among the rows."""
    g = torch.Generator().manual_seed(rows + cols)
    x = (torch.randn(rows, cols + pad, generator=g) * 3).to(DTYPES[dtype])[:, :cols]
    w = torch.randn(cols, generator=g)
    bad = rows > 8
    if bad:
        x[2] = 0
        x[4, cols // 2] = float("inf")
        x[6, cols - 1] = float("nan")
    ts = 0.03 if fmt == "nvfp4" else None
    t = None if ts is None else torch.tensor([ts], device="cuda")
    dev = torch.empty(rows, cols + pad, dtype=DTYPES[dtype], device="cuda")[:, :cols]
    dev.copy_(x)
    q, r = sg.norm_before(dev, w.cuda(), eps=EPS, quantize=fmt, tensor_scale=t)
    keep = [i for i in range(rows) if not (bad and i in (4, 6))]
    x64 = x.double()
    r64 = 1 / torch.sqrt((x64 * x64).mean(1) + EPS)
    assert torch.allclose(r.cpu().double()[keep], r64[keep], rtol=1e-5, atol=0)
    h = (x64 * r64[:, None] * w.double())[keep]
    lo, hi = ((h * (1 + s * 1e-5)).float().numpy() for s in (-1, 1))
    v = [ref.values(*ref.quantize(a, fmt, ts), fmt, cols, ts) for a in (lo, hi)]
    got = q.dequantize().double().cpu()
    low, high = np.minimum(*v), np.maximum(*v)
    slack = 1e-6 * np.abs(high) + 1e-30
    mine = got[keep].numpy()
    assert ((mine >= low - slack) & (mine <= high + slack)).all()
    assert (low == high).mean() > 0.9
    codes = q.codes.transpose(1, 2).reshape(-1, q.codes.shape[1] * 16)[:rows]
    assert not bool(codes[keep][:, cols // 2:].any())
    if bad:
        assert got[6].isnan().all() and not got[2].any()
        # inf * (1 / inf): its own block is NaN, the others are 0.
        block = 16 if fmt == "nvfp4" else 32
        at = cols // 2 // block * block
        assert got[4, at:at + block].isnan().all()
        rest = torch.cat([got[4, :at], got[4, at + block:]])
        assert not rest.any()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("cols", [8, 24, 264, 520, 4104])
def test_before_quantized_padding(sg, cols, dtype, fmt):
    """Codes and scales past the row's end are zeros, whatever the row holds; with no eps a row of
    zeros has an infinite statistic, and is NaN."""
    rows = 400
    x = torch.randn(rows, cols, generator=torch.Generator().manual_seed(cols)).to(DTYPES[dtype])
    x[1], x[3, 0], x[5, cols - 1] = 0, float("nan"), float("inf")
    q, r = sg.norm_before(x.cuda(), eps=0.0, quantize=fmt)
    assert torch.isinf(r[1])
    v = q.dequantize()
    assert v[1].isnan().all() and v[3].isnan().all() and v[5, cols - 1].isnan()
    assert not v[[0, 2, 4]].isnan().any()
    codes = q.codes.transpose(1, 2).reshape(-1, q.codes.shape[1] * 16)[:rows]
    assert not bool(codes[:, cols // 2:].any())
    block = 16 if fmt == "nvfp4" else 32
    # [rows/128][blocks/4][row % 32][row / 32 % 4][4]
    s = q.scales.reshape(q.codes.shape[0], -1, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(
        q.codes.shape[0] * 128, -1)[:rows]
    assert not bool(s[:, -(-cols // block):].any())


@pytest.mark.parametrize("wdtype", ["fp32", "same", "none"])
def test_weight_types(sg, wdtype):
    wd = torch.float32 if wdtype == "fp32" else torch.bfloat16
    c = Case(20, 384, "bf16", "none", weighted=wdtype != "none", wdtype=wd)
    y, r, h, rn, mag = forward(c)
    out = sg.norm_after(cuda(c.block), cuda(c.residual), cuda(c.w), scale=c.scale, eps=EPS,
                        next_norm=True, next_weight=cuda(c.nw))
    near(out[0], y, c.e * 4 * mag + c.u * y.abs() * 1.01 + 1e-7, "y")
    near(out[2], h, c.e * 8 * (h.abs() + mag * rn[:, None] * 2) + c.u * h.abs() * 1.01 + 1e-7, "h")
    rs, rns = saved(c)
    got = sg.norm_after_backward(cuda(c.dy), cuda(c.block), cuda(rs), cuda(c.w), scale=c.scale,
                                 dh=cuda(c.dh), y=cuda(c.y), next_rstd=cuda(rns),
                                 next_weight=cuda(c.nw))
    assert (got[2] is None) == (wdtype == "none") and (got[4] is None) == (wdtype == "none")
    t, tm = norm_grad(ones(c, c.nw) * f64(c.dh), f64(c.y), f64(rns))
    near(got[0], t + f64(c.dy), 2 * c.e * (tm + f64(c.dy).abs()) + c.u * (t + f64(c.dy)).abs() * 1.01
         + 1e-6, "dresidual")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("off,pad", [(0, 8), (1, 0), (3, 5), (8, 24)])
def test_strides_and_alignment(sg, dtype, off, pad):
    """Views of any offset and row stride give what contiguous tensors give, up to the
    order of the sums, and leave what is around them."""
    c = Case(37, 520, dtype, "rows")
    r, rn = saved(c)

    def view(t):
        t = t.cuda()
        buf = torch.full((off + t.shape[0] * (t.shape[1] + pad),), 3.0, dtype=t.dtype, device="cuda")
        v = buf[off:].view(t.shape[0], -1)[:, :t.shape[1]]
        v.copy_(t)
        return v
    outs = []
    for f in (cuda, view):
        a = sg.norm_after(f(c.block), f(c.residual), cuda(c.w), gate=f(c.gate), scale=c.scale,
                          eps=EPS, next_weight=cuda(c.nw))
        b = sg.norm_after_backward(f(c.dy), f(c.block), cuda(r), cuda(c.w), gate=f(c.gate),
                                   scale=c.scale, dh=f(c.dh), y=f(c.y), next_rstd=cuda(rn),
                                   next_weight=cuda(c.nw))
        outs.append(a + b)
    for x, z in zip(*outs):
        tol = 2 * c.u + 64 * 2.0 ** -24
        assert torch.allclose(x.double(), z.double(), rtol=tol, atol=tol * 4)


def test_empty_rows_and_zero_rows(sg):
    z = torch.zeros((0, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    h, r = sg.norm_before(z, w)
    assert h.shape == (0, 64) and r.shape == (0,)
    _, db, dw, dg, dn = sg.norm_after_backward(z, z, r, w, gate=w, dh=z, y=z, next_rstd=r,
                                               next_weight=w)
    assert not bool(dw.any()) and not bool(dg.any()) and not bool(dn.any()) and db.shape == (0, 64)
    x = torch.zeros((3, 64), device="cuda")
    h, r = sg.norm_before(x, w, eps=1e-6)
    assert not bool(h.any()) and torch.allclose(r, torch.full_like(r, 1e3))


def test_not_a_number_stays_in_its_row(sg):
    x = torch.randn((6, 300), device="cuda")
    x[2, 17], x[4, 200] = float("nan"), float("inf")
    y, r, h, rn = sg.norm_after(x, torch.zeros_like(x), next_norm=True)
    ok = torch.tensor([0, 1, 3, 5])
    assert bool(torch.isfinite(h[ok]).all()) and bool(torch.isnan(h[2]).all())
    assert bool(torch.isnan(h[4, 200]))
    q, _ = sg.norm_before(x, quantize="nvfp4")
    v = q.dequantize()
    assert bool(torch.isfinite(v[ok]).all()) and bool(torch.isnan(v[2]).all())


def test_other_stream_and_graph(sg):
    c = Case(50, 1024, "bf16", "shared")
    r, rn = saved(c)
    ins = [cuda(v) for v in (c.dy, c.block, r, c.w, c.gate, c.dh, c.y, rn, c.nw)]

    def call(stream=None):
        dy, b, r_, w, gate, dh, y, rn_, nw = ins
        f = sg.norm_after(b, y, w, gate=gate, next_weight=nw, stream=stream)
        return f + sg.norm_after_backward(dy, b, r_, w, gate=gate, dh=dh, y=y, next_rstd=rn_,
                                          next_weight=nw, stream=stream)
    want = call()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = call(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(s):
        call()                     # the stream's workspace exists before the capture
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = call()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_refusals(sg):
    x = torch.randn((4, 32), device="cuda")
    w = torch.ones(32, device="cuda")
    with pytest.raises(ValueError, match="no columns"):
        sg.norm_before(x[:, :0])
    with pytest.raises(TypeError):
        sg.norm_before(x.double())
    with pytest.raises(ValueError, match="shape"):
        sg.norm_before(x, w[:31])
    with pytest.raises(TypeError, match="weight"):
        sg.norm_before(x, w.half())
    with pytest.raises(ValueError, match="fmt"):
        sg.norm_before(x, w, quantize="int4")
    with pytest.raises(ValueError, match="tensor_scale"):
        sg.norm_before(x, w, tensor_scale=torch.ones(1, device="cuda"))
    with pytest.raises(sg.SgemmError, match="eps"):
        sg.norm_before(x, w, eps=-1.0)
    with pytest.raises(sg.SgemmError, match="eps"):
        sg.norm_before(x, w, eps=float("nan"))
    with pytest.raises(ValueError, match="block"):
        sg.norm_after(x[:3], x, w)
    with pytest.raises(TypeError, match="block"):
        sg.norm_after(x.half(), x, w)
    with pytest.raises(ValueError, match="gate"):
        sg.norm_after(x, x, w, gate=x[:, :31])
    with pytest.raises(sg.SgemmError, match="scale"):
        sg.norm_after(x, x, w, scale=float("inf"))
    with pytest.raises(ValueError, match="next"):
        sg.norm_after(x, x, w, next_norm=False, quantize="nvfp4")
    with pytest.raises(ValueError, match="dh"):
        sg.norm_after_backward(x, x, w[:4], w, y=x)
    with pytest.raises(ValueError, match="rstd"):
        sg.norm_after_backward(x, x, w, w)
    with pytest.raises(ValueError, match="overlap"):
        sg.norm_after_backward(x[:1].expand(4, 32), x, w[:4])


@pytest.mark.parametrize("gate", ["none", "rows", "shared"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", [(3, 16392), (160, 20000), (2, 20001), (4, 32768), (2, 32770)])
def test_forward_of_wide_rows(sg, rows, cols, dtype, gate):
    test_forward(sg, rows, cols, dtype, gate)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", [(3, 16392), (2, 20001), (2, 32768)])
def test_quantized_output_of_wide_rows(sg, rows, cols, dtype, fmt):
    test_quantized_output(sg, rows, cols, dtype, fmt)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", [(3, 16392), (2, 32768), (320, 20000)])
def test_before_quantized_of_wide_rows(sg, rows, cols, dtype, fmt):
    test_before_quantized(sg, rows, cols, 0, dtype, fmt)
