"""Each half of the norms on its own in each kernel that the choice by width and alignment
has for it: registers, ring, streaming.  Tolerances as in test_gpu_norms.py."""
import numpy as np
import pytest
import torch

import mx4_reference as ref
from test_gpu_norms import (DTYPES, EPS, Case, cuda, f64, forward, near, norm_grad, ones, saved,  # noqa: F401
                            sg)

pytestmark = pytest.mark.gpu

# Registers up to 4096 columns (fp32, odd) or 8192; then the ring while a row fits it, with one
# stage or more; then streaming.
SHAPES = [(5, 5000), (400, 9000), (2, 9001), (330, 16384), (2, 12288), (160, 8196), (2, 40001)]


@pytest.mark.parametrize("gate", ["none", "rows", "shared"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_gradient_of_the_norm_after_alone(sg, rows, cols, dtype, gate):  # noqa: F811
    c = Case(rows, cols, dtype, gate)
    r, _ = saved(c)
    e, small = c.e + 12 * 2.0 ** -24, 1e-6
    dy = cuda(c.dy)
    args = (dy, cuda(c.block), cuda(r), cuda(c.w))
    got = sg.norm_after_backward(*args, gate=cuda(c.gate), scale=c.scale)
    assert got[0] is dy and got[4] is None
    t, n, w = f64(c.dy), f64(c.block) * f64(r)[:, None], f64(c.w)
    gv = c.scale * (torch.ones(cols, dtype=torch.float64) if c.gate is None else f64(c.gate))
    db, dbm = norm_grad(w * gv * t, f64(c.block), f64(r))
    near(got[1], db, 2 * e * dbm + c.u * db.abs() * 1.01 + small, "dblock")
    ec = c.ec + 24 * 2.0 ** -24
    near(got[2], (gv * t * n).sum(0), 2 * ec * (gv * t * n).abs().sum(0) + small, "dweight")
    dg = c.scale * t * n * w
    if gate == "rows":
        near(got[3], dg, 2 * e * dg.abs() + c.u * dg.abs() * 1.01 + small, "dgate")
    elif gate == "shared":
        near(got[3], dg.sum(0), 2 * ec * dg.abs().sum(0) + small, "dgate")
    again = sg.norm_after_backward(*args, gate=cuda(c.gate), scale=c.scale)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dy", [True, False])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_gradient_of_the_norm_before_alone(sg, rows, cols, dtype, dy, weighted):  # noqa: F811
    c = Case(rows, cols, dtype, "none", weighted=weighted)
    _, rn = saved(c)
    e, small = c.e + 12 * 2.0 ** -24, 1e-6
    dx, dw = sg.norm_before_backward(cuda(c.dh), cuda(c.y), cuda(rn), cuda(c.nw),
                                     dy=cuda(c.dy) if dy else None)
    t, tm = norm_grad(ones(c, c.nw) * f64(c.dh), f64(c.y), f64(rn))
    if dy:
        t, tm = t + f64(c.dy), tm + f64(c.dy).abs()
    near(dx, t, e * tm + c.u * t.abs() * 1.01 + small, "dx")
    if weighted:
        nn = f64(c.dh) * f64(c.y) * f64(rn)[:, None]
        near(dw, nn.sum(0), 2 * (c.ec + e) * nn.abs().sum(0) + small, "dw")
    else:
        assert dw is None


@pytest.mark.parametrize("gate", ["none", "rows", "shared"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", [(7, 513), (400, 520)] + SHAPES)
def test_norm_after_alone(sg, rows, cols, dtype, gate):  # noqa: F811
    c = Case(rows, cols, dtype, gate)
    y, r, _, _, mag = forward(c)
    got = sg.norm_after(cuda(c.block), cuda(c.residual), cuda(c.w), gate=cuda(c.gate),
                        scale=c.scale, eps=EPS)
    assert len(got) == 2
    near(got[0], y, (c.e + 8 * 2.0 ** -24) * mag + c.u * y.abs() * 1.01 + 1e-7, "y")
    near(got[1], r, (c.e + 2.0 ** -22) * r, "rstd")


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("rows,cols", [(1, 4096), (3, 17), (130, 200), (2, 9000), (3, 9001), (2, 70000)])
def test_values_of_the_quantised_norm_before(sg, rows, cols, dtype, fmt):  # noqa: F811
    """Numbers whose 64-bit quotient is not within 1e-5 of a rounding boundary have the
    reference's value; near one either neighbour is right."""
    c = Case(rows, cols, dtype, "none")
    ts = 0.03 if fmt == "nvfp4" else None
    t = None if ts is None else torch.tensor([ts], device="cuda")
    q, r = sg.norm_before(cuda(c.block), cuda(c.w), eps=EPS, quantize=fmt, tensor_scale=t)
    r64 = (f64(c.block).square().mean(1) + EPS) ** -0.5
    near(r, r64, (c.e + 2.0 ** -22) * r64, "rstd")
    h = f64(c.block) * r64[:, None] * ones(c, c.w)
    lo, hi = ((h * (1 + s * 1e-5)).float().numpy() for s in (-1, 1))
    v = [ref.values(*ref.quantize(x, fmt, ts), fmt, cols, ts) for x in (lo, hi)]
    got = q.dequantize().double().cpu().numpy()
    low, high = np.minimum(*v), np.maximum(*v)
    slack = 1e-6 * np.abs(high) + 1e-30
    assert ((got >= low - slack) & (got <= high + slack)).all()
    assert (low == high).mean() > 0.9 or cols < 100
