"""Norm gradients of rows whose statistic is large, in each kernel that takes them: all of the
formula's numbers fit the type, so all of the result's have to.  Tolerances as in
test_gpu_norms.py."""
import pytest
import torch

from test_gpu_norms import Case, cuda, f64, near, norm_grad, sg  # noqa: F401  (sg: fixture)

pytestmark = pytest.mark.gpu

# Registers (aligned, odd), ring, streaming.
SHAPES = [(5, 512), (33, 257), (4, 5000), (3, 9000), (2, 40001)]


def tiny(c, name):
    """The case's rows `name` at 1e-20 of their size, and their statistic without eps."""
    t = (getattr(c, name).double() * 1e-20).to(getattr(c, name).dtype)
    setattr(c, name, t)
    return (t.double().square().mean(1) ** -0.5).float()


@pytest.mark.parametrize("dy", [True, False])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_before(sg, rows, cols, dtype, dy):  # noqa: F811
    c = Case(rows, cols, dtype, "none")
    rn = tiny(c, "y")
    dx, dw = sg.norm_before_backward(cuda(c.dh), cuda(c.y), cuda(rn), cuda(c.nw),
                                     dy=cuda(c.dy) if dy else None)
    e = c.e + 12 * 2.0 ** -24
    t, tm = norm_grad(f64(c.nw) * f64(c.dh), f64(c.y), f64(rn))
    if dy:
        t, tm = t + f64(c.dy), tm + f64(c.dy).abs()
    near(dx, t, e * tm + c.u * t.abs() * 1.01 + 1e-6, "dx")
    nn = f64(c.dh) * f64(c.y) * f64(rn)[:, None]
    near(dw, nn.sum(0), 2 * (c.ec + e) * nn.abs().sum(0) + 1e-6, "dw")


@pytest.mark.parametrize("gate", ["none", "rows", "shared"])
@pytest.mark.parametrize("both", [True, False])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_after(sg, rows, cols, dtype, both, gate):  # noqa: F811
    c = Case(rows, cols, dtype, gate)
    r = tiny(c, "block")
    rn = (f64(c.y).square().mean(1) ** -0.5).float()
    more = dict(dh=cuda(c.dh), y=cuda(c.y), next_rstd=cuda(rn), next_weight=cuda(c.nw))
    got = sg.norm_after_backward(cuda(c.dy), cuda(c.block), cuda(r), cuda(c.w), gate=cuda(c.gate),
                                 scale=c.scale, **(more if both else {}))
    e = c.e + 12 * 2.0 ** -24
    t, tm = f64(c.dy), f64(c.dy).abs()
    if both:
        d, dm = norm_grad(f64(c.nw) * f64(c.dh), f64(c.y), f64(rn))
        t, tm = t + d, tm + dm
    g = c.scale * (torch.ones(cols, dtype=torch.float64) if c.gate is None else f64(c.gate))
    db, _ = norm_grad(f64(c.w) * g * t, f64(c.block), f64(r))
    _, dbm = norm_grad(f64(c.w) * g.abs() * tm, f64(c.block), f64(r))
    near(got[1], db, 2 * e * dbm + c.u * db.abs() * 1.01 + 1e-6, "dblock")
    n = f64(c.block) * f64(r)[:, None]
    near(got[2], (g * t * n).sum(0), 2 * (c.ec + 24 * 2.0 ** -24) * (g.abs() * tm * n.abs()).sum(0) + 1e-6,
         "dweight")


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("after", [True, False])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("rows,cols", [(7, 77), (400, 264), (7, 8201), (7, 9001), (7, 9005),
                                       (7, 16383), (7, 20001)])
def test_padding_of_rows_that_are_not_numbers(sg, rows, cols, dtype, after, fmt):  # noqa: F811
    """Codes and scales past the row's end are zeros, whatever the row holds."""
    x = Case(rows, cols, dtype, "none").block
    x[1], x[3, 0], x[5, cols - 1] = 0, float("nan"), float("inf")
    if after:
        q = sg.norm_after(torch.ones_like(x).cuda(), x.cuda(), scale=0.0, eps=0.0, quantize=fmt)[2]
    else:
        q, _ = sg.norm_before(x.cuda(), eps=0.0, quantize=fmt)
    byte = q.codes.transpose(1, 2).reshape(-1, q.codes.shape[1] * 16)[:rows]
    code = torch.stack((byte & 15, byte >> 4), 2).view(rows, -1)
    assert not bool(code[:, cols:].any())
    s = q.scales.permute(0, 3, 2, 1, 4).reshape(-1, q.scales.shape[1] * 4)[:rows]
    assert not bool(s[:, -(-cols // (16 if fmt == "nvfp4" else 32)):].any())
    v = q.dequantize()
    assert bool(v[3].isnan().all()) and not bool(v[[0, 2, 4]].isnan().any())
