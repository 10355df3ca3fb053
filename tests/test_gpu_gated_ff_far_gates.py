"""The gated feed-forward block where a gate is far from zero: its activation and slope, up to the
largest numbers of the type."""
import pytest
import torch

from test_gpu_gated_ff import DTYPES

pytestmark = pytest.mark.gpu


@pytest.fixture()
def sg(cuda):
    import dense_fp32_gemm_09_gb300 as sg
    return sg


def own(rows, dtype):
    """One token a row, one input a token."""
    return torch.eye(rows, dtype=DTYPES[dtype], device="cuda")


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_slopes_of_the_largest_gates(sg, dtype, name):
    """act' is 0 or 1 to the last bit there, so each gradient is 0 or the number it goes by."""
    dt = DTYPES[dtype]
    top = torch.finfo(dt).max
    sizes = [s for s in (31.0, 200.0, 6e4, 1e19, 1e30, 1e36, 1.7e36, 1.8e36, 1e37, 1e38, top) if s <= top]
    g = torch.tensor([[-s for s in sizes] + sizes], device="cuda").to(dt)
    u, n = torch.ones_like(g), g.shape[1]
    slope = (g > 0).to(dt)
    eye, x = own(n, dtype), torch.ones(1, n, dtype=dt, device="cuda")
    zero = torch.zeros_like(eye)
    dx, dwg, dwu, h = sg.gated_ff_backward(u, x, eye, zero, (g, u), activation=name, return_h=True)
    assert torch.allclose(dx, slope, rtol=0, atol=1e-11)
    assert torch.allclose(dwg, slope.t().expand(n, n), rtol=0, atol=1e-11)
    value = torch.where(g > 0, g, torch.zeros_like(g))
    assert torch.allclose(h, value, rtol=0, atol=1e-11)
    assert torch.allclose(dwu, value.t().expand(n, n), rtol=0, atol=1e-11)


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_nan_gates(sg, dtype, name):
    """A NaN of what was kept reaches h, its token's dx and its output's rows of the weights'
    gradients, and nothing else."""
    n = 8
    g = torch.linspace(-4, 4, n * n, device="cuda").view(n, n).to(DTYPES[dtype])
    u, x, eye = torch.ones_like(g), torch.ones_like(g), own(n, dtype)
    want = sg.gated_ff_backward(u, x, eye, eye, (g, u), activation=name, return_h=True)
    bad = g.clone()
    bad[2, 5] = float("nan")
    dx, dwg, dwu, h = sg.gated_ff_backward(u, x, eye, eye, (bad, u), activation=name, return_h=True)
    assert bool(dx[2].isnan().all()) and bool(h[2, 5].isnan())
    assert bool(dwg[5].isnan().all()) and bool(dwu[5].isnan().all())
    others = [i for i in range(n) if i != 2]
    assert torch.equal(dx[others], want[0][others]) and torch.equal(h[others], want[3][others])
    others = [i for i in range(n) if i != 5]
    assert torch.equal(dwg[others], want[1][others]) and torch.equal(dwu[others], want[2][others])
    assert torch.equal(h[:, others], want[3][:, others])
