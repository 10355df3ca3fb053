"""The gated feed-forward block where a gate is far from zero: its activation and slope against
the formula in 64 bits, up to the largest numbers of the type.

Tolerances.  u is half a step of the type (2^-8, 2^-11).  CUDA's bound for the fast exponential of
-z is 2 + 1.173 |z| steps (2^-23 of it), z itself is off by up to 2^-22 of its size (three roundings
and two constants), which the exponential multiplies by z; a reciprocal and four products add less
than 2^-20.  An exponential below 2^-126 is off by 2^-149 at most beside that."""
import pytest
import torch

from test_gpu_gated_ff import DTYPES, U

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


# z = -76 to -98 (gelu: g = -9.5 to -10.3), where e^-z passes 2^126 and then the largest fp32 number.
FAR = {"silu": [-80.0, -86.0, -87.0, -87.5, -88.0, -89.0, -90.0, -92.0, -94.0, -98.0],
       "gelu_tanh": [-9.5, -9.75, -9.875, -9.9375, -10.0, -10.0625, -10.125, -10.1875, -10.25, -10.3125]}


UP, DH = 2.0 ** 110, 2.0 ** 12      # (their product, and act(g) times either, are ordinary fp32 numbers)


def argument(g, name):
    """z and its slope."""
    if name == "silu":
        return g, torch.ones_like(g)
    k = 2 * (2 / torch.pi) ** 0.5
    return k * (g + 0.044715 * g ** 3), k * (1 + 3 * 0.044715 * g * g)


def activation(g, name):
    """(act, act') in 64 bits, through the sigmoid: 1 + tanh is 0 in 64 bits from z = -37 down."""
    z, by = argument(g, name)
    s = torch.sigmoid(z)
    return g * s, s * (1 + g * by * torch.sigmoid(-z))


def exponential_off(g, name):
    """How far s may be off, beside its size and by itself."""
    z = argument(g, name)[0]
    return (3 + 1.173 * z.abs() + 2 * z.abs()) * 2.0 ** -23 + 2.0 ** -20, 2.0 ** -149


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("tokens", [10, 40])       # the kernel of few tokens, and tiles
def test_small_activations_times_large_numbers(sg, name, tokens):
    """bf16: act(g) near the smallest numbers, times an up projection near the largest."""
    gates = FAR[name]
    n = len(gates)
    g = torch.tensor(gates, device="cuda").double()
    x = own(n, "bf16").repeat(-(-tokens // n), 1)[:tokens]
    wg = g.bfloat16().repeat(n, 1).t().contiguous()
    wu = torch.full_like(wg, UP)
    assert torch.equal(wg[:, 0].double(), g)
    want = (activation(g, name)[0] * UP).expand(tokens, n)
    rel, small = exponential_off(g, name)
    tol = (want.abs() * (rel + U["bf16"] * (1 + rel)) + g.abs() * small * UP * 1.01).expand(tokens, n)
    for keep in (None, "full", "8bit"):
        h = sg.gated_ff(x, wg, wu, activation=name, keep=keep)
        if keep is not None:
            h, kept = h
        assert bool(((h.double() - want).abs() <= tol).all()), keep
    # The gradient of what was kept in full: each number of dw is one product.
    kept = (wg.t()[:1].contiguous(), wu.t()[:1].contiguous())
    one, eye = torch.ones(1, n, dtype=torch.bfloat16, device="cuda"), own(n, "bf16")
    _, dwg, dwu, h = sg.gated_ff_backward(one * DH, one, eye, eye, kept, activation=name, return_h=True)
    assert bool(((h.double() - want[:1]).abs() <= tol[:1]).all())
    # dg = dh u slope and du = dh act(g): two roundings of half a step (of each, and of its sum).
    a, slope = activation(g, name)
    far = g.abs() * 200 * small * UP * DH           # (the slope is s (1 + up to 200 |g|))
    want = (slope * UP * DH)[:, None]
    assert bool(((dwg.double() - want).abs() <= want.abs() * (rel[:, None] + 2.01 * U["bf16"]) + far[:, None]).all())
    want, far = (a * DH)[:, None], g.abs() * small * DH * 1.01
    assert bool(((dwu.double() - want).abs() <= want.abs() * (rel[:, None] + 2.01 * U["bf16"]) + far[:, None]).all())
