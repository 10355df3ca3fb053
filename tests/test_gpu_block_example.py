"""The gated residual block of examples/: its passes against the same block in 64 bits
with the quantised numbers put in by hand."""
import importlib.util
import os

import pytest
import torch

from conftest import REPO

pytestmark = pytest.mark.gpu


@pytest.fixture()
def example(cuda):
    path = os.path.join(REPO, "examples", "gated_residual_block.py")
    spec = importlib.util.spec_from_file_location("gated_residual_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("tokens,width,inner", [(1, 256, 512), (300, 384, 640), (513, 1000, 1025)])
def test_block(example, tokens, width, inner, fmt):
    """Every bf16 result is off by its rounding (2^-9 on average over a tensor, u = 2^-8 at
    most), taken through at most four passes: 4 u = 2^-6 in norm."""
    block = example.Block(width, inner, fmt, seed=width)
    g = torch.Generator("cuda").manual_seed(tokens)
    x, dy, dh = (torch.randn((tokens, width), generator=g, device="cuda").bfloat16()
                 for _ in range(3))
    y, h_next, saved = block.forward(x)
    dx, grads = block.backward(dy, dh, saved)
    _, h, rstd, a, b, rstd_b, _, rstd_y = saved

    def q(t):
        return example.quantize(t, fmt).dequantize().double()
    h64 = h.dequantize().double()
    n = x.double() * (x.double().square().mean(1, keepdim=True) + 1e-6).rsqrt()
    assert rel(h64, n * block.w_before.double()) < 0.2          # what four bits leave
    up, down = (m.forward_weight.dequantize().double() for m in (block.up, block.down))
    assert rel(a, h64 @ up.t()) < 2 ** -6
    assert rel(b, q(a) @ down.t()) < 2 ** -6
    nb = b.double() * (b.double().square().mean(1, keepdim=True) + 1e-6).rsqrt()
    want = x.double() + block.scale * block.gate.double() * nb * block.w_after.double()
    assert rel(y, want) < 2 ** -6
    ny = want * (want.square().mean(1, keepdim=True) + 1e-6).rsqrt()
    assert rel(h_next, ny * block.w_next.double()) < 2 ** -6
    # Gradients: the norms by differentiating them in 64 bits, the products as they are.
    leaf = lambda t: t.detach().double().requires_grad_()
    bb, xx, gate, wa, wn = map(leaf, (b, x, block.gate, block.w_after, block.w_next))
    yy = xx + block.scale * gate * bb * (bb.square().mean(1, keepdim=True) + 1e-6).rsqrt() * wa
    hh = yy * (yy.square().mean(1, keepdim=True) + 1e-6).rsqrt() * wn
    (yy * dy.double()).sum().add((hh * dh.double()).sum()).backward()
    for name, want in (("gate", gate.grad), ("w_after", wa.grad), ("w_next", wn.grad)):
        assert rel(grads[name], want) < 2 ** -6, name
    db = bb.grad.bfloat16()
    back_down, back_up = (m.backward_weight.dequantize().double() for m in (block.down, block.up))
    da = q(db) @ back_down.t()
    # Numbers within rounding of a 4-bit boundary may fall to either side of it: a step of
    # half the value at worst for some 2^-8 of them.
    loose = 2 ** -6 + 2 ** -4
    assert rel(grads["down"], q(db.t()) @ q(a.t()).t()) < loose
    dh_up = q(da.bfloat16()) @ back_up.t()
    assert rel(grads["up"], q(da.bfloat16().t()) @ q(h64.bfloat16().t()).t()) < 2 * loose
    xl, wb = leaf(x), leaf(block.w_before)
    ((xl * (xl.square().mean(1, keepdim=True) + 1e-6).rsqrt() * wb) * dh_up).sum().backward()
    assert rel(dx, xx.grad + xl.grad) < 2 * loose
    assert rel(grads["w_before"], wb.grad) < 2 * loose


def test_runs_as_a_command(example, capsys):
    example.main(["--tokens", "64", "--width", "256", "--inner", "512", "--steps", "1"])
    assert "us a step" in capsys.readouterr().out
