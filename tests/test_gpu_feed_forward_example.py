"""The feed-forward block of examples/: its passes against the same block in 64 bits with the kept
and quantised numbers put in by hand."""
import importlib.util
import os

import pytest
import torch

from conftest import REPO

pytestmark = pytest.mark.gpu


@pytest.fixture()
def example(cuda):
    path = os.path.join(REPO, "examples", "feed_forward_block.py")
    spec = importlib.util.spec_from_file_location("feed_forward_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


def act(g, name):
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c = (2 / torch.pi) ** 0.5
    th = torch.tanh(c * (g + 0.044715 * g ** 3))
    return g / 2 * (1 + th), (1 + th) / 2 + g / 2 * (1 - th * th) * c * (1 + 3 * 0.044715 * g * g)


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("tokens,width,inner", [(1, 256, 512), (300, 384, 640), (513, 1000, 1025)])
def test_block(example, tokens, width, inner, name):
    """Every bf16 result is off by its rounding (u = 2^-8 at most), taken through at most four
    of them: 4 u = 2^-6 in norm."""
    from gated_residual_block import quantize
    block = example.Block(width, inner, name, seed=width)
    g = torch.Generator("cuda").manual_seed(tokens)
    x, dy = (torch.randn((tokens, width), generator=g, device="cuda").bfloat16() for _ in range(2))
    y, saved = block.forward(x)
    dx, grads = block.backward(dy, saved)
    kept_x, mean, rstd, kept_n, (kept_g, kept_u) = saved
    q = lambda t: quantize(t, "nvfp4").dequantize().double()
    u = 2.0 ** -6

    # Forward, up to what is kept, and from there on.
    x64 = x.double()
    n = (x64 - x64.mean(1, keepdim=True)) * (x64.var(1, unbiased=False, keepdim=True) + 1e-5) ** -0.5
    n = n * block.w.double() + block.b.double()
    assert rel(kept_x.dequantize(), x64) < 2.0 ** -6 and rel(kept_n.dequantize(), n) < 2.0 ** -6
    pre = [n @ w.double().t() for w in (block.w_gate, block.w_up)]
    gate, up = kept_g.dequantize().double(), kept_u.dequantize().double()
    # Half a step of a 127th of a block's largest number, which is at most 8 times its mean in norm.
    assert rel(gate, pre[0]) < 2.0 ** -5 and rel(up, pre[1]) < 2.0 ** -5
    h = act(pre[0], name)[0] * pre[1]
    down = block.down.forward_weight.dequantize().double()
    want = x64 + q(h.bfloat16()) @ down.t()
    assert rel(y, want) < 2.0 ** -4           # (4-bit codes of h that a rounding moves)
    assert rel(block.infer(x), want) < 2.0 ** -4

    # Backward, from what was kept.
    a, slope = act(gate, name)
    dh = (q(dy) @ block.down.backward_weight.dequantize().double().t()).bfloat16().double()
    dg, du = dh * up * slope, dh * a
    kn = kept_n.dequantize().double()
    assert rel(grads["gate"], dg.t() @ kn) < u and rel(grads["up"], du.t() @ kn) < u
    dn = dg @ block.w_gate.double() + du @ block.w_up.double()
    again = a * up
    assert rel(grads["down"], q(dy.t()) @ q(again.bfloat16().t()).t()) < 2.0 ** -4
    m, r = mean.double()[:, None], rstd.double()[:, None]
    nh = (kept_x.dequantize().double() - m) * r
    gn = dn * block.w.double()
    dx_want = dy.double() + r * (gn - gn.mean(1, keepdim=True) - nh * (gn * nh).mean(1, keepdim=True))
    assert rel(dx, dx_want) < u
    assert rel(grads["w"], (dn * nh).sum(0)) < u and rel(grads["b"], dn.sum(0)) < u


def test_gradient_against_differences(example):
    """The block's gradient along a direction against differences of a 64-bit block with the same
    weights: 8 bits keep each number to 2^-7 of its block, 4-bit factors to 2^-3."""
    block = example.Block(256, 512, seed=3)
    g = torch.Generator("cuda").manual_seed(5)
    x, dy, step = (torch.randn((64, 256), generator=g, device="cuda").bfloat16() for _ in range(3))
    y, saved = block.forward(x)
    dx, _ = block.backward(dy, saved)
    down = block.down.forward_weight.dequantize().double()

    def loss(t):
        d = t - t.mean(1, keepdim=True)
        n = d * (d.square().mean(1, keepdim=True) + 1e-5) ** -0.5 * block.w.double() + block.b.double()
        h = act(n @ block.w_gate.double().t(), "silu")[0] * (n @ block.w_up.double().t())
        return ((t + h @ down.t()) * dy.double()).sum()

    x64, s64 = x.double(), step.double()
    want = float(loss(x64 + 1e-4 * s64) - loss(x64 - 1e-4 * s64)) / 2e-4
    scale = float(dx.double().norm() * s64.norm()) / 256 ** 0.5       # of a random direction
    assert abs(float((dx.double() * s64).sum()) - want) < 0.25 * scale + 0.02 * abs(want)


def test_main(example, capsys):
    example.main(["--tokens", "200", "--width", "256", "--inner", "512", "--steps", "2"])
    out = capsys.readouterr().out
    assert "200 tokens" in out and "kept" in out
