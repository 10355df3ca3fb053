#!/usr/bin/env python3
"""A pre-norm feed-forward block whose training keeps its activations in 8 bits.

    n  = layer_norm(x) * w + b                  x kept in 8 bits as the norm reads it
    h  = act(n . Wg^T) * (n . Wu^T)             both pre-activations kept in 8 bits
    y  = x + h . Wd^T                           4-bit product

The backward pass reads the checkpoints in the place of x, n and the pre-activations, and
makes h again from them, so that h need not be kept at all: per token and layer 8-bit codes of
2 width + 2 inner numbers stay, and their scales, where bf16 activations would be
2 width + 3 inner numbers of two bytes.

    python examples/feed_forward_block.py [--tokens 4096] [--width 2048] [--inner 4096]
                                          [--activation silu|gelu_tanh] [--steps 5]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

import torch  # noqa: E402

import dense_fp32_gemm_09_gb300 as sg  # noqa: E402
from gated_residual_block import Linear  # noqa: E402


def held_bytes(*kept):
    return sum(q.codes.numel() + 4 * q.scales.numel() for q in kept)


class Block:
    def __init__(self, width: int, inner: int, activation: str = "silu", device="cuda", seed: int = 0):
        g = torch.Generator(device).manual_seed(seed)
        rand = lambda *shape: torch.randn(shape, generator=g, device=device)
        self.activation = activation
        self.w, self.b = 1 + 0.1 * rand(width), 0.1 * rand(width)
        self.w_gate = (rand(inner, width) / width ** 0.5).bfloat16()
        self.w_up = (rand(inner, width) / width ** 0.5).bfloat16()
        self.down = Linear(rand(width, inner) / inner ** 0.5, "nvfp4")

    def forward(self, x):
        """(y, what backward needs)."""
        n, mean, rstd, kept_x = sg.layer_norm(x, self.w, self.b, keep="8bit")
        kept_n = sg.act8_quantize(n)
        h, kept = sg.gated_ff(n, self.w_gate, self.w_up, activation=self.activation, keep="8bit")
        return x + self.down.forward(h), (kept_x, mean, rstd, kept_n, kept)

    def infer(self, x):
        """y, with nothing kept."""
        n, _, _ = sg.layer_norm(x, self.w, self.b)
        h = sg.gated_ff(n, self.w_gate, self.w_up, activation=self.activation)
        return x + self.down.forward(h)

    def backward(self, dy, saved):
        """Gradients of x and of every parameter, by name."""
        kept_x, mean, rstd, kept_n, kept = saved
        dh = self.down.backward_input(dy)
        dn, dw_gate, dw_up, h = sg.gated_ff_backward(dh, kept_n, self.w_gate, self.w_up, kept,
                                                     activation=self.activation, return_h=True)
        dw_down = self.down.backward_weight_of(dy, h)
        dx, dw, db = sg.layer_norm_backward(dn, kept_x, mean, rstd, self.w, dy=dy)
        return dx, {"gate": dw_gate, "up": dw_up, "down": dw_down, "w": dw, "b": db}


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--width", type=int, default=2048)
    ap.add_argument("--inner", type=int, default=4096)
    ap.add_argument("--activation", choices=("silu", "gelu_tanh"), default="silu")
    ap.add_argument("--steps", type=int, default=5)
    a = ap.parse_args(argv)
    block = Block(a.width, a.inner, a.activation)
    x = torch.randn(a.tokens, a.width, device="cuda").bfloat16()
    dy = torch.randn_like(x)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for step in range(a.steps + 3):
        if step == 3:
            start.record()
        y, saved = block.forward(x)
        dx, grads = block.backward(dy, saved)
    end.record()
    torch.cuda.synchronize()
    kept = held_bytes(saved[0], saved[3], *saved[4])
    full = 2 * a.tokens * (2 * a.width + 3 * a.inner)
    norms = {k: round(float(v.float().norm()), 3) for k, v in grads.items()}
    print(f"{a.tokens} tokens, width {a.width}, inner {a.inner}, {a.activation}: "
          f"{start.elapsed_time(end) / a.steps * 1e3:.0f} us a step forward and backward, "
          f"{kept / 2 ** 20:.1f} MiB kept ({full / 2 ** 20:.1f} in bf16); "
          f"|y| {float(y.float().norm()):.3f} |dx| {float(dx.float().norm()):.3f} {norms}")


if __name__ == "__main__":
    main()
