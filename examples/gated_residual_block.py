#!/usr/bin/env python3
"""A gated residual block with 4-bit linear layers, forward and backward.

    h  = norm(x) * w1                           quantised as it leaves the norm
    a  = h . W1^T                               4-bit product
    b  = a . W2^T                               quantise, 4-bit product
    y  = x + scale * gate * (norm(b) * w2)      and the next block's norm in the same pass

The weights are quantised once, along both of their dimensions: the forward pass
multiplies along a layer's inputs, the gradient of its input along its outputs.  The
gradient of a weight multiplies along the tokens, so both of its operands are quantised
transposed.  Every product accumulates in float32.

    python examples/gated_residual_block.py [--tokens 2048] [--width 1024] [--inner 4096]
                                            [--format nvfp4|mxfp4] [--steps 5]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import dense_fp32_gemm_09_gb300 as sg  # noqa: E402


class Linear:
    """y = x . W^T with W (out, in) held in 4 bits, for both directions of training."""

    def __init__(self, weight, fmt: str):
        self.fmt = fmt
        self.out_features, self.in_features = weight.shape
        self.forward_weight = quantize(weight, fmt)            # blocks along the inputs
        self.backward_weight = quantize(weight.t(), fmt)       # blocks along the outputs

    def forward(self, x):
        """`x`: a matrix, or an Mx4 that is quantised already."""
        q = x if isinstance(x, sg.Mx4) else quantize(x, self.fmt)
        return sg.mx4_matmul(q, self.forward_weight, dtype=torch.bfloat16)

    def backward(self, dy, x):
        """(gradient of x, gradient of W) from the gradient of y."""
        return self.backward_input(dy), self.backward_weight_of(dy, x)

    def backward_input(self, dy):
        return sg.mx4_matmul(quantize(dy, self.fmt), self.backward_weight, dtype=torch.bfloat16)

    def backward_weight_of(self, dy, x):
        return sg.mx4_matmul(quantize(dy.t(), self.fmt), quantize(x.t(), self.fmt))


def quantize(x, fmt: str):
    """nvfp4 with the tensor's own scale, so that no block's scale falls out of e4m3."""
    scale = None
    if fmt == "nvfp4":
        scale = (x.abs().amax().float() / (6 * 448)).clamp_(min=1e-30).view(1)
    return sg.mx4_quantize(x, fmt, tensor_scale=scale)


class Block:
    def __init__(self, width: int, inner: int, fmt: str, device="cuda", seed: int = 0):
        g = torch.Generator(device).manual_seed(seed)
        rand = lambda *shape: torch.randn(shape, generator=g, device=device)
        self.fmt, self.scale = fmt, 0.5
        self.up = Linear(rand(inner, width) / width ** 0.5, fmt)
        self.down = Linear(rand(width, inner) / inner ** 0.5, fmt)
        self.w_before, self.w_after, self.w_next = (1 + 0.1 * rand(width) for _ in range(3))
        self.gate = torch.sigmoid(rand(width)).bfloat16()

    def forward(self, x):
        """(y, h of the next block, what backward needs)."""
        h, rstd = sg.norm_before(x, self.w_before, quantize=self.fmt)
        a = self.up.forward(h)
        b = self.down.forward(a)
        y, rstd_b, h_next, rstd_y = sg.norm_after(b, x, self.w_after, gate=self.gate,
                                                  scale=self.scale, next_weight=self.w_next)
        return y, h_next, (x, h, rstd, a, b, rstd_b, y, rstd_y)

    def backward(self, dy, dh_next, saved):
        """Gradients of x and of every parameter, by name."""
        x, h, rstd, a, b, rstd_b, y, rstd_y = saved
        dres, db, dw_after, dgate, dw_next = sg.norm_after_backward(
            dy, b, rstd_b, self.w_after, gate=self.gate, scale=self.scale, dh=dh_next, y=y,
            next_rstd=rstd_y, next_weight=self.w_next)
        da, dw_down = self.down.backward(db, a)
        dh, dw_up = self.up.backward(da, h.dequantize(torch.bfloat16))
        dx, dw_before = sg.norm_before_backward(dh, x, rstd, self.w_before, dy=dres)
        return dx, {"up": dw_up, "down": dw_down, "w_before": dw_before, "w_after": dw_after,
                    "gate": dgate, "w_next": dw_next}


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=4096)
    ap.add_argument("--format", choices=("nvfp4", "mxfp4"), default="nvfp4")
    ap.add_argument("--steps", type=int, default=5)
    a = ap.parse_args(argv)
    block = Block(a.width, a.inner, a.format)
    x = torch.randn(a.tokens, a.width, device="cuda").bfloat16()
    dy, dh = torch.randn_like(x), torch.randn_like(x)
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    for step in range(a.steps + 3):
        if step == 3:
            start.record()
        y, h, saved = block.forward(x)
        dx, grads = block.backward(dy, dh, saved)
    end.record()
    torch.cuda.synchronize()
    norms = {k: round(float(v.float().norm()), 3) for k, v in grads.items()}
    print(f"{a.format}: {a.tokens} tokens, width {a.width}, inner {a.inner}: "
          f"{start.elapsed_time(end) / a.steps * 1e3:.0f} us a step forward and backward; "
          f"|y| {float(y.float().norm()):.3f} |dx| {float(dx.float().norm()):.3f} {norms}")


if __name__ == "__main__":
    main()
