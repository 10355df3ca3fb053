"""4-bit operands: quantisation, its inverse and the product of two quantised matrices.

A matrix is held as e2m1 codes with one 8-bit scale per block of 16 (``"nvfp4"``: e4m3
scales and an optional float32 scale for the whole tensor) or 32 (``"mxfp4"``: powers of
two) consecutive columns.  ``include/sgemm.h`` states the formats and their layout.
"""
from __future__ import annotations

import torch

from . import _tensors as _t

FORMATS = {"nvfp4": 0, "mxfp4": 1}
BLOCK = {"nvfp4": 16, "mxfp4": 32}


def mx4_shapes(rows: int, cols: int, fmt: str):
    """Shapes of the two uint8 buffers of a rows x cols matrix: (codes, scales)."""
    blocks, padded = -(-rows // 128), -(-cols // 128)
    return (blocks, 4 * padded, 128, 16), (blocks, padded * (2 if fmt == "nvfp4" else 1), 32, 4, 4)


def _format(fmt) -> int:
    code = FORMATS.get(fmt)
    if code is None:
        raise ValueError(f"fmt must be one of {sorted(FORMATS)}, got {fmt!r}")
    return code


class Mx4:
    """A quantised rows x cols matrix: its two buffers, its format and, for nvfp4, the
    scale of the whole tensor (one float32 on the device, None for 1)."""

    __slots__ = ("codes", "scales", "rows", "cols", "fmt", "tensor_scale")

    def __init__(self, codes, scales, rows: int, cols: int, fmt: str, tensor_scale=None):
        _format(fmt)
        shapes = mx4_shapes(rows, cols, fmt)
        for t, name, shape in ((codes, "codes", shapes[0]), (scales, "scales", shapes[1])):
            _t.cuda_tensor(t, name)
            if t.dtype != torch.uint8 or t.shape != shape or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous uint8 tensor of shape {shape}")
        _t.same_device(scales, "scales", codes.device)
        if tensor_scale is not None and fmt != "nvfp4":
            raise ValueError("only nvfp4 has a tensor scale")
        self.codes, self.scales, self.rows, self.cols, self.fmt = codes, scales, rows, cols, fmt
        self.tensor_scale = _t.one_float(tensor_scale, "tensor_scale", codes.device)

    @property
    def shape(self):
        return self.rows, self.cols

    @property
    def device(self):
        return self.codes.device

    def dequantize(self, dtype=torch.float32, *, stream=None):
        return mx4_dequantize(self, dtype, stream=stream)

    def __repr__(self):
        return f"Mx4({self.rows} x {self.cols}, {self.fmt}, {self.device})"


def _empty(call, rows: int, cols: int, fmt: str, tensor_scale) -> Mx4:
    codes, scales = mx4_shapes(rows, cols, fmt)
    q = Mx4.__new__(Mx4)
    q.codes, q.scales = call.empty(codes, torch.uint8), call.empty(scales, torch.uint8)
    q.rows, q.cols, q.fmt, q.tensor_scale = rows, cols, fmt, tensor_scale
    return q


def mx4_quantize(x, fmt: str = "nvfp4", *, tensor_scale=None, stream=None) -> Mx4:
    """Quantises the rows of a 2-D float32, bfloat16 or float16 CUDA view.  A view with
    unit row stride (``x.t()``) is read as the transpose that it is, without a copy.
    ``tensor_scale`` (nvfp4 only) is one positive float32 on the device: usually
    amax(x) / (6 * 448), which puts the largest block scale at the top of e4m3."""
    code = _format(fmt)
    _t.cuda_tensor(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    rows, cols = x.shape
    trans = int(not (cols <= 1 or x.stride(1) == 1))
    ld = _t.row_ld(x.t() if trans else x, "x")
    dt = _t.dtype_code(x.dtype, "x")
    if tensor_scale is not None and fmt != "nvfp4":
        raise ValueError("only nvfp4 has a tensor scale")
    ts = _t.one_float(tensor_scale, "tensor_scale", x.device)
    if max(rows, cols) > _t.INT_MAX:
        raise ValueError("x: a size does not fit the library's 32-bit ints")
    call = _t.Call(x.device, stream)
    q = _empty(call, rows, cols, fmt, ts)
    call.run("sgemm_mx4_quantize", trans, rows, cols, dt, x.data_ptr(), ld, code, _t.ptr(ts),
             q.codes.data_ptr(), q.scales.data_ptr())
    return q


def mx4_dequantize(q: Mx4, dtype=torch.float32, out=None, *, stream=None):
    """The rows x cols numbers that `q` holds, rounded once to `dtype` (or into ``out``)."""
    if not isinstance(q, Mx4):
        raise TypeError("q must be an Mx4")
    call = _t.Call(q.device, stream)
    if out is None:
        dt, ld = _t.dtype_code(dtype, "dtype"), max(q.cols, 1)
        out = call.empty((q.rows, q.cols), dtype)
    else:
        ld = _t.matrix(out, "out", q.shape, None, q.device)
        dt = _t.dtype_code(out.dtype, "out")
    call.run("sgemm_mx4_dequantize", q.rows, q.cols, FORMATS[q.fmt], q.codes.data_ptr(),
             q.scales.data_ptr(), _t.ptr(q.tensor_scale), dt, out.data_ptr(), ld)
    return out


def mx4_matmul(a: Mx4, b: Mx4, out=None, *, dtype=torch.float32, alpha: float = 1.0,
               beta: float = 0.0, stream=None):
    """C = alpha * A . B^T + beta * C for A (M x K) and B (N x K), both quantised along K
    in one format: activations times a layer's weight with one row per output.  Sums are
    held in float32.  ``out`` may be an (M, N) float32, bfloat16 or float16 view; with
    beta == 0 it is only written, otherwise it is the C of the formula."""
    if not isinstance(a, Mx4) or not isinstance(b, Mx4):
        raise TypeError("a and b must be Mx4")
    if a.cols != b.cols:
        raise ValueError(f"inner dimensions differ: a is {a.shape}, b is {b.shape}")
    if a.fmt != b.fmt:
        raise ValueError(f"formats differ: a is {a.fmt}, b is {b.fmt}")
    if a.device != b.device:
        raise ValueError(f"a and b must be on one device: {a.device}, {b.device}")
    M, N = a.rows, b.rows
    call = _t.Call(a.device, stream)
    if out is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs `out` (the C that is scaled)")
        dt, ld = _t.dtype_code(dtype, "dtype"), max(N, 1)
        out = call.empty((M, N), dtype)
    else:
        ld = _t.matrix(out, "out", (M, N), None, a.device)
        dt = _t.dtype_code(out.dtype, "out")
    call.run("sgemm_mx4_matmul", M, N, a.cols, FORMATS[a.fmt], alpha, a.codes.data_ptr(),
             a.scales.data_ptr(), _t.ptr(a.tensor_scale), b.codes.data_ptr(),
             b.scales.data_ptr(), _t.ptr(b.tensor_scale), beta, dt, out.data_ptr(), ld)
    return out
