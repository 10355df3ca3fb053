"""4-bit operands: quantisation, its inverse and the product of two quantised matrices.

A matrix is held as e2m1 codes with one 8-bit scale per block of 16 (``"nvfp4"``: e4m3
scales and an optional float32 scale for the whole tensor) or 32 (``"mxfp4"``: powers of
two) consecutive columns.  ``include/sgemm.h`` states the formats and their layout.

Results are outside torch's graph, also of inputs that require a gradient: quantisation has none, and
a product's is two more products (``examples/gated_residual_block.py``).  With ``stream`` a
call runs on that stream, in no order with the current one; as everywhere in torch, inputs
made on another stream must be kept until it is done with them.
"""
from __future__ import annotations

import math

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
    scale of the whole tensor (one float32 on the device, None for 1).  Its shape, format and
    buffers stay; ``tensor_scale`` may be set, which scales the numbers held."""

    __slots__ = ("_rows", "_cols", "_fmt", "_ts", "_codes", "_scales", "_both")

    def __init__(self, codes, scales, rows: int, cols: int, fmt: str, tensor_scale=None):
        code = _format(fmt)
        self._rows, self._cols, self._fmt, self._ts = rows, cols, fmt, tensor_scale
        self._codes, self._scales, self._both = codes, scales, None
        if scales is None or _t.fast().mx4_holds(self._stored(), rows, cols, code) is None:
            self._addresses()          # on another device, or something to refuse

    @classmethod
    def _new(cls, call, rows: int, cols: int, fmt: str, tensor_scale):
        """An unwritten matrix: one allocation, codes first."""
        padded = -(-rows // 128) * -(-cols // 128)
        both = call.empty(padded * (9216 if fmt == "nvfp4" else 8704), torch.uint8)
        return cls._of(both, rows, cols, fmt, tensor_scale)

    @classmethod
    def _of(cls, both, rows: int, cols: int, fmt: str, tensor_scale):
        """The matrix in one buffer, codes first."""
        q = cls.__new__(cls)
        q._rows, q._cols, q._fmt, q._ts = rows, cols, fmt, tensor_scale
        q._codes, q._scales, q._both = None, None, both
        return q

    def _stored(self):
        """The tensors as the binding takes them: (codes, scales, tensor scale), or both
        buffers in one and no scales."""
        if self._both is not None:
            return self._both, None, self._ts
        return self._codes, self._scales, self._ts

    def _addresses(self):
        """(codes, scales, tensor scale) as the library takes them, of buffers that fit."""
        shapes = mx4_shapes(self._rows, self._cols, self._fmt)
        if self._both is not None:
            sizes = [math.prod(shape) for shape in shapes]
            if self._both.dtype != torch.uint8 or self._both.shape != (sum(sizes),):
                raise ValueError("the matrix's buffer is not the one it was made with")
            at = self._both.data_ptr()
            return at, at + sizes[0], _t.ptr(self._scale_of(self._ts))
        for t, name, shape in zip((self._codes, self._scales), ("codes", "scales"), shapes):
            _t.cuda_tensor(t, name)
            if t.dtype != torch.uint8 or t.shape != shape or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous uint8 tensor of shape {shape}")
        _t.same_device(self._scales, "scales", self._codes.device)
        return self._codes.data_ptr(), self._scales.data_ptr(), _t.ptr(self._scale_of(self._ts))

    def _scale_of(self, t):
        if t is not None and self._fmt != "nvfp4":
            raise ValueError("only nvfp4 has a tensor scale")
        return _t.one_float(t, "tensor_scale", self.device)

    @property
    def rows(self):
        return self._rows

    @property
    def cols(self):
        return self._cols

    @property
    def fmt(self):
        return self._fmt

    @property
    def device(self):
        return (self._codes if self._both is None else self._both).device

    @property
    def tensor_scale(self):
        return self._ts

    @tensor_scale.setter
    def tensor_scale(self, t):
        self._ts = self._scale_of(t)

    def _views(self):
        if self._both is None:
            return self._codes, self._scales
        codes, scales = mx4_shapes(self._rows, self._cols, self._fmt)
        n = math.prod(codes)
        return self._both[:n].view(codes), self._both[n:].view(scales)

    @property
    def codes(self):
        return self._views()[0]

    @property
    def scales(self):
        return self._views()[1]

    @property
    def shape(self):
        return self._rows, self._cols

    def dequantize(self, dtype=torch.float32, *, stream=None):
        return mx4_dequantize(self, dtype, stream=stream)

    def __repr__(self):
        return f"Mx4({self.rows} x {self.cols}, {self.fmt}, {self.device})"


def mx4_quantize(x, fmt: str = "nvfp4", *, tensor_scale=None, stream=None) -> Mx4:
    """Quantises the rows of a 2-D float32, bfloat16 or float16 CUDA view.  A view with
    unit row stride (``x.t()``) is read as the transpose that it is, without a copy.
    ``tensor_scale`` (nvfp4 only) is one float32 >= 0 on the device: usually amax(x) / (6 * 448),
    which puts the largest block scale at the top of e4m3.  Where that is 0, as for a matrix
    of zeros, every number held is 0."""
    code = _format(fmt)
    if stream is None:
        both = _t.fast().mx4_quantize(x, code, tensor_scale)
        if both is not None:
            _t.checked(both, "sgemm_mx4_quantize")
            return Mx4._of(both, *x.shape, fmt, tensor_scale)
    _t.cuda_tensor(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    rows, cols = x.shape
    trans = 0 if cols <= 1 or x.stride(1) == 1 else 1
    ld = _t.row_ld(x.t() if trans else x, "x")
    dt = _t.dtype_code(x.dtype, "x")
    device = x.device
    if tensor_scale is not None:
        if fmt != "nvfp4":
            raise ValueError("only nvfp4 has a tensor scale")
        _t.one_float(tensor_scale, "tensor_scale", device)
    call = _t.Call(device, stream)
    q = Mx4._new(call, rows, cols, fmt, tensor_scale)
    codes, scales, ts = q._addresses()
    call.run("sgemm_mx4_quantize", trans, rows, cols, dt, x.data_ptr(), ld, code, ts, codes, scales)
    return q


def mx4_dequantize(q: Mx4, dtype=torch.float32, out=None, *, stream=None):
    """The rows x cols numbers that `q` holds, rounded once to `dtype` (or into ``out``)."""
    if not isinstance(q, Mx4):
        raise TypeError("q must be an Mx4")
    if stream is None and out is None:
        out = _t.fast().mx4_dequantize(q._stored(), q._rows, q._cols, FORMATS[q._fmt],
                                       _t.dtype_code(dtype, "dtype"))
        if out is not None:
            _t.checked(out, "sgemm_mx4_dequantize")
            return out
    call = _t.Call(q.device, stream)
    if out is None:
        dt, ld = _t.dtype_code(dtype, "dtype"), max(q.cols, 1)
        out = call.empty((q.rows, q.cols), dtype)
    else:
        ld = _t.matrix(out, "out", q.shape, None, q.device)
        dt = _t.dtype_code(out.dtype, "out")
    codes, scales, ts = q._addresses()
    call.run("sgemm_mx4_dequantize", q.rows, q.cols, FORMATS[q.fmt], codes, scales, ts, dt,
             out.data_ptr(), ld)
    return out


def mx4_matmul(a: Mx4, b: Mx4, out=None, *, dtype=torch.float32, alpha: float = 1.0,
               beta: float = 0.0, stream=None):
    """C = alpha * A . B^T + beta * C for A (M x K) and B (N x K), both quantised along K
    in one format: activations times a layer's weight with one row per output.  Sums are
    held in float32.  ``out`` may be an (M, N) float32, bfloat16 or float16 view; with
    beta == 0 it is only written, otherwise it is the C of the formula."""
    if not isinstance(a, Mx4) or not isinstance(b, Mx4):
        raise TypeError("a and b must be Mx4")
    if a._cols != b._cols:
        raise ValueError(f"inner dimensions differ: a is {a.shape}, b is {b.shape}")
    if a._fmt != b._fmt:
        raise ValueError(f"formats differ: a is {a.fmt}, b is {b.fmt}")
    M, N = a._rows, b._rows
    if stream is None and out is None and beta == 0.0:
        out = _t.fast().mx4_matmul(a._stored(), b._stored(), M, N, a._cols, FORMATS[a._fmt], alpha,
                                   _t.dtype_code(dtype, "dtype"))
        if out is not None:
            _t.checked(out, "sgemm_mx4_matmul")
            return out
    if a.device != b.device:
        raise ValueError(f"a and b must be on one device: {a.device}, {b.device}")
    call = _t.Call(a.device, stream)
    if out is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs `out` (the C that is scaled)")
        dt, ld = _t.dtype_code(dtype, "dtype"), max(N, 1)
        out = call.empty((M, N), dtype)
    else:
        ld = _t.matrix(out, "out", (M, N), None, a.device)
        dt = _t.dtype_code(out.dtype, "out")
    a_codes, a_scales, a_ts = a._addresses()
    b_codes, b_scales, b_ts = b._addresses()
    call.run("sgemm_mx4_matmul", M, N, a.cols, FORMATS[a.fmt], alpha, a_codes, a_scales, a_ts,
             b_codes, b_scales, b_ts, beta, dt, out.data_ptr(), ld)
    return out
