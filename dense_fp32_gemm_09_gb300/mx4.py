"""4-bit operands: quantisation, its inverse and the product of two quantised matrices.

A matrix is held as e2m1 codes with one 8-bit scale per block of 16 (``"nvfp4"``: e4m3
scales and an optional float32 scale for the whole tensor) or 32 (``"mxfp4"``: powers of
two) consecutive columns.  ``include/sgemm.h`` states the formats and their layout.
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
    scale of the whole tensor (one float32 on the device, None for 1)."""

    __slots__ = ("rows", "cols", "fmt", "tensor_scale", "device", "_codes", "_scales", "_both",
                 "_ptrs")

    def __init__(self, codes, scales, rows: int, cols: int, fmt: str, tensor_scale=None):
        ptrs = _t.fast().stored_addresses(codes, scales, rows, cols, _format(fmt), tensor_scale)
        if ptrs is None:          # another device, or something to refuse
            for t, name, shape in zip((codes, scales), ("codes", "scales"),
                                      mx4_shapes(rows, cols, fmt)):
                _t.cuda_tensor(t, name)
                if t.dtype != torch.uint8 or t.shape != shape or not t.is_contiguous():
                    raise ValueError(f"{name} must be a contiguous uint8 tensor of shape {shape}")
            _t.same_device(scales, "scales", codes.device)
            if tensor_scale is not None:
                if fmt != "nvfp4":
                    raise ValueError("only nvfp4 has a tensor scale")
                _t.one_float(tensor_scale, "tensor_scale", codes.device)
            ptrs = codes.data_ptr(), scales.data_ptr(), _t.ptr(tensor_scale)
        self.rows, self.cols, self.fmt, self.tensor_scale = rows, cols, fmt, tensor_scale
        self.device = codes.device
        self._codes, self._scales, self._both, self._ptrs = codes, scales, None, ptrs

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
        at = both.data_ptr()
        q.rows, q.cols, q.fmt, q.tensor_scale, q.device = rows, cols, fmt, tensor_scale, both.device
        q._codes, q._scales, q._both = None, None, both
        q._ptrs = (at, at + -(-rows // 128) * -(-cols // 128) * 8192,
                   None if tensor_scale is None else tensor_scale.data_ptr())
        return q

    def _views(self):
        if self._codes is None:
            codes, scales = mx4_shapes(self.rows, self.cols, self.fmt)
            n = math.prod(codes)
            self._codes = self._both[:n].view(codes)
            self._scales = self._both[n:].view(scales)

    @property
    def codes(self):
        self._views()
        return self._codes

    @property
    def scales(self):
        self._views()
        return self._scales

    @property
    def shape(self):
        return self.rows, self.cols

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
    codes, scales, ts = q._ptrs
    call.run("sgemm_mx4_quantize", trans, rows, cols, dt, x.data_ptr(), ld, code, ts, codes, scales)
    return q


def mx4_dequantize(q: Mx4, dtype=torch.float32, out=None, *, stream=None):
    """The rows x cols numbers that `q` holds, rounded once to `dtype` (or into ``out``)."""
    if not isinstance(q, Mx4):
        raise TypeError("q must be an Mx4")
    if stream is None and out is None and _t.current(q.device):
        out = _t.fast().mx4_dequantize(q._ptrs, q.rows, q.cols, FORMATS[q.fmt],
                                       _t.dtype_code(dtype, "dtype"))
        _t.checked(out, "sgemm_mx4_dequantize")
        return out
    call = _t.Call(q.device, stream)
    if out is None:
        dt, ld = _t.dtype_code(dtype, "dtype"), max(q.cols, 1)
        out = call.empty((q.rows, q.cols), dtype)
    else:
        ld = _t.matrix(out, "out", q.shape, None, q.device)
        dt = _t.dtype_code(out.dtype, "out")
    codes, scales, ts = q._ptrs
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
    if a.cols != b.cols:
        raise ValueError(f"inner dimensions differ: a is {a.shape}, b is {b.shape}")
    if a.fmt != b.fmt:
        raise ValueError(f"formats differ: a is {a.fmt}, b is {b.fmt}")
    if a.device != b.device:
        raise ValueError(f"a and b must be on one device: {a.device}, {b.device}")
    M, N = a.rows, b.rows
    if stream is None and out is None and beta == 0.0 and _t.current(a.device):
        out = _t.fast().mx4_matmul(a._ptrs, b._ptrs, M, N, a.cols, FORMATS[a.fmt], alpha,
                                   _t.dtype_code(dtype, "dtype"))
        _t.checked(out, "sgemm_mx4_matmul")
        return out
    call = _t.Call(a.device, stream)
    if out is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs `out` (the C that is scaled)")
        dt, ld = _t.dtype_code(dtype, "dtype"), max(N, 1)
        out = call.empty((M, N), dtype)
    else:
        ld = _t.matrix(out, "out", (M, N), None, a.device)
        dt = _t.dtype_code(out.dtype, "out")
    a_codes, a_scales, a_ts = a._ptrs
    b_codes, b_scales, b_ts = b._ptrs
    call.run("sgemm_mx4_matmul", M, N, a.cols, FORMATS[a.fmt], alpha, a_codes, a_scales, a_ts,
             b_codes, b_scales, b_ts, beta, dt, out.data_ptr(), ld)
    return out
