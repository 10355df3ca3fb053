"""8-bit activation checkpoints: what a backward pass needs, kept at half the size of 2-byte
numbers or a quarter of float32.

A row is held as int8 codes with one float32 scale per 64 consecutive columns: value =
code * scale, scale = amax / 127, code the nearest integer to x * (127 / amax).
``include/sgemm.h`` states the format and its layout.  ``layer_norm`` and ``gated_ff``
(``keep="8bit"``) write checkpoints in their own pass, and their ``_backward`` functions read
them in the place of matrices.

Results are outside torch's graph, also of inputs that require a gradient.  ``stream`` as in
``mx4``.
"""
from __future__ import annotations

import torch

from . import _tensors as _t

BLOCK = 64


def act8_shapes(rows: int, cols: int):
    """Shapes of the two buffers of a rows x cols matrix: (int8 codes, float32 scales)."""
    blocks = -(-cols // BLOCK)
    return (rows, BLOCK * blocks), (rows, blocks)


class Act8:
    """A rows x cols matrix held in 8 bits.  Its shape and buffers stay; ``codes`` and
    ``scales`` are contiguous tensors of ``act8_shapes``."""

    __slots__ = ("_rows", "_cols", "_codes", "_scales")

    def __init__(self, codes, scales, rows: int, cols: int):
        if rows < 0 or cols < 0:
            raise ValueError(f"a matrix of {rows} x {cols}")
        self._rows, self._cols, self._codes, self._scales = rows, cols, codes, scales
        self._addresses()

    @classmethod
    def _new(cls, call, rows: int, cols: int):
        """An unwritten matrix."""
        codes, scales = act8_shapes(rows, cols)
        return cls._of(call.empty(codes, torch.int8), call.empty(scales, torch.float32), rows, cols)

    @classmethod
    def _of(cls, codes, scales, rows: int, cols: int):
        """The matrix in buffers that fit."""
        q = cls.__new__(cls)
        q._rows, q._cols, q._codes, q._scales = rows, cols, codes, scales
        return q

    def _addresses(self):
        """(codes, scales) as the library takes them, of buffers that fit."""
        shapes = act8_shapes(self._rows, self._cols)
        for t, name, shape, dtype in zip((self._codes, self._scales), ("codes", "scales"), shapes,
                                         (torch.int8, torch.float32)):
            _t.cuda_tensor(t, name)
            if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape}")
        _t.same_device(self._scales, "scales", self._codes.device)
        return self._codes.data_ptr(), self._scales.data_ptr()

    @property
    def rows(self):
        return self._rows

    @property
    def cols(self):
        return self._cols

    @property
    def shape(self):
        return self._rows, self._cols

    @property
    def device(self):
        return self._codes.device

    @property
    def codes(self):
        return self._codes

    @property
    def scales(self):
        return self._scales

    def dequantize(self, dtype=torch.float32, *, stream=None):
        return act8_dequantize(self, dtype, stream=stream)

    def __repr__(self):
        return f"Act8({self.rows} x {self.cols}, {self.device})"


def held(q, name: str, shape, device):
    """(codes, scales) of a checkpoint that a call expects to have this shape."""
    if tuple(q.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(q.shape)}")
    _t.same_device(q, name, device)
    return q._addresses()


def act8_quantize(x, *, stream=None) -> Act8:
    """The rows of a 2-D float32, bfloat16 or float16 CUDA view with unit column stride, in 8
    bits.  A block of 64 columns with an infinity or a NaN is NaN; one whose largest magnitude
    is below 2^-100 is zeros."""
    if stream is None:
        out = _t.fast().act8_quantize(x)
        if out is not None:
            _t.checked(out, "sgemm_act8_quantize")
            return Act8._of(*out, *x.shape)
    call = _t.Call(_t.cuda_tensor(x, "x").device, stream)
    dt, ld = _t.dtype_code(x.dtype, "x"), _t.row_ld(x, "x")
    rows, cols = x.shape
    q = Act8._new(call, rows, cols)
    call.run("sgemm_act8_quantize", rows, cols, dt, x.data_ptr(), ld, *q._addresses())
    return q


def act8_dequantize(q: Act8, dtype=torch.float32, out=None, *, stream=None):
    """The rows x cols numbers that `q` holds, rounded once to `dtype` (or into ``out``)."""
    if not isinstance(q, Act8):
        raise TypeError("q must be an Act8")
    if stream is None and out is None:
        out = _t.fast().act8_dequantize(q._codes, q._scales, q._rows, q._cols,
                                        _t.dtype_code(dtype, "dtype"))
        if out is not None:
            _t.checked(out, "sgemm_act8_dequantize")
            return out
    call = _t.Call(q.device, stream)
    if out is None:
        dt, ld = _t.dtype_code(dtype, "dtype"), max(q.cols, 1)
        out = call.empty((q.rows, q.cols), dtype)
    else:
        ld = _t.matrix(out, "out", q.shape, None, q.device)
        dt = _t.dtype_code(out.dtype, "out")
    call.run("sgemm_act8_dequantize", q.rows, q.cols, *q._addresses(), dt, out.data_ptr(), ld)
    return out
