"""Layer norm and its gradient.

    m = mean(x)    r = (mean((x - m)^2) + eps)^-1/2    y = (x - m) * r * weight + bias

All sums are float32, the variance from differences to the mean.  Results are outside torch's
graph, also of inputs that require a gradient: ``layer_norm_backward`` is the gradient, to be
called by hand or from a ``torch.autograd.Function``.  ``stream`` as in ``mx4``.
"""
from __future__ import annotations

import ctypes

import torch

from . import _tensors as _t
from . import norms as _norms
from .act8 import Act8, held


def layer_norm(x, weight=None, bias=None, *, eps: float = 1e-5, keep: str | None = None,
               stream=None):
    """(y, mean, rstd) of the rows of a 2-D float32, bfloat16 or float16 CUDA view with unit
    column stride.  ``weight`` and ``bias`` (cols,) are both float32 or both of x's type; mean
    and rstd are float32.  With ``keep="8bit"`` also x as an ``Act8``, for the backward pass:
    (y, mean, rstd, kept)."""
    if keep not in (None, "8bit"):
        raise ValueError(f"keep must be None or '8bit', got {keep!r}")
    if stream is None:
        out = _t.fast().layer_norm(x, weight, bias, eps, keep is not None)
        if out is not None:
            _t.checked(out, "sgemm_layer_norm_forward")
            return out[:3] if keep is None else (*out[:3], Act8._of(*out[3:], *x.shape))
    call = _t.Call(_t.cuda_tensor(x, "x").device, stream)
    rows, cols, dt, ld = _norms._rows(x, "x")
    wt = _norms._weights(cols, x, ("weight", weight), ("bias", bias))
    y = call.empty((rows, cols), x.dtype)
    mean, rstd = call.empty((rows,), torch.float32), call.empty((rows,), torch.float32)
    kept = None if keep is None else Act8._new(call, rows, cols)
    codes, scales = (None, None) if kept is None else kept._addresses()
    call.run("sgemm_layer_norm_forward", rows, cols, dt, x.data_ptr(), ld, _t.ptr(weight),
             _t.ptr(bias), wt, eps, y.data_ptr(), cols, mean.data_ptr(), rstd.data_ptr(), codes,
             scales)
    return (y, mean, rstd) if kept is None else (y, mean, rstd, kept)


def layer_norm_backward(dh, x, mean, rstd, weight=None, *, dy=None, stream=None):
    """(dx, dweight, dbias) of ``layer_norm`` from the gradient ``dh`` of its result.  ``x`` is
    the norm's input or an ``Act8`` of it; ``dy``, the gradient that reaches x past the norm, is
    added to dx in the same pass.  dweight (None without a weight) and dbias are float32 sums
    over the rows, in a fixed order."""
    if stream is None:
        held_x = (None, x._codes, x._scales) if isinstance(x, Act8) else (x, None, None)
        fits = held_x[0] is x or x.shape == getattr(dh, "shape", None)
        out = _t.fast().layer_norm_backward(dh, *held_x, mean, rstd, weight, dy) if fits else None
        if out is not None:
            _t.checked(out, "sgemm_layer_norm_backward")
            return out
    call = _t.Call(_t.cuda_tensor(dh, "dh").device, stream)
    rows, cols, dt, lddh = _norms._rows(dh, "dh")
    codes = scales = x_at = None
    ldx = cols
    if isinstance(x, Act8):
        codes, scales = held(x, "x", dh.shape, dh.device)
    else:
        ldx = _t.matrix(x, "x", dh.shape, dh.dtype, dh.device)
        x_at = x.data_ptr()
    lddy = 0 if dy is None else _t.matrix(dy, "dy", dh.shape, dh.dtype, dh.device)
    _t.vector(mean, "mean", rows, torch.float32, dh.device)
    _t.vector(rstd, "rstd", rows, torch.float32, dh.device)
    wt = _norms._weights(cols, dh, ("weight", weight))
    dx = call.empty((rows, cols), dh.dtype)
    dweight = None if weight is None else call.empty((cols,), torch.float32)
    dbias = call.empty((cols,), torch.float32)
    # From torch's allocator, so that a captured graph owns what it uses.
    size = ctypes.c_size_t(0)
    with torch.cuda.device(dh.device):
        _t.check(_t.function("sgemm_layer_norm_backward_workspace")(rows, cols,
                                                                    ctypes.byref(size)),
                 "sgemm_layer_norm_backward_workspace")
    ws = call.empty((size.value,), torch.uint8)
    call.run("sgemm_layer_norm_backward", rows, cols, dt, dh.data_ptr(), lddh, _t.ptr(dy), lddy,
             x_at, ldx, codes, scales, mean.data_ptr(), rstd.data_ptr(),
             _t.ptr(weight), wt, dx.data_ptr(), cols, _t.ptr(dweight), dbias.data_ptr(),
             ws.data_ptr(), size.value)
    return dx, dweight, dbias
