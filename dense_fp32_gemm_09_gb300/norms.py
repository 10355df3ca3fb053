"""Norms before and after a residual block, fused with its gate and residual scale.

    after:   r  = (mean(block^2) + eps)^-1/2
             y  = residual + scale * gate * (block * r * weight)
    before:  r' = (mean(y^2) + eps)^-1/2
             h  = y * r' * next_weight

``norm_before`` is the second line on its own, ``norm_after`` the first, or both in one
pass.  ``h`` may leave the pass as a 4-bit matrix (``mx4.Mx4``).  All sums are float32.

Results are outside torch's graph, also of inputs that require a gradient: the ``_backward``
functions are the gradients, to be called by hand or from a ``torch.autograd.Function``.
``stream`` as in ``mx4``.
"""
from __future__ import annotations

import ctypes

import torch

from . import _tensors as _t
from . import mx4 as _mx4

NOT_QUANTIZED = -1


def _rows(x, name: str):
    _t.cuda_tensor(x, name)
    dt = _t.dtype_code(x.dtype, name)
    ld = _t.row_ld(x, name)
    rows, cols = x.shape
    if cols == 0:
        raise ValueError(f"{name} has rows of no columns")
    return rows, cols, dt, ld


def _weights(cols: int, x, *named):
    """Type code of the weights given (all of one type: float32 or x's)."""
    dtype = None
    for name, w in named:
        if w is None:
            continue
        _t.vector(w, name, cols, dtype, x.device)
        if w.dtype not in (torch.float32, x.dtype):
            raise TypeError(f"{name} must be float32 or {x.dtype}, got {w.dtype}")
        dtype = w.dtype
    return _t.DTYPE_CODES[dtype or torch.float32]


def _gate(gate, x):
    """Leading dimension of a (rows, cols) gate, 0 for a (cols,) one or none."""
    if gate is None:
        return 0
    _t.cuda_tensor(gate, "gate")
    if gate.dim() == 1:
        _t.vector(gate, "gate", x.shape[1], x.dtype, x.device)
        return 0
    return _t.matrix(gate, "gate", x.shape, x.dtype, x.device)


def _forward(stream, x, block, weight, gate, scale, eps, next_norm, next_weight, quantize,
             tensor_scale):
    if stream is None:
        fmt = NOT_QUANTIZED if quantize is None else _mx4._format(quantize)
        out = _t.fast().norm_forward(x, block, weight, gate, scale, eps, next_norm, next_weight,
                                     fmt, tensor_scale)
        if out is not None:
            _t.checked(out, "sgemm_norm_forward")
            if quantize is None:
                return out
            y, rstd, both, next_rstd = out
            return y, rstd, _mx4.Mx4._of(both, *x.shape, quantize, tensor_scale), next_rstd
    name = "residual" if block is not None else "x"
    call = _t.Call(_t.cuda_tensor(x, name).device, stream)
    rows, cols, dt, ldr = _rows(x, name)
    ldb = 0 if block is None else _t.matrix(block, "block", x.shape, x.dtype, x.device)
    wt = _weights(cols, x, ("weight", weight), ("next_weight", next_weight))
    ldg = _gate(gate, x)
    y = rstd = h = next_rstd = q = None
    fmt = NOT_QUANTIZED
    if block is not None:
        y, rstd = call.empty((rows, cols), x.dtype), call.empty((rows,), torch.float32)
    ts = None
    if next_norm:
        next_rstd = call.empty((rows,), torch.float32)
        if quantize is None:
            if tensor_scale is not None:
                raise ValueError("tensor_scale goes with quantize='nvfp4'")
            h = call.empty((rows, cols), x.dtype)
        else:
            fmt = _mx4._format(quantize)
            if tensor_scale is not None and quantize != "nvfp4":
                raise ValueError("only nvfp4 has a tensor scale")
            ts = _t.one_float(tensor_scale, "tensor_scale", x.device)
            q = _mx4.Mx4._new(call, rows, cols, quantize, ts)
    codes, scales, _ = (None, None, None) if q is None else q._addresses()
    call.run("sgemm_norm_forward", rows, cols, dt, _t.ptr(block), ldb, x.data_ptr(), ldr,
             _t.ptr(weight), _t.ptr(next_weight), wt, _t.ptr(gate), ldg, scale, eps, _t.ptr(y),
             cols, _t.ptr(rstd), int(next_norm), _t.ptr(h), cols, _t.ptr(next_rstd), fmt,
             _t.ptr(ts), codes, scales)
    return y, rstd, h if q is None else q, next_rstd


def norm_before(x, weight=None, *, eps: float = 1e-6, quantize: str | None = None,
                tensor_scale=None, stream=None):
    """(h, rstd) of the norm before a block: h = x * rstd * weight with rstd =
    (mean(x^2) + eps)^-1/2 per row.  ``x`` is a 2-D float32, bfloat16 or float16 CUDA view
    with unit column stride; ``weight`` (cols,) is float32 or of x's type.  With
    ``quantize="nvfp4"`` or ``"mxfp4"`` h is an ``Mx4``, quantised from float32."""
    _, _, h, rstd = _forward(stream, x, None, None, None, 1.0, eps, True, weight, quantize,
                             tensor_scale)
    return h, rstd


def norm_after(block, residual, weight=None, *, gate=None, scale: float = 1.0, eps: float = 1e-6,
               next_norm: bool | None = None, next_weight=None, quantize: str | None = None,
               tensor_scale=None, stream=None):
    """y = residual + scale * gate * norm(block): (y, rstd).

    ``gate`` is (rows, cols), (cols,) for one gate shared by all rows, or None for ones.
    With ``next_norm`` (implied by ``next_weight`` or ``quantize``) the norm before the
    next block runs in the same pass: (y, rstd, h, next_rstd), with h as in
    ``norm_before`` and computed from y before it is rounded."""
    if block is None:
        raise TypeError("block must be a torch.Tensor")
    if next_norm is None:
        next_norm = next_weight is not None or quantize is not None
    elif not next_norm and (next_weight is not None or quantize is not None):
        raise ValueError("next_weight and quantize need the next norm")
    if not next_norm and tensor_scale is not None:
        raise ValueError("tensor_scale goes with quantize='nvfp4'")
    out = _forward(stream, residual, block, weight, gate, scale, eps, next_norm, next_weight,
                   quantize, tensor_scale)
    return out if next_norm else out[:2]


def _backward(stream, ref, dy, dh, y, next_rstd, next_weight, block, rstd, weight, gate, scale):
    if stream is None:
        out = _t.fast().norm_backward(ref, dy, dh, y, next_rstd, next_weight, block, rstd, weight,
                                      gate, scale)
        if out is not None:
            _t.checked(out, "sgemm_norm_backward_ws")
            return out
    call = _t.Call(_t.cuda_tensor(ref, "dy" if dy is not None else "dh").device, stream)
    rows, cols, dt, _ = _rows(ref, "dy" if dy is not None else "dh")
    check = lambda t, name: 0 if t is None else _t.matrix(t, name, ref.shape, ref.dtype, ref.device)
    lddy, lddh, ldy, ldb = check(dy, "dy"), check(dh, "dh"), check(y, "y"), check(block, "block")
    for r, name in ((rstd, "rstd"), (next_rstd, "next_rstd")):
        if r is not None:
            _t.vector(r, name, rows, torch.float32, ref.device)
    wt = _weights(cols, ref, ("weight", weight), ("next_weight", next_weight))
    ldg = _gate(gate, ref)
    dx = dblock = dweight = dgate = dnext = None
    if dh is not None:
        dx = call.empty((rows, cols), ref.dtype)
        if next_weight is not None:
            dnext = call.empty((cols,), torch.float32)
    if block is not None:
        dblock = call.empty((rows, cols), ref.dtype)
        if weight is not None:
            dweight = call.empty((cols,), torch.float32)
        if gate is not None:
            dgate = call.empty((rows, cols), ref.dtype) if ldg else \
                call.empty((cols,), torch.float32)
    # From torch's allocator, so that a captured graph owns what it uses.
    ws = None
    if dweight is not None or dnext is not None or (dgate is not None and not ldg):
        size = ctypes.c_size_t(0)
        with torch.cuda.device(ref.device):
            _t.check(_t.function("sgemm_norm_backward_workspace")(rows, cols, ctypes.byref(size)),
                     "sgemm_norm_backward_workspace")
        ws = call.empty((size.value,), torch.uint8)
    call.run("sgemm_norm_backward_ws", rows, cols, dt, _t.ptr(dy), lddy, _t.ptr(dh), lddh, _t.ptr(y),
             ldy, _t.ptr(next_rstd), _t.ptr(next_weight), _t.ptr(block), ldb, _t.ptr(rstd),
             _t.ptr(weight), wt, _t.ptr(gate), ldg, scale, _t.ptr(dx), cols, _t.ptr(dblock), cols,
             _t.ptr(dgate), cols, _t.ptr(dweight), _t.ptr(dnext), _t.ptr(ws),
             0 if ws is None else ws.numel())
    return dx, dblock, dweight, dgate, dnext


def norm_before_backward(dh, x, rstd, weight=None, *, dy=None, stream=None):
    """(dx, dweight) of ``norm_before`` from the gradient of h; ``dy``, the gradient that
    reaches x past the block, is added to dx in the same pass.  dweight is float32 (None
    without a weight)."""
    if dh is None or x is None or rstd is None:
        raise TypeError("dh, x and rstd must be torch.Tensors")
    dx, _, _, _, dw = _backward(stream, dh, dy, dh, x, rstd, weight, None, None, None, None, 1.0)
    return dx, dw


def norm_after_backward(dy, block, rstd, weight=None, *, gate=None, scale: float = 1.0, dh=None,
                        y=None, next_rstd=None, next_weight=None, stream=None):
    """(dresidual, dblock, dweight, dgate, dnext_weight) of ``norm_after``.

    Without the next norm dresidual is ``dy`` itself.  With it, ``dh`` is the gradient of
    h, ``y`` and ``next_rstd`` are what the forward pass returned, and ``dy`` (the gradient
    that reaches y past the next block, or None) joins in.  The gradients of the weights
    and of a shared gate are float32 sums over the rows, in a fixed order; what was not
    given has the gradient None."""
    ref = dy if dy is not None else dh
    if ref is None or block is None or rstd is None:
        raise TypeError("block, rstd and one of dy and dh must be torch.Tensors")
    if dh is None and (y is not None or next_rstd is not None or next_weight is not None):
        raise ValueError("y, next_rstd and next_weight go with dh")
    if dh is not None and (y is None or next_rstd is None):
        raise ValueError("dh needs y and next_rstd")
    out = _backward(stream, ref, dy, dh, y, next_rstd, next_weight, block, rstd, weight, gate, scale)
    return out if dh is not None else (dy,) + out[1:]
