"""The gated feed-forward block and its gradient.

    g = x . w_gate^T        u = x . w_up^T        h = act(g) * u

with x (tokens, inputs) and the weights (outputs, inputs), all bfloat16 or all float16.  Sums
are held in float32, and h is made from them before anything is rounded.

Results are outside torch's graph, also of inputs that require a gradient:
``gated_ff_backward`` is the gradient, to be called by hand or from a
``torch.autograd.Function``.  ``stream`` as in ``mx4``.
"""
from __future__ import annotations

import ctypes

import torch

from . import _tensors as _t
from .act8 import Act8, held

ACTIVATIONS = {"silu": 0, "gelu_tanh": 1}
KEEP = {None: 0, "full": 1, "8bit": 2}
_X, _GATE, _UP, _FP16 = 1, 2, 4, 8       # (`packed` of include/sgemm.h)


def _activation(name) -> int:
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {name!r}")
    return code


def _dtype(t, name: str) -> int:
    if t.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    return _t.dtype_code(t.dtype, name)


def _layer(ref, name: str, w_gate, w_up, inputs=None):
    """(outputs, inputs, leading dimensions) of the two weights, of ref's type and device."""
    ldg = _t.matrix(w_gate, "w_gate", None, ref.dtype, ref.device)
    ldu = _t.matrix(w_up, "w_up", w_gate.shape, ref.dtype, ref.device)
    N, K = w_gate.shape
    if inputs is not None and inputs != K:
        raise ValueError(f"inner dimensions differ: x has {inputs} columns, the weights have {K}")
    if N == 0 or K == 0:
        raise ValueError("the weights have no rows or no columns")
    return N, K, ldg, ldu


# Forward calls of up to so many tokens read every matrix in place, unless they keep 8-bit checkpoints.
_FEW_TOKENS = 16


def _packed(bit: int, t, ld: int) -> int:
    """`bit` where the kernels read a copy of a matrix: its rows are not 16-byte aligned."""
    aligned = t.data_ptr() % 16 == 0 and (t.shape[0] <= 1 or ld % 8 == 0)
    return 0 if aligned else bit


def _workspace(call, M: int, N: int, K: int, backward: int, packed: int):
    """From torch's allocator, so that a captured graph owns what it uses."""
    size = ctypes.c_size_t(0)
    _t.check(_t.function("sgemm_gated_ff_workspace")(M, N, K, backward, packed,
                                                     ctypes.byref(size)),
             "sgemm_gated_ff_workspace")
    return (call.empty((size.value,), torch.uint8) if size.value else None), size.value


def gated_ff(x, w_gate, w_up, *, activation: str = "silu", keep: str | None = None, stream=None):
    """h = act(x . w_gate^T) * (x . w_up^T), with act ``"silu"`` or ``"gelu_tanh"``.

    With ``keep`` also what the backward pass needs, (h, (gate, up)): the pre-activations as
    matrices of x's type (``"full"``) or as ``Act8`` (``"8bit"``), made from the float32 sums in
    the same pass."""
    act = _activation(activation)
    if keep not in KEEP:
        raise ValueError(f"keep must be None, 'full' or '8bit', got {keep!r}")
    if stream is None:
        out = _t.fast().gated_ff(x, w_gate, w_up, act, KEEP[keep])
        if out is not None:
            _t.checked(out, "sgemm_gated_ff_forward")
            h, gate, up, gs, us = out
            if keep == "8bit":
                gate, up = Act8._of(gate, gs, *h.shape), Act8._of(up, us, *h.shape)
            return h if keep is None else (h, (gate, up))
    call = _t.Call(_t.cuda_tensor(x, "x").device, stream)
    dt, ldx = _dtype(x, "x"), _t.row_ld(x, "x")
    M = x.shape[0]
    N, K, ldg, ldu = _layer(x, "x", w_gate, w_up, x.shape[1])
    h = call.empty((M, N), x.dtype)
    kept, ldk, at = None, N, (None, None, None, None)
    if keep == "full":
        ldk = -(-N // 8) * 8               # rows that the kernels read in whole vectors
        kept = tuple(call.empty((M, ldk), x.dtype)[:, :N] for _ in range(2))
        at = (kept[0].data_ptr(), kept[1].data_ptr(), None, None)
    elif keep == "8bit":
        kept = tuple(Act8._new(call, M, N) for _ in range(2))
        (gate, gs), (up, us) = (q._addresses() for q in kept)
        at = (gate, up, gs, us)
    packed = _packed(_X, x, ldx) | _packed(_GATE, w_gate, ldg) | _packed(_UP, w_up, ldu)
    if M <= _FEW_TOKENS and keep != "8bit":
        packed = 0
    ws, size = _workspace(call, M, N, K, 0, packed)
    call.run("sgemm_gated_ff_forward", M, N, K, dt, act, x.data_ptr(), ldx, w_gate.data_ptr(), ldg,
             w_up.data_ptr(), ldu, h.data_ptr(), N, KEEP[keep], at[0], at[1], ldk, at[2], at[3],
             _t.ptr(ws), size)
    return h if kept is None else (h, kept)


def gated_ff_backward(dh, x, w_gate, w_up, kept, *, activation: str = "silu",
                      return_h: bool = False, stream=None):
    """(dx, dw_gate, dw_up) of ``gated_ff`` from the gradient of h.  ``x`` is the block's input
    or an ``Act8`` of it, ``kept`` what ``gated_ff(..., keep=...)`` returned.  With ``return_h``
    also h, made again from what was kept: (dx, dw_gate, dw_up, h).  Gradients are of dh's type; the
    gradients of the pre-activations, which the products multiply, are rounded to it too, float16
    with powers of two that keep float32's range.  The numbers of an ``Act8`` x are taken whole, in
    two parts (``include/sgemm.h``)."""
    act = _activation(activation)
    if not isinstance(kept, (tuple, list)) or len(kept) != 2:
        raise TypeError("kept must be the (gate, up) that gated_ff(..., keep=...) returned")
    gate, up = kept
    in8 = isinstance(gate, Act8)
    if in8 != isinstance(up, Act8):
        raise TypeError("gate and up must be kept in one form")
    if stream is None:
        held_x = (None, x._codes, x._scales) if isinstance(x, Act8) else (x, None, None)
        held_k = (gate._codes, up._codes, gate._scales, up._scales) if in8 else \
            (gate, up, None, None)
        fits = not in8 or gate.shape == up.shape == getattr(dh, "shape", None)
        if held_x[0] is not x:             # (the library's rows are padded: it sees no width)
            fits = fits and x.shape[1:] == getattr(w_gate, "shape", ())[1:]
        out = _t.fast().gated_ff_backward(dh, *held_x, w_gate, w_up, *held_k, act, return_h) \
            if fits else None
        if out is not None:
            _t.checked(out, "sgemm_gated_ff_backward")
            return out if return_h else out[:3]
    call = _t.Call(_t.cuda_tensor(dh, "dh").device, stream)
    dt, lddh = _dtype(dh, "dh"), _t.row_ld(dh, "dh")
    N, K, ldg, ldu = _layer(dh, "dh", w_gate, w_up)
    M = dh.shape[0]
    if dh.shape[1] != N:
        raise ValueError(f"dh must be ({M}, {N}), got {tuple(dh.shape)}")
    x_codes = x_scales = x_at = None
    ldx = K
    packed = _packed(_GATE, w_gate, ldg) | _packed(_UP, w_up, ldu)
    if dh.dtype == torch.float16:
        packed |= _FP16
    if isinstance(x, Act8):
        x_codes, x_scales = held(x, "x", (M, K), dh.device)
        packed |= _X
    else:
        ldx = _t.matrix(x, "x", (M, K), dh.dtype, dh.device)
        x_at = x.data_ptr()
        packed |= _packed(_X, x, ldx)
    ldk, gs, us = N, None, None
    if in8:
        form = KEEP["8bit"]
        (g_at, gs), (u_at, us) = (held(q, n, (M, N), dh.device) for q, n in
                                  ((gate, "gate"), (up, "up")))
    else:
        form = KEEP["full"]
        ldk = _t.matrix(gate, "gate", (M, N), dh.dtype, dh.device)
        if _t.matrix(up, "up", (M, N), dh.dtype, dh.device) != ldk:
            raise ValueError("gate and up must have one row stride")
        g_at, u_at = gate.data_ptr(), up.data_ptr()
    dx = call.empty((M, K), dh.dtype)
    dwg, dwu = (call.empty((N, K), dh.dtype) for _ in range(2))
    h = call.empty((M, N), dh.dtype) if return_h else None
    ws, size = _workspace(call, M, N, K, 1, packed)
    call.run("sgemm_gated_ff_backward", M, N, K, dt, act, dh.data_ptr(), lddh, x_at, ldx, x_codes,
             x_scales, w_gate.data_ptr(), ldg, w_up.data_ptr(), ldu, form, g_at, u_at, ldk, gs, us,
             dx.data_ptr(), K, dwg.data_ptr(), K, dwu.data_ptr(), K, _t.ptr(h), N, _t.ptr(ws), size)
    return (dx, dwg, dwu, h) if return_h else (dx, dwg, dwu)
