"""Argument checks and allocation shared by the 4-bit and norm entry points."""
from __future__ import annotations

import torch

from ._abi import check, load

DTYPE_CODES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
INT_MAX = 2**31 - 1

# The public forms of these two build objects around the same numbers (a few microseconds
# on a call of ten).
_current_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def dtype_code(dtype, name: str) -> int:
    code = DTYPE_CODES.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be float32, bfloat16 or float16, got {dtype}")
    return code


def cuda_tensor(t, name: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t


def row_ld(t, name: str) -> int:
    """Leading dimension of a 2-D view whose rows have unit stride and do not overlap."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = t.shape
    step, unit = t.stride()
    if unit == 1 and cols <= step <= INT_MAX and 1 < rows <= INT_MAX:      # the usual case
        return step
    if cols > 1 and unit != 1:
        raise ValueError(f"{name} must have unit stride along its columns")
    if rows > 1 and step < cols:
        raise ValueError(f"{name}: its rows overlap (row stride {step} < row width {cols})")
    ld = max(step, cols, 1) if rows > 1 else max(cols, 1)
    if ld > INT_MAX or rows > INT_MAX:
        raise ValueError(f"{name}: a size or stride does not fit the library's 32-bit ints")
    return ld


def matrix(t, name: str, shape=None, dtype=None, device=None) -> int:
    """Checks a 2-D CUDA operand against what the call expects; its leading dimension."""
    cuda_tensor(t, name)
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    same_device(t, name, device)
    return row_ld(t, name)


def vector(t, name: str, n: int, dtype=None, device=None):
    cuda_tensor(t, name)
    if t.dim() != 1 or t.shape[0] != n:
        raise ValueError(f"{name} must have shape ({n},), got {tuple(t.shape)}")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    same_device(t, name, device)
    return t


def same_device(t, name: str, device) -> None:
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def one_float(t, name: str, device):
    """A one-element float32 tensor on `device`, or None."""
    if t is None:
        return None
    cuda_tensor(t, name)
    if t.numel() != 1 or t.dtype != torch.float32:
        raise TypeError(f"{name} must be one float32 number")
    same_device(t, name, device)
    return t


def ptr(t):
    return None if t is None else t.data_ptr()


_fast = None


def fast():
    """The compiled binding of the usual calls: each returns its outputs, a status of the
    library where that is not 0, or None for a call that is not of the usual form."""
    global _fast
    if _fast is None:
        import ctypes
        import importlib.machinery
        import importlib.util
        import os

        from . import build
        lib = load()
        path = build.fast_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build the library for this torch first "
                               "(python -m dense_fp32_gemm_09_gb300.build)")
        loader = importlib.machinery.ExtensionFileLoader("_fast_calls", path)
        module = importlib.util.module_from_spec(
            importlib.util.spec_from_loader("_fast_calls", loader))
        loader.exec_module(module)
        module.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in (
            "sgemm_mx4_quantize", "sgemm_mx4_dequantize", "sgemm_mx4_matmul",
            "sgemm_norm_forward", "sgemm_norm_backward_ws", "sgemm_norm_backward_workspace")))
        _fast = module
    return _fast


def checked(result, name: str) -> None:
    """Raises where a fast call returned a status instead of its outputs."""
    if type(result) is int:
        check(result, name)


_functions = {}


def function(name: str):
    """The library's entry point `name` (looked up once)."""
    fn = _functions.get(name)
    if fn is None:
        fn = _functions[name] = getattr(load(), name)
    return fn


class Call:
    """Device and stream of one library call.  Buffers that the call returns are
    allocated for the stream that writes them."""

    __slots__ = ("device", "index", "handle", "given")

    def __init__(self, device, stream):
        self.device = device
        self.index = device.index
        self.given = stream
        if stream is None:
            self.handle = _current_stream(self.index)
        else:
            self.handle = int(getattr(stream, "cuda_stream", stream))

    def empty(self, shape, dtype):
        if self.given is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        s = self.given
        if not isinstance(s, torch.cuda.Stream):
            s = torch.cuda.ExternalStream(self.handle, device=self.device) if self.handle else \
                torch.cuda.default_stream(self.device)
        with torch.cuda.stream(s):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def run(self, name: str, *args) -> None:
        fn = _functions.get(name) or function(name)
        if _current_device() == self.index:
            status = fn(*args, self.handle)
        else:
            with torch.cuda.device(self.device):
                status = fn(*args, self.handle)
        if status:
            check(status, name)
