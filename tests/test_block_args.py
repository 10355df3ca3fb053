"""The C entry points of the 4-bit operands and the norms refuse bad arguments before
they touch the GPU (no device needed: the addresses are never used)."""
import ctypes

import pytest

P = 1 << 20          # fake device addresses, far apart
A, B, C, D, E, F, G, H = (P + i * (1 << 40) for i in range(8))
F32, BF16, F16, NV, MX = 0, 1, 2, 0, 1


def sizes(lib, rows, cols, fmt):
    c, s = ctypes.c_size_t(0), ctypes.c_size_t(0)
    return lib.sgemm_mx4_sizes(rows, cols, fmt, ctypes.byref(c), ctypes.byref(s)), c.value, s.value


def test_sizes(lib):
    assert sizes(lib, 1, 1, NV) == (0, 128 * 64, 128 * 8)
    assert sizes(lib, 129, 4096, NV) == (0, 256 * 2048, 256 * 256)
    assert sizes(lib, 128, 4097, MX) == (0, 128 * 4224 // 2, 128 * 4224 // 32)
    assert sizes(lib, 0, 64, MX) == (0, 0, 0) and sizes(lib, 64, 0, MX) == (0, 0, 0)
    assert sizes(lib, 2**30, 2**30, NV)[1] == 2**59
    assert sizes(lib, -1, 4, NV)[0] == -1 and sizes(lib, 4, 4, 2)[0] == -1
    assert sizes(lib, 2**30 + 1, 4, NV)[0] == -4
    assert lib.sgemm_mx4_sizes(4, 4, NV, None, None) == -1


def test_shapes_match_sizes(lib):
    import math
    from dense_fp32_gemm_09_gb300.mx4 import mx4_shapes
    for rows, cols in ((1, 1), (128, 128), (129, 4097), (1000, 96), (0, 5)):
        for fmt, code in (("nvfp4", NV), ("mxfp4", MX)):
            shapes = mx4_shapes(rows, cols, fmt)
            assert (0, *map(math.prod, shapes)) == sizes(lib, rows, cols, code)


@pytest.mark.parametrize("args,status", [
    ((0, -1, 4, F32, A, 4, NV, None, B, C), -1),
    ((0, 2**30 + 1, 4, F32, A, 4, NV, None, B, C), -4),
    ((2, 4, 4, F32, A, 4, NV, None, B, C), -1),
    ((0, 4, 4, 7, A, 4, NV, None, B, C), -1),
    ((0, 4, 4, F32, A, 4, 5, None, B, C), -1),
    ((0, 4, 8, F32, A, 7, NV, None, B, C), -1),          # ld below the row width
    ((1, 8, 4, F32, A, 7, NV, None, B, C), -1),          # stored 4 x 8
    ((0, 4, 4, F32, None, 4, NV, None, B, C), -1),
    ((0, 4, 4, F32, A, 4, NV, None, None, C), -1),
    ((0, 4, 4, F32, A, 4, NV, None, B, None), -1),
    ((0, 4, 4, F32, A + 2, 4, NV, None, B, C), -1),      # not aligned to its elements
    ((0, 4, 4, BF16, A + 1, 4, NV, None, B, C), -1),
    ((0, 4, 4, F32, A, 4, NV, None, B + 8, C), -1),      # codes not 16-byte aligned
    ((0, 4, 4, F32, A, 4, MX, D, B, C), -1),             # mxfp4 has no tensor scale
    ((0, 4, 4, F32, A, 4, NV, None, A, C), -1),          # codes over X
    ((0, 4, 4, F32, A, 4, NV, None, B, B + 4096), -1),   # scales over codes
])
def test_quantize_refusals(lib, args, status):
    assert lib.sgemm_mx4_quantize(*args, None) == status
    assert lib.sgemm_last_error() != b""


@pytest.mark.parametrize("args,status", [
    ((4, -1, 4, NV, 1.0, A, B, None, C, D, None, 0.0, F32, E, 4), -1),
    ((4, 4, 4, 9, 1.0, A, B, None, C, D, None, 0.0, F32, E, 4), -1),
    ((4, 4, 4, NV, 1.0, A, B, None, C, D, None, 0.0, 9, E, 4), -1),
    ((4, 4, 4, NV, 1.0, A, B, None, C, D, None, 0.0, F32, E, 3), -1),
    ((4, 4, 4, NV, 1.0, None, B, None, C, D, None, 0.0, F32, E, 4), -1),
    ((4, 4, 4, NV, 1.0, A, B, None, C, None, None, 0.0, F32, E, 4), -1),
    ((4, 4, 4, NV, 1.0, A, B, None, C, D, None, 0.0, F32, None, 4), -1),
    ((4, 4, 4, NV, float("nan"), A, B, None, C, D, None, 0.0, F32, E, 4), -1),
    ((4, 4, 4, NV, 1.0, A, B, None, C, D, None, float("nan"), F32, E, 4), -1),
    ((4, 4, 4, NV, 1.0, A, B, None, C, D, None, 0.0, F32, A + 64, 4), -1),   # C over A
    ((4, 4, 4, NV, 1.0, A, B, F, C, D, None, 0.0, F32, F, 4), -1),           # C over a scale
    ((4, 4, 4, MX, 1.0, A, B, F, C, D, None, 0.0, F32, E, 4), -1),
    ((2**30 + 1, 4, 4, NV, 1.0, A, B, None, C, D, None, 0.0, F32, E, 4), -4),
])
def test_matmul_refusals(lib, args, status):
    assert lib.sgemm_mx4_matmul(*args, None) == status
    assert lib.sgemm_last_error() != b""


def forward(lib, rows=4, cols=8, dtype=F32, block=A, ldb=8, res=B, ldr=8, w=None, nw=None, wt=F32,
            gate=None, ldg=0, scale=1.0, eps=1e-6, y=C, ldy=8, rstd=D, next=1, h=E, ldh=8,
            nrstd=F, fmt=-1, ts=None, codes=None, scales=None):
    return lib.sgemm_norm_forward(rows, cols, dtype, block, ldb, res, ldr, w, nw, wt, gate, ldg,
                                  scale, eps, y, ldy, rstd, next, h, ldh, nrstd, fmt, ts, codes,
                                  scales, None)


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(cols=0), dict(dtype=3), dict(wt=-1), dict(eps=-1.0), dict(eps=float("inf")),
    dict(scale=float("nan")), dict(next=2), dict(res=None), dict(y=None), dict(rstd=None),
    dict(block=None), dict(next=0), dict(h=None), dict(nrstd=None), dict(fmt=4), dict(fmt=NV),
    dict(fmt=NV, h=None), dict(fmt=MX, h=None, codes=G, scales=H, ts=P), dict(ldb=7), dict(ldh=3),
    dict(gate=P, ldg=5), dict(y=B), dict(h=A), dict(h=C), dict(rstd=F), dict(block=A + 2),
    dict(fmt=NV, h=None, codes=G + 4, scales=H), dict(ts=P),
])
def test_forward_refusals(lib, change):
    assert forward(lib, **change) == -1
    assert lib.sgemm_last_error() != b""


def test_forward_limits(lib):
    assert forward(lib, rows=2**30 + 1) == -4
    assert forward(lib, rows=0, block=None) == 0


def backward(lib, rows=4, cols=8, dtype=F32, dy=A, lddy=8, dh=B, lddh=8, y=C, ldy=8, nrstd=D, nw=None,
             block=E, ldb=8, rstd=F, w=None, wt=F32, gate=None, ldg=0, scale=1.0, dx=G, lddx=8,
             dblock=H, lddb=8, dgate=None, lddg=8, dw=None, dnw=None):
    return lib.sgemm_norm_backward(rows, cols, dtype, dy, lddy, dh, lddh, y, ldy, nrstd, nw, block,
                                   ldb, rstd, w, wt, gate, ldg, scale, dx, lddx, dblock, lddb, dgate,
                                   lddg, dw, dnw, None)


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(cols=0), dict(dtype=9), dict(wt=9), dict(scale=float("inf")),
    dict(dy=None, dh=None), dict(dh=None, dnw=P), dict(y=None), dict(nrstd=None), dict(dx=None),
    dict(rstd=None), dict(dblock=None), dict(block=None), dict(block=None, dblock=None, dw=P),
    dict(dgate=P), dict(lddy=7), dict(lddx=7), dict(dx=A), dict(dblock=G), dict(dw=E),
    dict(dw=P, dnw=P), dict(dy=A + 1), dict(dh=None, block=None, dblock=None),
])
def test_backward_refusals(lib, change):
    assert backward(lib, **change) == -1
    assert lib.sgemm_last_error() != b""


def test_binding_names():
    import dense_fp32_gemm_09_gb300 as sg
    for name in sg.__all__:
        assert getattr(sg, name) is not None
    with pytest.raises(AttributeError):
        sg.no_such_operator
