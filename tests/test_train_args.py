"""The C entry points of the 8-bit checkpoints, layer norm and the gated feed-forward block refuse
bad arguments before they touch the GPU (no device needed: the addresses are never used)."""
import ctypes

import pytest

P = 1 << 20          # fake device addresses, far apart
A, B, C, D, E, F, G, H, I, J, K, L = (P + i * (1 << 40) for i in range(12))
F32, BF16, F16 = 0, 1, 2


def two(fn, *args):
    a, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    return fn(*args, ctypes.byref(a), ctypes.byref(b)), a.value, b.value


def test_act8_sizes(lib):
    assert two(lib.sgemm_act8_sizes, 1, 1) == (0, 64, 4)
    assert two(lib.sgemm_act8_sizes, 3, 65) == (0, 384, 24)
    assert two(lib.sgemm_act8_sizes, 0, 64) == (0, 0, 0) and two(lib.sgemm_act8_sizes, 9, 0) == (0, 0, 0)
    assert two(lib.sgemm_act8_sizes, 2**30, 2**30)[1] == 2**60
    assert two(lib.sgemm_act8_sizes, -1, 4)[0] == -1
    assert two(lib.sgemm_act8_sizes, 4, 2**30 + 1)[0] == -4
    assert lib.sgemm_act8_sizes(4, 4, None, None) == -1


def test_act8_shapes_match_sizes(lib):
    import math
    from dense_fp32_gemm_09_gb300.act8 import act8_shapes
    for rows, cols in ((1, 1), (7, 64), (129, 4097), (0, 5)):
        codes, scales = map(math.prod, act8_shapes(rows, cols))
        assert two(lib.sgemm_act8_sizes, rows, cols) == (0, codes, 4 * scales)


@pytest.mark.parametrize("args,status", [
    ((-1, 4, F32, A, 4, B, C), -1), ((2**30 + 1, 4, F32, A, 4, B, C), -4),
    ((4, 4, 5, A, 4, B, C), -1), ((4, 8, F32, A, 7, B, C), -1), ((4, 4, F32, None, 4, B, C), -1),
    ((4, 4, F32, A, 4, None, C), -1), ((4, 4, F32, A, 4, B, None), -1),
    ((4, 4, F32, A + 2, 4, B, C), -1), ((4, 4, BF16, A + 1, 4, B, C), -1),
    ((4, 4, F32, A, 4, B + 8, C), -1), ((4, 4, F32, A, 4, B, C + 4), -1),
    ((4, 4, F32, A, 4, A + 16, C), -1), ((4, 4, F32, A, 4, B, B + 128), -1),
])
def test_act8_quantize_refusals(lib, args, status):
    assert lib.sgemm_act8_quantize(*args, None) == status
    assert lib.sgemm_last_error() != b""


@pytest.mark.parametrize("args,status", [
    ((-1, 4, A, B, F32, C, 4), -1), ((4, 2**30 + 1, A, B, F32, C, 4), -4),
    ((4, 4, A, B, 9, C, 4), -1), ((4, 4, A, B, F32, C, 3), -1), ((4, 4, None, B, F32, C, 4), -1),
    ((4, 4, A, None, F32, C, 4), -1), ((4, 4, A, B, F32, None, 4), -1),
    ((4, 4, A + 4, B, F32, C, 4), -1), ((4, 4, A, B, F32, A, 4), -1), ((4, 4, A, B, F16, C + 1, 4), -1),
])
def test_act8_dequantize_refusals(lib, args, status):
    assert lib.sgemm_act8_dequantize(*args, None) == status
    assert lib.sgemm_last_error() != b""


def test_nothing_to_do(lib):
    assert lib.sgemm_act8_quantize(0, 4, F32, None, 4, None, None, None) == 0
    assert lib.sgemm_act8_dequantize(4, 0, None, None, F32, None, 1, None) == 0
    assert forward(lib, rows=0, x=None, y=None) == 0
    assert ff_forward(lib, M=0, x=None, h=None) == 0


def forward(lib, rows=4, cols=8, dtype=F32, x=A, ldx=8, w=None, b=None, wt=F32, eps=1e-5, y=B, ldy=8,
            mean=C, rstd=D, codes=None, scales=None):
    return lib.sgemm_layer_norm_forward(rows, cols, dtype, x, ldx, w, b, wt, eps, y, ldy, mean, rstd,
                                        codes, scales, None)


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(cols=0), dict(dtype=3), dict(wt=7), dict(eps=-1.0), dict(eps=float("inf")),
    dict(eps=float("nan")), dict(x=None), dict(y=None), dict(mean=None), dict(rstd=None),
    dict(ldx=7), dict(ldy=7), dict(y=A), dict(mean=D), dict(codes=E), dict(scales=E),
    dict(codes=E + 4, scales=F), dict(codes=B, scales=F), dict(x=A + 1), dict(w=B), dict(w=E + 2),
    dict(b=B), dict(b=E + 1, wt=BF16), dict(rows=2, codes=E, scales=E + 64),
])
def test_layer_norm_refusals(lib, change):
    assert forward(lib, **change) == -1
    assert lib.sgemm_last_error() != b""


def backward(lib, rows=4, cols=8, dtype=F32, dh=A, lddh=8, dy=None, lddy=8, x=B, ldx=8, codes=None,
             scales=None, mean=C, rstd=D, w=None, wt=F32, dx=E, lddx=8, dw=None, db=None, ws=None, n=0):
    return lib.sgemm_layer_norm_backward(rows, cols, dtype, dh, lddh, dy, lddy, x, ldx, codes, scales,
                                         mean, rstd, w, wt, dx, lddx, dw, db, ws, n, None)


@pytest.mark.parametrize("change", [
    dict(rows=-1), dict(cols=0), dict(dtype=3), dict(wt=-1), dict(dh=None), dict(x=None),
    dict(codes=F, scales=G), dict(x=None, codes=F), dict(x=None, scales=G), dict(mean=None),
    dict(rstd=None), dict(dx=None), dict(lddh=7), dict(lddy=7, dy=F), dict(ldx=3), dict(lddx=3),
    dict(dx=A), dict(dx=B), dict(dy=E), dict(dw=E), dict(dw=F, db=F), dict(dh=A + 2),
    dict(x=None, codes=F + 8, scales=G), dict(w=E),
])
def test_layer_norm_backward_refusals(lib, change):
    assert backward(lib, **change) == -1
    assert lib.sgemm_last_error() != b""


def test_limits(lib):
    assert forward(lib, rows=2**30 + 1) == -4 and backward(lib, rows=2**30 + 1) == -4
    assert ff_forward(lib, M=2**30 + 1) == -4 and ff_backward(lib, K=2**30 + 1) == -4
    assert lib.sgemm_layer_norm_backward_workspace(4, -1, ctypes.byref(ctypes.c_size_t())) == -1
    assert lib.sgemm_layer_norm_backward_workspace(4, 4, None) == -1


def ff_forward(lib, M=4, N=8, K=16, dtype=BF16, act=0, x=A, ldx=16, wg=B, ldg=16, wu=C, ldu=16, h=D,
               ldh=8, keep=0, gate=None, up=None, ldk=8, gs=None, us=None, ws=None, n=0):
    return lib.sgemm_gated_ff_forward(M, N, K, dtype, act, x, ldx, wg, ldg, wu, ldu, h, ldh, keep, gate,
                                      up, ldk, gs, us, ws, n, None)


@pytest.mark.parametrize("change", [
    dict(M=-1), dict(N=0), dict(K=0), dict(dtype=F32), dict(dtype=4), dict(act=2), dict(act=-1),
    dict(keep=3), dict(keep=-1), dict(x=None), dict(wg=None), dict(wu=None), dict(h=None),
    dict(ldx=15), dict(ldg=15), dict(ldu=15), dict(ldh=7), dict(x=A + 1), dict(h=A), dict(h=B),
    dict(gate=E), dict(keep=1), dict(keep=1, gate=E, up=E), dict(keep=1, gate=E, up=F, ldk=7),
    dict(keep=1, gate=E, up=F, gs=G), dict(keep=1, gate=D, up=F), dict(keep=2, gate=E, up=F),
    dict(keep=2, gate=E, up=F, gs=G), dict(keep=2, gate=E, up=F, gs=G, us=G),
    dict(keep=2, gate=E + 8, up=F, gs=G, us=H), dict(keep=2, gate=A, up=F, gs=G, us=H),
])
def test_gated_ff_refusals(lib, change):
    assert ff_forward(lib, **change) == -1
    assert lib.sgemm_last_error() != b""


def ff_backward(lib, M=4, N=8, K=16, dtype=BF16, act=0, dh=A, lddh=8, x=B, ldx=16, xc=None, xs=None,
                wg=C, ldg=16, wu=D, ldu=16, keep=1, gate=E, up=F, ldk=8, gs=None, us=None, dx=G,
                lddx=16, dwg=H, lddwg=16, dwu=I, lddwu=16, h=None, ldh=8, ws=None, n=0):
    return lib.sgemm_gated_ff_backward(M, N, K, dtype, act, dh, lddh, x, ldx, xc, xs, wg, ldg, wu, ldu,
                                       keep, gate, up, ldk, gs, us, dx, lddx, dwg, lddwg, dwu, lddwu, h,
                                       ldh, ws, n, None)


@pytest.mark.parametrize("change", [
    dict(M=-1), dict(N=0), dict(K=0), dict(dtype=F32), dict(act=2), dict(keep=0), dict(keep=3),
    dict(dh=None), dict(x=None), dict(xc=J, xs=K), dict(x=None, xc=J), dict(x=None, xc=J + 8, xs=K),
    dict(wg=None), dict(wu=None), dict(gate=None), dict(up=None), dict(dx=None), dict(dwg=None),
    dict(dwu=None), dict(lddh=7), dict(ldx=15), dict(ldg=15), dict(ldk=7), dict(lddx=15),
    dict(lddwg=15), dict(lddwu=15), dict(h=J, ldh=7), dict(dx=A), dict(dwg=C), dict(dwu=H), dict(h=E),
    dict(keep=2), dict(keep=2, gs=J), dict(gs=J), dict(keep=2, gs=J, us=K, gate=E + 4), dict(dx=G + 1),
])
def test_gated_ff_backward_refusals(lib, change):
    assert ff_backward(lib, **change) == -1
    assert lib.sgemm_last_error() != b""


def test_gated_ff_workspace(lib):
    n = ctypes.c_size_t(0)
    ask = lambda *a: lib.sgemm_gated_ff_workspace(*a, ctypes.byref(n))
    assert ask(0, 8, 8, 0, 0) == 0 and n.value == 0
    for bad in ((-1, 8, 8, 0, 0), (8, 0, 8, 0, 0), (8, 8, 0, 1, 0), (8, 8, 8, 2, 0), (8, 8, 8, 0, 8),
                (8, 8, 8, 0, -1)):
        assert ask(*bad) == -1
    assert lib.sgemm_gated_ff_workspace(8, 8, 8, 0, 0, None) == -1
    sizes = []
    for packed in range(8):
        assert ask(100, 200, 300, 1, packed) == 0
        sizes.append(n.value)
    assert all(sizes[a | b] >= sizes[a] for a in range(8) for b in range(8))
    assert sizes[0] >= 2 * 100 * 200 * 2 and sizes[1] >= sizes[0] + 100 * 300 * 2
