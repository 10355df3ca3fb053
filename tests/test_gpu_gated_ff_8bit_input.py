"""The weights' gradients of the feed-forward block from an input in 8 bits: of the numbers that it holds,
code * scale, not of their roundings to the block's type.

The products take an input as its rounding and the rounding of what is left: off by u^2 of itself
(u = 2^-8 of bf16, 2^-11 of fp16, half a step), in fp16 by 2^-25 at least."""
import pytest
import torch

from test_gpu_gated_ff import DTYPES, MANY, SHAPES, T, U, Case, depth, near
from test_gpu_gated_ff_far_gates import activation

pytestmark = pytest.mark.gpu


@pytest.fixture()
def sg(cuda):
    import dense_fp32_gemm_09_gb300 as sg
    return sg


def held(sg, x):
    """An input and the numbers that its 8 bits hold."""
    q = sg.act8_quantize(x)
    return q, q.dequantize().double()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("K", [1, 64, 65, 777, 1000, 4096])
def test_one_token(sg, dtype, K):
    """dg = 3 and du = 192 to the bit, so dw is the one product 3 x or 192 x, rounded once: the nearest number,
    or its neighbour where 3 x is within 2 u^2 of itself of the middle of two, which are 2 u (or 4 u) of
    it apart: one of 1 / u numbers at most."""
    dt, N = DTYPES[dtype], 24
    q, x = held(sg, torch.randn(1, K, device="cuda", generator=torch.Generator("cuda").manual_seed(K)).float() + 1.5)
    one = lambda v: torch.full((1, N), v, device="cuda", dtype=dt)
    w = torch.zeros(N, K, device="cuda", dtype=dt)
    _, dwg, dwu = sg.gated_ff_backward(one(3), q, w, w, (one(64), one(1)))
    for got, by in ((dwg, 3), (dwu, 192)):
        want = (by * x).to(dt)
        off = (got.double() - want.double()).abs()
        step = torch.finfo(dt).eps * want.double().abs() * 1.01
        assert bool((off <= step).all())
        assert int((off[0] > 0).sum()) <= max(1, 2 * K * U[dtype] * 4)


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("M,N,K", [(300, 520, 136), (500, 1024, 512), (900, 100, 6000), (1000, 640, 1001), (4000, 64, 320)])
def test_two_roundings_and_no_third(sg, M, N, K, dtype, name):
    """Against 64 bits, in norm: the rounding of the terms (dg, du) and that of the result are
    independent and of one size, so the error is 2^(1/2) of a result's that is rounded once; with the
    input rounded too it would be 3^(1/2), 1.73."""
    c = Case(M, N, K, dtype)
    q, x = held(sg, c.x)
    _, kept = sg.gated_ff(c.x, c.wg, c.wu, activation=name, keep="8bit")
    got = sg.gated_ff_backward(c.dh, q, c.wg, c.wu, kept, activation=name)
    g, u = (k.dequantize().double() for k in kept)
    a, slope = activation(g, name)
    dh = c.dh.double()
    for out, d in ((got[1], dh * u * slope), (got[2], dh * a)):
        want = d.t() @ x
        off, once = (out.double() - want).norm(), (want.to(c.dt).double() - want).norm()
        assert float(off / once) < 1.5


def check(sg, c, name="silu"):
    q, x = held(sg, c.x)
    _, kept = sg.gated_ff(c.x, c.wg, c.wu, activation=name, keep="full")
    got = sg.gated_ff_backward(c.dh, q, c.wg, c.wu, kept, activation=name)
    g, u = (k.double() for k in kept)
    a, slope = activation(g, name)
    dh = c.dh.double()
    for out, d, off in ((got[1], dh * u * slope, 2.0 ** -17 * (dh * u).abs()), (got[2], dh * a, 2.0 ** -19 * (dh * a).abs())):
        want = d.t() @ x
        ed = c.u * 1.01 * d.abs() + off + 2.0 ** -39 * d.abs().amax(0)
        ex = c.u ** 2 * 1.02 * x.abs() + T[dtype_of(c)]
        tol = ed.t() @ (x.abs() + ex) + d.abs().t() @ ex + depth(2 * c.M) * (d.abs().t() @ x.abs())
        near(out, want, tol * 1.01 + c.u * 1.01 * (want.abs() + tol) + c.t, "dw")


def dtype_of(c):
    return "bf16" if c.dt == torch.bfloat16 else "fp16"


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("M,N,K", SHAPES + MANY)
def test_every_shape(sg, M, N, K, dtype):
    """Tiles and parts of both halves of the contraction."""
    check(sg, Case(M, N, K, dtype))


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_no_third_term_of_infinities(sg, dtype):
    """A NaN block of x is NaN in its columns of the weights' gradients, and nowhere else."""
    c = Case(70, 96, 200, dtype)
    x = c.x.clone()
    x[5, 70] = float("inf")
    _, kept = sg.gated_ff(c.x, c.wg, c.wu, keep="full")
    got = sg.gated_ff_backward(c.dh, sg.act8_quantize(x), c.wg, c.wu, kept)
    want = sg.gated_ff_backward(c.dh, sg.act8_quantize(c.x), c.wg, c.wu, kept)
    cols = [i for i in range(200) if not 64 <= i < 128]
    assert torch.equal(got[0], want[0])
    for a, b in zip(got[1:], want[1:]):
        assert torch.equal(a[:, cols], b[:, cols]) and bool(a[:, 64:128].isnan().all())


@pytest.mark.parametrize("dtype,code", [("bf16", 1), ("fp16", 2)])
@pytest.mark.parametrize("M,N,K", [(1, 8, 64), (13, 71, 133), (300, 200, 136), (700, 96, 1000), (5000, 40, 72)])
def test_workspace(sg, M, N, K, dtype, code):
    """Through the C entry, with exactly what sgemm_gated_ff_workspace says for an x in 8 bits."""
    import ctypes
    lib, s, c = sg.load(), torch.cuda.current_stream().cuda_stream, Case(M, N, K, dtype)
    q = sg.act8_quantize(c.x)
    _, kept = sg.gated_ff(c.x, c.wg, c.wu, keep="full")
    g, u = (t.contiguous() for t in kept)
    want = sg.gated_ff_backward(c.dh, q, c.wg, c.wu, kept)
    out = [torch.empty_like(t) for t in want]
    n = ctypes.c_size_t(0)
    bits = 1 | (6 if K % 8 and N > 1 else 0) | (8 if code == 2 else 0)
    assert lib.sgemm_gated_ff_workspace(M, N, K, 1, bits, ctypes.byref(n)) == 0
    ws = torch.full((n.value + 256,), 255, dtype=torch.uint8, device="cuda")
    args = (M, N, K, code, 0, c.dh.data_ptr(), N, None, K, q.codes.data_ptr(), q.scales.data_ptr(), c.wg.data_ptr(), K,
            c.wu.data_ptr(), K, 1, g.data_ptr(), u.data_ptr(), N, None, None, out[0].data_ptr(), K, out[1].data_ptr(), K,
            out[2].data_ptr(), K, None, 0, ws.data_ptr())
    assert lib.sgemm_gated_ff_backward(*args, n.value - 1, s) == -6
    assert lib.sgemm_gated_ff_backward(*args, n.value, s) == 0
    torch.cuda.synchronize()
    assert bool((ws[n.value:] == 255).all())
    assert all(torch.equal(a, b) for a, b in zip(out, want))
