"""The feed-forward block's gradient in fp16 where the gradients of the pre-activations, dg and du,
are outside the numbers that fp16 holds though dx and the weights' gradients are not.

Tolerances.  The products take each row of (dg, du), for dx, and each column of dg and of du, for the
weights' gradients, times a power of two that brings its largest magnitude to 2^14 at least: a number is
off by half a step, 2^-11 of it, or by half of fp16's smallest number, 2^-25, beside 2^14: 2^-39 of
the largest.  The sigmoid s of z is off by rel = (3 + 3.2 |z|) 2^-23 + 2^-20 of itself for z < 0, by that of
1 - s for z > 0 (CUDA's bound for the fast exponential, 2 + 1.173 |z| steps; z's own roundings; a reciprocal
and a few products); 1 - s by as much, and its rounding, 2^-23, or all of it.  Sums and the last rounding
as in test_gpu_gated_ff.py."""
import pytest
import torch

from test_gpu_gated_ff import depth, near
from test_gpu_gated_ff_far_gates import activation, argument

pytestmark = pytest.mark.gpu
U, T, DT = 2.0 ** -11, 2.0 ** -25, torch.float16


@pytest.fixture()
def sg(cuda):
    import dense_fp32_gemm_09_gb300 as sg
    return sg


def activation_off(g, name):
    """How far the activation and its slope may be off."""
    z, by = argument(g, name)
    s, t = torch.sigmoid(z), torch.sigmoid(-z)
    rel = (3 + 3.2 * z.abs().clamp(max=100)) * 2.0 ** -23 + 2.0 ** -20
    rest = rel * s * t + torch.minimum(torch.full_like(t, 2.0 ** -23), 4 * t)
    rel, steep = rel * t + 2.0 ** -22, (g * by).abs()
    return s * rel * g.abs(), s * (rel * (1 + steep * t) + steep * (rest + 2.0 ** -21 * t) + 2.0 ** -22)


def check(sg, dh, x, wg, wu, g, u, name="silu", kept=None):
    """The gradient against 64 bits; g and u as kept."""
    got = sg.gated_ff_backward(dh, x, wg, wu, kept or (g, u), activation=name)
    x64 = x.dequantize().double() if isinstance(x, sg.Act8) else x.double()
    if kept:
        g, u = (q.dequantize() for q in kept)
    dh, wg, wu, g, u = (t.double() for t in (dh, wg, wu, g, u))
    M, N = dh.shape
    a, slope = activation(g, name)
    dg, du = dh * u * slope, dh * a
    off_a, off_slope = activation_off(g, name)
    off_g, off_u = off_slope * (dh * u).abs(), off_a * dh.abs()
    top = torch.maximum(dg.abs().amax(1), du.abs().amax(1))[:, None]
    want = dg @ wg + du @ wu
    tol = (off_g + U * 1.01 * dg.abs() + 2.0 ** -39 * top) @ wg.abs() + \
        (off_u + U * 1.01 * du.abs() + 2.0 ** -39 * top) @ wu.abs() + \
        depth(2 * N) * (dg.abs() @ wg.abs() + du.abs() @ wu.abs())
    assert float(want.abs().max()) < 6e4
    near(got[0], want, tol * 1.01 + U * 1.01 * (want.abs() + tol) + T, "dx")
    ex = U * 1.01 * x64.abs() + T if isinstance(x, sg.Act8) else torch.zeros_like(x64)
    for out, d, off, what in ((got[1], dg, off_g, "dw_gate"), (got[2], du, off_u, "dw_up")):
        want = d.t() @ x64
        ed = off + U * 1.01 * d.abs() + 2.0 ** -39 * d.abs().amax(0)
        tol = ed.t() @ (x64.abs() + ex) + d.abs().t() @ ex + depth(M) * (d.abs().t() @ x64.abs())
        assert float(want.abs().max()) < 6e4
        near(out, want, tol * 1.01 + U * 1.01 * (want.abs() + tol) + T, what)
    return got


def numbers(seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    return lambda *s: torch.randn(s, generator=gen, device="cuda")


def powers(seed, lo, hi, *shape):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randint(lo, hi + 1, shape, generator=gen, device="cuda").float().exp2()


def test_large(sg):
    """dh = 300 and act(g) = 300: du = 90000."""
    M, N, K = 4, 8, 16
    full = lambda v, *s: torch.full(s, v, dtype=DT, device="cuda")
    check(sg, full(300, M, N), full(2.0 ** -6, M, K), full(2.0 ** -8, N, K), full(2.0 ** -8, N, K),
          full(300, M, N), full(300, M, N))


def test_small(sg):
    """dh = 2^-20: dg and du of 2^-28 and less, times weights and inputs of 2^10."""
    r = numbers(1)
    M, N, K = 300, 520, 72
    dh, u = (powers(2, -22, -19, M, N) * r(M, N).sign()).to(DT), (r(M, N) / 256).to(DT)
    check(sg, dh, (r(M, K) * 1024).to(DT), (r(N, K) * 1024).to(DT), (r(N, K) * 1024).to(DT), (r(M, N) / 64).to(DT), u)


# Few and many tiles, with and without parts of dx's and of the weights' contraction, rows off 16 bytes.
@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 100, 40), (3, 5, 7), (17, 130, 100), (300, 520, 136), (900, 100, 6000),
                                   (9000, 64, 300), (40, 3000, 520), (1000, 4100, 520), (2600, 2100, 200)])
def test_rows_and_columns_of_different_sizes(sg, M, N, K, name):
    """Each row of dh and each column of u of a size of its own: none sets another's precision."""
    r = numbers(M + N + K)
    dh = (r(M, N) * powers(1, -12, 6, M, 1)).to(DT)
    g, u = (r(M, N) * 3 + powers(4, 0, 9, 1, N)).to(DT), (r(M, N) * powers(2, -8, 7, 1, N)).to(DT)
    x, wg, wu = ((r(*s) / 1024).to(DT) for s in ((M, K), (N, K), (N, K)))
    first = check(sg, dh, x, wg, wu, g, u, name)
    again = sg.gated_ff_backward(dh, x, wg, wu, (g, u), activation=name)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    check(sg, dh, sg.act8_quantize(x), wg, wu, None, None, name, (sg.act8_quantize(g), sg.act8_quantize(u)))


def test_one_large_row(sg):
    """A row 2^30 times as large as the others leaves their dx as it is alone."""
    M, N, K = 60, 96, 72
    r = numbers(3)
    dh, u, g = (r(M, N) / 256).to(DT), r(M, N).to(DT), (r(M, N) * 2).to(DT)
    x, wg, wu = ((r(*s) / 1024).to(DT) for s in ((M, K), (N, K), (N, K)))
    dh[7] = (dh[7].double() * 2.0 ** 14).to(DT)
    u[7] = (u[7].double() * 2.0 ** 12).to(DT)
    g[7] = g[7].abs() * 256
    x[7] = x[7] / 1024
    got = sg.gated_ff_backward(dh, x, wg / 64, wu / 64, (g, u))
    others = [i for i in range(M) if i != 7]
    assert torch.isfinite(got[0]).all()
    alone = sg.gated_ff_backward(dh[others], x[others], wg / 64, wu / 64, (g[others], u[others]))
    assert torch.equal(got[0][others], alone[0])


def test_infinities_stay_in_their_row_and_columns(sg):
    M, N, K = 50, 96, 72
    r = numbers(5)
    dh, u, g = r(M, N).to(DT), r(M, N).to(DT), r(M, N).to(DT)
    x, wg, wu = ((r(*s) / 8).to(DT) for s in ((M, K), (N, K), (N, K)))
    want = check(sg, dh, x, wg, wu, g, u)
    dh[4, 9], dh[30, 11] = float("inf"), float("nan")
    got = sg.gated_ff_backward(dh, x, wg, wu, (g, u))
    rows, cols = [i for i in range(M) if i not in (4, 30)], [i for i in range(N) if i not in (9, 11)]
    assert torch.equal(got[0][rows], want[0][rows]) and not bool(torch.isfinite(got[0][[4, 30]]).any())
    for a, b in zip(got[1:], want[1:]):
        assert torch.equal(a[cols], b[cols]) and not bool(torch.isfinite(a[[9, 11]]).any())


def test_zeros(sg):
    """Rows and columns of dh that are zero, and all of it."""
    M, N, K = 40, 200, 64
    r = numbers(6)
    dh, u, g = r(M, N).to(DT), r(M, N).to(DT), r(M, N).to(DT)
    x, wg, wu = ((r(*s) / 8).to(DT) for s in ((M, K), (N, K), (N, K)))
    dh[3] = 0
    dh[:, 100] = 0
    got = check(sg, dh, x, wg, wu, g, u)
    assert not bool(got[0][3].any()) and not bool(got[1][100].any()) and not bool(got[2][100].any())
    for t in sg.gated_ff_backward(torch.zeros_like(dh), x, wg, wu, (g, u)):
        assert not bool(t.any())


def large(seed=7, M=200, N=136, K=72):
    """Everything that a call takes, with dg and du beyond fp16."""
    r = numbers(seed)
    dh, g, u = (r(M, N) * 64).to(DT), (r(M, N) * 16 + 400).to(DT), (r(M, N) * 100).to(DT)
    x, wg, wu = ((r(*s) / 1024).to(DT) for s in ((M, K), (N, K), (N, K)))
    return dh, x, wg, wu, (g, u)


def test_both_ways_into_the_library(sg, monkeypatch):
    args = large()
    want = sg.gated_ff_backward(*args, return_h=True)
    assert all(bool(torch.isfinite(t).all()) for t in want[:3])

    class Nothing:
        def __getattr__(self, name):
            return lambda *a: None

    import dense_fp32_gemm_09_gb300._tensors as tensors
    monkeypatch.setattr(tensors, "_fast", Nothing())
    got = sg.gated_ff_backward(*args, return_h=True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_graphs_and_streams_beside_each_other(sg):
    """The largest magnitudes are the call's own: two graphs and an eager call at once."""
    data = [large(seed) for seed in (7, 8, 9)]
    want = [sg.gated_ff_backward(*a) for a in data]
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in range(3)]
    for a in data[:2]:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(sg.gated_ff_backward(*a))
        graphs.append(graph)
    for _ in range(10):
        for graph, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        with torch.cuda.stream(streams[2]):
            eager = sg.gated_ff_backward(*data[2])
    torch.cuda.synchronize()
    for got, ref in zip(outs + [eager], want):
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (3, 5, 7), (200, 136, 72), (700, 96, 1000)])
def test_workspace(sg, M, N, K):
    """Through the C entry: a workspace of exactly the size asked for, whatever it held, and one of the
    size for bf16 is refused."""
    import ctypes
    lib, s = sg.load(), torch.cuda.current_stream().cuda_stream
    dh, x, wg, wu, (g, u) = large(M + N, M, N, K)
    dx, dwg, dwu = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu)
    size = ctypes.c_size_t(0)

    def need(bits):
        assert lib.sgemm_gated_ff_workspace(M, N, K, 1, bits, ctypes.byref(size)) == 0
        return size.value

    def call(ws, n):
        return lib.sgemm_gated_ff_backward(
            M, N, K, 2, 0, dh.data_ptr(), N, x.data_ptr(), K, None, None, wg.data_ptr(), K, wu.data_ptr(), K, 1,
            g.data_ptr(), u.data_ptr(), N, None, None, dx.data_ptr(), K, dwg.data_ptr(), K, dwu.data_ptr(), K,
            None, 0, ws.data_ptr(), n, s)

    # (One row has no stride: it is read in place from any 16 bytes.)
    bits = (1 if K % 8 and M > 1 else 0) | (6 if K % 8 and N > 1 else 0)
    n, small = need(8 | bits), need(bits)
    ws = torch.full((n + 256,), 255, dtype=torch.uint8, device="cuda")
    assert small < n and call(ws, small) == -6 and call(ws, n - 1) == -6
    want = sg.gated_ff_backward(dh, x, wg, wu, (g, u))
    for _ in range(2):
        assert call(ws, n) == 0
        torch.cuda.synchronize()
        assert bool((ws[n:] == 255).all())
        for a, b in zip((dx, dwg, dwu), want):
            assert torch.equal(a, b) and bool(torch.isfinite(a).all())
