"""The norms' gradients inside captured CUDA graphs: what the sums over rows go through must
outlive later, larger calls on the same stream, and two graphs must not share it."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture()
def sg(cuda):
    import dense_fp32_gemm_09_gb300 as sg
    return sg


def inputs(rows, cols, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    x, dh = (torch.randn(rows, cols, generator=g, device="cuda") for _ in range(2))
    return x, dh, torch.rsqrt(x.square().mean(1) + 1e-6), torch.ones(cols, device="cuda")


def entry(lib, stream, x, dh, rstd, w, dx, dw):
    rows, cols = x.shape
    return lib.sgemm_norm_backward(rows, cols, 0, None, 0, dh.data_ptr(), cols, x.data_ptr(), cols,
                                   rstd.data_ptr(), w.data_ptr(), None, 0, None, None, 0, None, 0,
                                   1.0, dx.data_ptr(), cols, None, 0, None, 0, None, dw.data_ptr(),
                                   stream.cuda_stream)


@pytest.mark.parametrize("warm", [True, False])
def test_library_workspace_stays_while_a_graph_holds_it(sg, warm):
    """The C entry: captured at 1024 columns (its workspace made before the capture, or in it),
    then a wider gradient on the same stream outgrows that workspace."""
    lib, s = sg.load(), torch.cuda.Stream()
    small, large = inputs(700, 1024, 1), inputs(700, 8192, 2)
    out = [(torch.empty_like(t[0]), torch.empty_like(t[3])) for t in (small, large)]
    want = [sg.norm_before_backward(t[1], t[0], t[2], t[3]) for t in (small, large)]
    torch.cuda.synchronize()
    if warm:
        assert entry(lib, s, *small, *out[0]) == 0
        s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        status = entry(lib, s, *small, *out[0])
    assert status == 0
    for _ in range(2):
        assert entry(lib, s, *large, *out[1]) == 0
    s.synchronize()
    assert torch.equal(out[1][1], want[1][1])
    for _ in range(3):
        out[0][1].fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0][0], want[0][0]) and torch.equal(out[0][1], want[0][1])


def test_graphs_of_one_stream_have_their_own_sums(sg):
    """Two graphs captured on one stream, replayed side by side on two others, beside eager
    calls on the stream of the capture."""
    s, others = torch.cuda.Stream(), [torch.cuda.Stream() for _ in range(2)]
    data = [inputs(4000, 4096, 3 + i) for i in range(3)]
    call = lambda t: sg.norm_before_backward(t[1], t[0], t[2], t[3])
    want = [call(t) for t in data]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for t in data[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(call(t))
        graphs.append(g)
    for _ in range(20):
        for g, o in zip(graphs, others):
            with torch.cuda.stream(o):
                g.replay()
        with torch.cuda.stream(s):
            eager = call(data[2])
    torch.cuda.synchronize()
    for got, ref in zip(outs + [eager], want):
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 64), (3000, 64), (3000, 1000), (900, 1025),
                                       (900, 3001), (700, 4096), (700, 4100), (500, 8192),
                                       (400, 8200), (340, 20000)])
def test_callers_workspace(sg, rows, cols):
    """The size that the query gives is enough for every type and alignment, nothing is written
    past it, and one that is missing or too small is refused."""
    lib, stream = sg.load(), torch.cuda.current_stream()
    size = ctypes.c_size_t(0)
    assert lib.sgemm_norm_backward_workspace(rows, cols, ctypes.byref(size)) == 0
    assert lib.sgemm_norm_backward_workspace(rows, -1, ctypes.byref(size)) == -1
    assert lib.sgemm_norm_backward_workspace(rows, cols, None) == -1
    assert lib.sgemm_norm_backward_workspace(rows, cols, ctypes.byref(size)) == 0
    ws = torch.full((size.value + 64,), 7, dtype=torch.uint8, device="cuda")
    x, dh, rstd, w = inputs(rows, cols, 9)
    for code, dtype in enumerate((torch.float32, torch.bfloat16, torch.float16)):
        for off in (0, 1):
            buf = torch.empty(4, rows * cols + off, dtype=dtype, device="cuda")
            xx, dd, dx, db = (b[off:].view(rows, cols) for b in buf)
            xx.copy_(x)
            dd.copy_(dh)
            sums = torch.full((3, cols), float("nan"), device="cuda")
            gate = torch.ones(cols, dtype=dtype, device="cuda")
            args = lambda at, n: lib.sgemm_norm_backward_ws(
                rows, cols, code, None, 0, dd.data_ptr(), cols, xx.data_ptr(), cols,
                rstd.data_ptr(), w.data_ptr(), xx.data_ptr(), cols, rstd.data_ptr(), w.data_ptr(),
                0, gate.data_ptr(), 0, 1.0, dx.data_ptr(), cols, db.data_ptr(), cols,
                sums[0].data_ptr(), cols, sums[1].data_ptr(), sums[2].data_ptr(), at, n,
                stream.cuda_stream)
            assert args(None, size.value) == -6 and args(ws.data_ptr(), 8) == -6
            assert args(ws.data_ptr() + 4, size.value) == -6
            assert args(ws.data_ptr(), size.value) == 0
            want = sg.norm_after_backward(None, xx, rstd, w, gate=gate, dh=dd, y=xx, next_rstd=rstd,
                                          next_weight=w)
            for got, ref in zip((dx, db, sums[1], sums[0], sums[2]), want):
                assert torch.equal(got, ref)
    assert bool((ws[size.value:] == 7).all())
