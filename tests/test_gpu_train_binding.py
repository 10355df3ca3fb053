"""The compiled step from Python to the C ABI and the Python code behind it give the same results,
on other streams, from several threads and inside captured graphs."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture()
def sg(cuda):
    import dense_fp32_gemm_09_gb300 as sg
    return sg


def inputs(M=300, N=200, K=136, seed=0, dtype=torch.bfloat16):
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")
    return {"x": r(M, K).to(dtype), "wg": (r(N, K) / K ** 0.5).to(dtype),
            "wu": (r(N, K) / K ** 0.5).to(dtype), "dh": r(M, N).to(dtype), "w": 1 + 0.2 * r(K),
            "b": 0.2 * r(K), "dy": r(M, K).to(dtype)}


def block(sg, t, stream=None):
    """Norm, feed-forward block and the gradients of both, with everything kept in 8 bits."""
    n, mean, rstd, kx = sg.layer_norm(t["x"], t["w"], t["b"], keep="8bit", stream=stream)
    kn = sg.act8_quantize(n, stream=stream)
    h, kept = sg.gated_ff(n, t["wg"], t["wu"], keep="8bit", stream=stream)
    dn, dwg, dwu, h2 = sg.gated_ff_backward(t["dh"], kn, t["wg"], t["wu"], kept, return_h=True,
                                            stream=stream)
    dx, dw, db = sg.layer_norm_backward(dn, kx, mean, rstd, t["w"], dy=t["dy"], stream=stream)
    f, full = sg.gated_ff(n, t["wg"], t["wu"], keep="full", activation="gelu_tanh", stream=stream)
    g = sg.gated_ff_backward(t["dh"], n, t["wg"], t["wu"], full, activation="gelu_tanh", stream=stream)
    return (n, mean, rstd, h, dn, dwg, dwu, h2, dx, dw, db, f, *g, sg.gated_ff(n, t["wg"], t["wu"]),
            kx.dequantize(torch.bfloat16, stream=stream), *(q.dequantize(stream=stream) for q in kept))


def same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("M,N,K", [(300, 200, 136), (1, 72, 64), (13, 131, 77), (1, 1, 1)])
def test_both_ways(sg, monkeypatch, M, N, K):
    t = inputs(M, N, K)
    want = block(sg, t)

    class Nothing:
        def __getattr__(self, name):
            return lambda *a: None

    import dense_fp32_gemm_09_gb300._tensors as tensors
    monkeypatch.setattr(tensors, "_fast", Nothing())
    assert same(block(sg, t), want)


def test_other_streams(sg):
    t = inputs()
    want = block(sg, t)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    given = block(sg, t, stream=s)
    with torch.cuda.stream(s):
        current = block(sg, t)
    torch.cuda.synchronize()
    assert same(given, want) and same(current, want)
    raw = block(sg, t, stream=s.cuda_stream)
    torch.cuda.synchronize()
    assert same(raw, want)


def test_graphs_beside_each_other(sg):
    """Two graphs captured on one stream, replayed side by side with an eager call: workspaces are
    each graph's own."""
    data = [inputs(1000, 520, 264, seed=i) for i in range(3)]
    want = [block(sg, t) for t in data]
    torch.cuda.synchronize()
    s, others = torch.cuda.Stream(), [torch.cuda.Stream() for _ in range(2)]
    graphs, outs = [], []
    for t in data[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(block(sg, t))
        graphs.append(g)
    for _ in range(10):
        for g, o in zip(graphs, others):
            with torch.cuda.stream(o):
                g.replay()
        with torch.cuda.stream(s):
            eager = block(sg, data[2])
    torch.cuda.synchronize()
    for got, ref in zip(outs + [eager], want):
        assert same(got, ref)


@pytest.mark.parametrize("cols", [64, 2047, 8192, 9000, 16384, 20001])
def test_norms_of_every_width_in_graphs(sg, cols):
    """Every kernel of the norm (one warp, one block, a cluster of blocks a row) is captured."""
    g = torch.Generator("cuda").manual_seed(cols)
    x, dh, dy = (torch.randn((50, cols), generator=g, device="cuda").bfloat16() for _ in range(3))
    w = torch.randn((cols,), generator=g, device="cuda")

    def call():
        y, mean, rstd, kept = sg.layer_norm(x, w, w, keep="8bit")
        return (y, mean, rstd, *sg.layer_norm_backward(dh, kept, mean, rstd, w, dy=dy),
                *sg.layer_norm_backward(dh, x, mean, rstd, w))

    want = call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want)


def test_threads(sg):
    data = [inputs(100 + 50 * i, 136 + 8 * i, 72 + i, seed=i) for i in range(4)]
    want = [block(sg, t) for t in data]
    torch.cuda.synchronize()
    wrong = []

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = block(sg, data[i])
                torch.cuda.current_stream().synchronize()
                if not same(got, want[i]):
                    wrong.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong


def test_launches_are_counted(sg):
    t = inputs()
    n = sg.launch_count()
    sg.act8_quantize(t["x"])
    assert sg.launch_count() == n + 1
    sg.gated_ff(t["x"], t["wg"], t["wu"])
    assert sg.launch_count() == n + 2
    sg.gated_ff(t["x"][:0], t["wg"], t["wu"])
    assert sg.launch_count() == n + 2


def test_results_are_outside_torchs_graph(sg):
    t = inputs()
    x = t["x"].clone().requires_grad_()
    assert not sg.gated_ff(x, t["wg"], t["wu"]).requires_grad
    assert not sg.layer_norm(x)[0].requires_grad
    assert sg.load().sgemm_device_status() == 0
