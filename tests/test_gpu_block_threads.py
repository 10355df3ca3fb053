"""The 4-bit and norm operators from several host threads at once, on one stream and on a
stream of each thread's own: every result is that of the same call alone."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu
THREADS, ROUNDS = 6, 8


@pytest.fixture()
def sg(cuda):
    import dense_fp32_gemm_09_gb300 as sg
    return sg


def block(sg, i):
    """One thread's work: sizes of its own, so that workspaces differ."""
    g = torch.Generator("cuda").manual_seed(i)
    rows, cols = 300 + 70 * i, 512 + 1000 * i + i % 2
    x, b, dh = (torch.randn(rows, cols, generator=g, device="cuda") for _ in range(3))
    w = torch.rand(cols, generator=g, device="cuda")
    torch.cuda.synchronize()

    def run():
        y, r, h, rn = sg.norm_after(b, x, w, gate=w, next_weight=w, quantize="nvfp4")
        grads = sg.norm_after_backward(dh, b, r, w, gate=w, dh=dh, y=y, next_rstd=rn, next_weight=w)
        return (y, r, rn, sg.mx4_matmul(h, h), h.dequantize()) + grads
    return run


@pytest.mark.parametrize("own_streams", [True, False])
def test_threads(sg, own_streams):
    work = [block(sg, i) for i in range(THREADS)]
    want = [run() for run in work]
    torch.cuda.synchronize()
    shared, bad = torch.cuda.Stream(), []

    def thread(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream() if own_streams else shared):
                for _ in range(ROUNDS):
                    got = work[i]()
                    torch.cuda.current_stream().synchronize()
                    bad.extend((i, k) for k, (a, b) in enumerate(zip(got, want[i]))
                               if not torch.equal(a, b))
        except Exception as e:      # noqa: BLE001  (reported below)
            bad.append((i, e))
    threads = [threading.Thread(target=thread, args=(i,)) for i in range(THREADS)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
