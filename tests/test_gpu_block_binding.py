"""The compiled binding of the usual calls behaves as the Python code of the same calls does."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture()
def sg(cuda):
    import dense_fp32_gemm_09_gb300 as sg
    return sg


def calls(sg):
    q = sg.mx4_quantize(torch.ones(1 << 14, 32, device="cuda"))
    w = torch.ones(1 << 14, 1 << 12, device="cuda")
    r = torch.ones(1 << 14, device="cuda")
    return {"quantize": lambda s: sg.mx4_quantize(w, stream=s),
            "dequantize": lambda s: sg.mx4_dequantize(q, stream=s),
            "matmul": lambda s: sg.mx4_matmul(q, q, stream=s),
            "norm_before": lambda s: sg.norm_before(w, stream=s),
            "norm_after": lambda s: sg.norm_after(w, w, stream=s),
            "backward": lambda s: sg.norm_before_backward(w, w, r, stream=s)}


@pytest.mark.parametrize("name", ["quantize", "dequantize", "matmul", "norm_before", "norm_after",
                                  "backward"])
@pytest.mark.parametrize("compiled", [True, False])
def test_out_of_memory_is_torch_s(sg, name, compiled):
    """An allocation past the process's own limit (nothing near the device's) raises torch's
    error, and the call works again without the limit."""
    call, s = calls(sg)[name], None if compiled else torch.cuda.current_stream()
    call(s)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    try:
        torch.cuda.set_per_process_memory_fraction(torch.cuda.memory_reserved() / total)
        held = []
        with pytest.raises(torch.OutOfMemoryError):
            for _ in range(1 << 16):      # whatever the allocator still has in hand
                held.append(call(s))
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    held.clear()
    call(s)
    torch.cuda.synchronize()


def test_other_threads_run_during_a_call(sg):
    """A call that has to wait in the library does not keep Python's lock.  The library's
    dequantisation is replaced by libc's usleep, whose argument is then the number of rows."""
    import ctypes
    import threading
    import time

    from dense_fp32_gemm_09_gb300 import _tensors
    names = ["sgemm_mx4_quantize", "sgemm_mx4_dequantize", "sgemm_mx4_matmul", "sgemm_norm_forward",
             "sgemm_norm_backward_ws", "sgemm_norm_backward_workspace"]
    entries = [ctypes.cast(getattr(sg.load(), n), ctypes.c_void_p).value for n in names]
    usleep = ctypes.cast(ctypes.CDLL(None).usleep, ctypes.c_void_p).value
    q = sg.mx4_quantize(torch.ones(400000, 4, device="cuda"))
    want = q.dequantize()
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.005)
    other = threading.Thread(target=tick)
    other.start()
    try:
        _tensors.fast().bind(entries[0], usleep, *entries[2:])
        start = time.perf_counter()
        q.dequantize()
        end = time.perf_counter()
    finally:
        _tensors.fast().bind(*entries)
        stop.set()
        other.join()
    assert end - start >= 0.39
    assert sum(start + 0.05 < t < end - 0.05 for t in ticks) >= 5
    assert torch.equal(q.dequantize(), want)
