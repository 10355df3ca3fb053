"""An Mx4 holds tensors, not addresses: what its attributes and tensors are when a call is
made is what the call uses."""
import pytest
import torch

from test_gpu_mx4 import sample, sg  # noqa: F401  (sg: fixture)

pytestmark = pytest.mark.gpu


def made(sg, fmt="nvfp4", rows=40, cols=200, ts=0.5, seed=1):  # noqa: F811
    t = None if ts is None else torch.tensor([ts], device="cuda")
    return sg.mx4_quantize(sample(rows, cols, "fp32", seed).cuda(), fmt, tensor_scale=t)


@pytest.mark.parametrize("given", [True, False])
def test_tensor_scale_can_be_set(sg, given):  # noqa: F811
    q = made(sg)
    old = q.tensor_scale
    if given:
        q = sg.Mx4(q.codes, q.scales, 40, 200, "nvfp4", old)
    before, w = q.dequantize(), made(sg, rows=30, seed=2)
    c = sg.mx4_matmul(q, w)
    q.tensor_scale = torch.full((1,), 4.0, device="cuda")
    assert torch.equal(q.dequantize(), before * 8) and torch.equal(sg.mx4_matmul(q, w), c * 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    side = sg.mx4_matmul(q, w, stream=s)
    s.synchronize()
    assert torch.equal(side, c * 8)
    q.tensor_scale = None
    assert torch.equal(q.dequantize(), before * 2)
    assert float(old) == 0.5
    with pytest.raises(TypeError, match="one float32"):
        q.tensor_scale = torch.ones(2, device="cuda")
    with pytest.raises(ValueError, match="CUDA"):
        q.tensor_scale = torch.ones(1)
    with pytest.raises(ValueError, match="nvfp4"):
        made(sg, "mxfp4", ts=None).tensor_scale = torch.ones(1, device="cuda")


@pytest.mark.parametrize("name,value", [("rows", 4000), ("cols", 8192), ("fmt", "mxfp4"),
                                        ("shape", (4000, 200)), ("device", "cpu"), ("codes", None),
                                        ("scales", None)])
def test_shape_format_and_buffers_stay(sg, name, value):  # noqa: F811
    q = made(sg)
    with pytest.raises(AttributeError):
        setattr(q, name, value)


def test_tensors_that_move(sg):  # noqa: F811
    """The memory of a given tensor may be replaced between calls; one that no longer fits is
    refused."""
    a, b = made(sg, ts=None), made(sg, ts=None, seed=3)
    codes, scales, keep = a.codes.clone(), a.scales.clone(), []
    q = sg.Mx4(codes, scales, 40, 200, "nvfp4")
    assert torch.equal(q.dequantize(), a.dequantize())
    keep.append((codes.detach(), scales.detach()))
    codes.set_(b.codes.clone())
    scales.set_(b.scales.clone())
    assert torch.equal(q.dequantize(), b.dequantize())
    w = made(sg, rows=5, seed=4)
    assert torch.equal(sg.mx4_matmul(w, q), sg.mx4_matmul(w, b))
    codes.set_(torch.zeros(1, 4, 128, 16, dtype=torch.uint8, device="cuda"))
    for call in (lambda: q.dequantize(), lambda: sg.mx4_matmul(w, q), lambda: sg.mx4_matmul(q, w)):
        with pytest.raises(ValueError, match="codes must be"):
            call()


def test_emptied_buffer_is_refused(sg):  # noqa: F811
    q = made(sg)
    q.codes.untyped_storage().resize_(0)
    with pytest.raises(sg.SgemmError, match="null"):
        q.dequantize()


def test_launches_are_counted(sg):  # noqa: F811
    """sgemm_launch_count counts kernels: one a call, none where C only stays as it is."""
    def count(call):
        before = sg.launch_count()
        call()
        return sg.launch_count() - before
    q, w, c = made(sg), made(sg, rows=30, seed=2), torch.ones(40, 30, device="cuda")
    empty = sg.mx4_quantize(torch.ones(40, 0, device="cuda"))
    none = sg.mx4_quantize(torch.ones(30, 0, device="cuda"))
    assert count(lambda: sg.mx4_matmul(q, w)) == 1 and count(q.dequantize) == 1
    assert count(lambda: sg.mx4_matmul(empty, none, c, beta=1.0)) == 0
    assert count(lambda: sg.mx4_matmul(q, w, c, alpha=0.0, beta=1.0)) == 0
    assert bool((c == 1).all())
    assert count(lambda: sg.mx4_matmul(q, w, c, alpha=0.0, beta=2.0)) == 1
    x, one = torch.ones(4, 64, device="cuda"), torch.ones(64, device="cuda")
    _, r = sg.norm_before(x)
    assert count(lambda: sg.norm_before_backward(x, x, r)) == 1
    assert count(lambda: sg.norm_before_backward(x, x, r, one)) == 2
