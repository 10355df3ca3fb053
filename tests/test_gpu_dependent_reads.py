"""A call's kernel may be set up while the kernel before it still runs, and has to read nothing that one
writes until it has ended.  Each input of each operator is written here by a kernel that takes about a
millisecond on one SM and lets the next one start at once (the layer norm of one row so wide that one
block streams it: a row of one number, whose result is its bias); the operator's own call follows in
the stream.  What it gives has to be what it gives of an input that has been there all along."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BEFORE = 1 << 19           # numbers of the row before the input, which is written last


@pytest.fixture(scope="module")
def sg(cuda):
    import dense_fp32_gemm_09_gb300 as sg
    return sg


def number(seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g, device="cuda")


class Late:
    """A tensor in a buffer that a slow kernel fills."""

    def __init__(self, sg, t, offset=0):
        self.sg = sg
        kind = t.dtype if t.dtype in (torch.float32, torch.bfloat16, torch.float16) else torch.float32
        self.code = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}[kind]
        size = t.numel() * t.element_size() // kind.itemsize
        assert t.is_contiguous() and size * kind.itemsize == t.numel() * t.element_size()
        n = BEFORE + offset + size
        self.want = torch.zeros(n, dtype=kind, device="cuda")
        self.want[BEFORE + offset:] = t.reshape(-1).view(kind)
        assert bool(torch.isfinite(self.want.float()).all())
        self.x = torch.ones(n, dtype=kind, device="cuda")
        self.buffer = torch.empty(n, dtype=kind, device="cuda")
        self.stats = torch.empty(2, device="cuda")
        self.view = self.buffer[BEFORE + offset:].view(t.dtype).view(t.shape)
        self.n = n

    def write(self):
        s = torch.cuda.current_stream().cuda_stream
        assert self.sg.load().sgemm_layer_norm_forward(
            1, self.n, self.code, self.x.data_ptr(), self.n, None, self.want.data_ptr(), self.code, 1e-5,
            self.buffer.data_ptr(), self.n, self.stats.data_ptr(), self.stats.data_ptr() + 4, None, None, s) == 0


def flat(out):
    """The tensors of a result that is there (of a 4-bit one its numbers: rows of padding may hold
    anything)."""
    if isinstance(out, torch.Tensor):
        return [out]
    if hasattr(out, "fmt"):
        return [out.dequantize()]
    if hasattr(out, "codes"):
        return [out.codes, out.scales]
    return [t for o in out if o is not None for t in flat(o)]


def bits(t):
    return t.contiguous().view(torch.uint8)


def check(sg, call, inputs, offsets=None):
    """call(**inputs) with each of the inputs late in turn."""
    stale = []
    for name, t in inputs.items():
        if t is None:
            continue
        late = Late(sg, t, (offsets or {}).get(name, 0))
        now = dict(inputs, **{name: late.view})
        late.write()
        torch.cuda.synchronize()
        assert torch.equal(bits(late.view), bits(t)), name       # the kernel writes what it should
        want = call(**now)
        torch.cuda.synchronize()
        want = flat(want)
        for _ in range(3):
            late.buffer.zero_()
            torch.cuda.synchronize()
            late.write()
            got = call(**now)
            torch.cuda.synchronize()
            if not all(torch.equal(bits(a), bits(b)) for a, b in zip(flat(got), want)):
                stale.append(name)
                break
    assert not stale, stale


DT = {"bf16": torch.bfloat16, "fp32": torch.float32, "fp16": torch.float16}
# Kernels: rows a warp, a block at a time, wide ones in shared memory, ragged, ragged alike, streaming.
NORMS = [(2000, 128, "bf16"), (2000, 128, "fp32"), (5, 1000, "bf16"), (700, 4096, "bf16"), (700, 4096, "fp32"),
         (400, 8192, "bf16"), (400, 10000, "bf16"), (40, 2047, "fp32"), (700, 2047, "bf16"), (400, 5001, "bf16"),
         (5, 40000, "bf16"), (5, 20001, "fp32"), (400, 16384, "bf16"), (330, 17001, "bf16"), (5, 70000, "fp32")]


@pytest.mark.parametrize("rows,cols,dtype", NORMS)
def test_layer_norm(sg, rows, cols, dtype):
    r = number(rows + cols)
    x, w, b = r(rows, cols).to(DT[dtype]), r(cols), r(cols)
    check(sg, lambda x, w, b: sg.layer_norm(x, w, b), dict(x=x, w=w, b=b))
    check(sg, lambda x, w, b: sg.layer_norm(x, w, b, keep="8bit"), dict(x=x, w=w.to(DT[dtype]), b=b.to(DT[dtype])))


@pytest.mark.parametrize("rows,cols,dtype", NORMS)
def test_layer_norm_backward(sg, rows, cols, dtype):
    r = number(rows + cols)
    x, dh, dy = (r(rows, cols).to(DT[dtype]) for _ in range(3))
    w, mean, rstd = r(cols), r(rows), r(rows).abs()
    call = lambda dh, x, mean, rstd, w, dy: sg.layer_norm_backward(dh, x, mean, rstd, w, dy=dy)
    check(sg, call, dict(dh=dh, x=x, mean=mean, rstd=rstd, w=w, dy=dy))
    # (Codes that are floats' bits, of ordinary numbers.)
    codes = torch.randint(1, 64, (rows, -(-cols // 64) * 64), dtype=torch.int8, device="cuda")
    scales = r(rows, -(-cols // 64)).abs()

    def kept(dh, codes, scales, mean, rstd, w, dy):
        return sg.layer_norm_backward(dh, sg.Act8(codes, scales, rows, cols), mean, rstd, w, dy=dy)

    check(sg, kept, dict(dh=dh, codes=codes, scales=scales, mean=mean, rstd=rstd, w=w.to(DT[dtype]), dy=dy))


@pytest.mark.parametrize("rows,cols,dtype", [(1, 64, "fp32"), (300, 4096, "bf16"), (300, 4096, "fp32"), (301, 1999, "fp32"),
                                             (301, 1999, "fp16"), (3000, 8192, "bf16"), (5, 8, "bf16")])
def test_act8(sg, rows, cols, dtype):
    r = number(rows + cols)
    check(sg, lambda x: sg.act8_quantize(x), dict(x=r(rows, cols).to(DT[dtype])))
    codes = torch.randint(1, 64, (rows, -(-cols // 64) * 64), dtype=torch.int8, device="cuda")
    check(sg, lambda codes, scales: sg.Act8(codes, scales, rows, cols).dequantize(DT[dtype]),
          dict(codes=codes, scales=r(rows, -(-cols // 64)).abs()))


FF = [(1, 64, 64), (1, 500, 4096), (3, 100, 77), (9, 333, 1000), (16, 64, 257), (17, 130, 100), (40, 300, 257),
      (300, 520, 136), (700, 96, 1000), (129, 257, 65)]


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,N,K", FF)
def test_gated_ff(sg, M, N, K, dtype, offset):
    r = number(M + N + K)
    x, wg, wu = (r(*s).to(DT[dtype]) for s in ((M, K), (N, K), (N, K)))
    at = dict(x=offset, wg=offset, wu=offset)
    check(sg, lambda x, wg, wu: sg.gated_ff(x, wg, wu), dict(x=x, wg=wg, wu=wu), at)
    check(sg, lambda x, wg, wu: sg.gated_ff(x, wg, wu, keep="8bit"), dict(x=x, wg=wg, wu=wu), at)


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("M,N,K", FF)
def test_gated_ff_backward(sg, M, N, K, dtype, offset):
    r = number(M + N + K)
    dt = DT[dtype]
    x, wg, wu = ((r(*s) / 8).to(dt) for s in ((M, K), (N, K), (N, K)))
    dh, g, u = (r(M, N).to(dt) for _ in range(3))
    at = dict.fromkeys(("x", "wg", "wu", "dh", "g", "u"), offset)
    call = lambda dh, x, wg, wu, g, u: sg.gated_ff_backward(dh, x, wg, wu, (g, u), return_h=True)
    check(sg, call, dict(dh=dh, x=x, wg=wg, wu=wu, g=g, u=u), at)
    codes = lambda n: torch.randint(1, 64, (M, -(-n // 64) * 64), dtype=torch.int8, device="cuda")
    scales = lambda n: r(M, -(-n // 64)).abs() / 32

    def kept(dh, xc, xs, wg, wu, gc, gs, uc, us):
        return sg.gated_ff_backward(dh, sg.Act8(xc, xs, M, K), wg, wu, (sg.Act8(gc, gs, M, N), sg.Act8(uc, us, M, N)),
                                    activation="gelu_tanh", return_h=True)

    check(sg, kept, dict(dh=dh, xc=codes(K), xs=scales(K), wg=wg, wu=wu, gc=codes(N), gs=scales(N), uc=codes(N),
                         us=scales(N)), at)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("rows,cols,dtype", [(1, 64, "fp32"), (300, 4096, "bf16"), (300, 1000, "fp32"), (301, 1999, "fp16"),
                                             (130, 257, "bf16")])
def test_mx4(sg, rows, cols, dtype, fmt):
    r = number(rows + cols)
    x, ts = r(rows, cols).to(DT[dtype]), torch.full((1,), 0.01, device="cuda")
    scaled = fmt == "nvfp4"
    call = lambda x, ts: sg.mx4_quantize(x, fmt, tensor_scale=ts)
    check(sg, call, dict(x=x, ts=ts if scaled else None))
    check(sg, lambda x, ts: sg.mx4_quantize(x.t(), fmt, tensor_scale=ts), dict(x=x, ts=ts if scaled else None))
    q = sg.mx4_quantize(x, fmt)
    codes, scales = torch.randint_like(q.codes, 1, 64), torch.randint_like(q.scales, 40, 64)
    held = lambda c, s, ts: sg.Mx4(c, s, rows, cols, fmt, ts)
    inputs = dict(codes=codes, scales=scales, ts=ts if scaled else None)
    check(sg, lambda codes, scales, ts: held(codes, scales, ts).dequantize(DT[dtype]), inputs)
    other = sg.mx4_quantize(r(200, cols), fmt)
    check(sg, lambda codes, scales, ts: sg.mx4_matmul(held(codes, scales, ts), other), inputs)
    check(sg, lambda codes, scales, ts: sg.mx4_matmul(other, held(codes, scales, ts)), inputs)


@pytest.mark.parametrize("M,N,K", [(1, 256, 512), (300, 512, 640), (2000, 2048, 512)])
def test_mx4_matmul_adds_to(sg, M, N, K):
    r = number(M)
    a, b = sg.mx4_quantize(r(M, K)), sg.mx4_quantize(r(N, K))
    # (A copy, as the call writes its C.)
    lib = dict(c=r(M, N))
    ready = torch.empty(M, N, device="cuda")

    def call(c):
        torch.mul(c, 1, out=ready)
        return sg.mx4_matmul(a, b, out=ready, beta=1.0)

    check(sg, call, lib)


@pytest.mark.parametrize("gate", ["full", "row", None])
@pytest.mark.parametrize("rows,cols,dtype", [(5, 128, "bf16"), (700, 1000, "fp32"), (700, 4096, "bf16"), (400, 8192, "bf16"),
                                             (40, 2047, "fp32"), (700, 2047, "bf16"), (5, 16000, "bf16"), (5, 20000, "bf16"),
                                             (5, 20001, "fp32"), (5, 40000, "fp16")])
def test_norms(sg, rows, cols, dtype, gate):
    r = number(rows + cols)
    dt = DT[dtype]
    block, res, dy, dh, y = (r(rows, cols).to(dt) for _ in range(5))
    gate = r(rows, cols).to(dt) if gate == "full" else r(cols).to(dt) if gate == "row" else None
    w, nw, rs, nrs = r(cols), r(cols), r(rows).abs(), r(rows).abs()
    forward = lambda block, res, w, gate, nw: sg.norm_after(block, res, w, gate=gate, scale=0.5, next_weight=nw)
    check(sg, forward, dict(block=block, res=res, w=w, gate=gate, nw=nw))
    one = lambda block, res, w, gate: sg.norm_after(block, res, w, gate=gate)
    check(sg, one, dict(block=block, res=res, w=w.to(dt), gate=gate))
    backward = lambda dy, block, rs, w, gate, dh, y, nrs, nw: sg.norm_after_backward(
        dy, block, rs, w, gate=gate, scale=0.5, dh=dh, y=y, next_rstd=nrs, next_weight=nw)
    check(sg, backward, dict(dy=dy, block=block, rs=rs, w=w, gate=gate, dh=dh, y=y, nrs=nrs, nw=nw))
    if gate is None:
        check(sg, lambda res, w: sg.norm_before(res, w), dict(res=res, w=w))
        check(sg, lambda res, w: sg.norm_before(res, w, quantize="nvfp4"), dict(res=res, w=w.to(dt)))
        check(sg, lambda dh, y, nrs, nw: sg.norm_before_backward(dh, y, nrs, nw), dict(dh=dh, y=y, nrs=nrs, nw=nw))


@pytest.mark.parametrize("ta,tb", [("N", "N"), ("T", "N"), ("N", "T")])
@pytest.mark.parametrize("M,N,K", [(64, 64, 64), (257, 300, 129), (256, 256, 4096), (1024, 1024, 512), (100, 2000, 77)])
def test_sgemm(sg, M, N, K, ta, tb):
    r = number(M)
    a = r(M, K) if ta == "N" else r(K, M)
    b = r(K, N) if tb == "N" else r(N, K)
    check(sg, lambda a, b: sg.sgemm(a.t() if ta == "T" else a, b.t() if tb == "T" else b), dict(a=a, b=b))
