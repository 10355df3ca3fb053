"""The gated feed-forward block and its gradient against their formulas in 64 bits.

Tolerances.  u is half an ulp of the operands' type (2^-8, 2^-11) and t = 2^-25 half the step of
fp16's subnormal numbers.  Products of 2-byte numbers are exact in fp32; a sum of K of them is at most
K / 16 + 16 additions deep (sixteen products at a time), each off by an ulp (2^-23) of the
magnitudes so far: s(K) = (K / 16 + 16) 2^-23 of the sum of the terms' magnitudes.  One-thread-a-sum
kernels take K additions of half an ulp, s(K) is then 4 sqrt(K) 2^-24 at four standard
deviations, which is less.  The activation's approximations are 2^-19 of its result.  |act'| <= 1.13.

Where every number is a small integer all of this is exact, up to the last rounding."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
T = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}
# tokens, outputs, inputs
SHAPES = [(1, 1, 1), (1, 8, 16), (3, 5, 7), (1, 1000, 200), (8, 333, 257), (16, 64, 64), (17, 130, 100),
          (1, 2048, 4096), (5, 100, 8), (33, 64, 72), (128, 128, 64), (129, 257, 65), (256, 256, 256),
          (300, 520, 136), (257, 1000, 2047), (1000, 640, 1024), (64, 4096, 512), (700, 96, 1000),
          (2000, 300, 64), (9, 2050, 1030), (513, 129, 320), (64, 8100, 250), (64, 8192, 256), (400, 2501, 200),
          (400, 2504, 200), (2500, 1000, 64)]
# Several rounds of tiles, every tile and split (test_gated_ff_choice.py).
MANY = [(2600, 2100, 200), (4700, 2600, 72), (1000, 4100, 520), (900, 100, 6000), (9000, 64, 300),
        (40, 3000, 520), (3000, 40, 520), (20000, 260, 250), (12000, 500, 1000),
        (30000, 512, 512), (700, 8192, 700), (30, 8200, 4100)]


@pytest.fixture()
def sg(cuda):
    import dense_fp32_gemm_09_gb300 as sg
    return sg


def depth(k):
    return (k / 16 + 16) * 2.0 ** -23


def act(g, name):
    """(act, act') in 64 bits."""
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    c = (2 / torch.pi) ** 0.5
    th = torch.tanh(c * (g + 0.044715 * g ** 3))
    return g / 2 * (1 + th), (1 + th) / 2 + g / 2 * (1 - th * th) * c * (1 + 3 * 0.044715 * g * g)


class Case:
    def __init__(self, M, N, K, dtype, seed=0):
        g = torch.Generator("cuda").manual_seed(M * 7 + N * 3 + K + seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")
        dt = DTYPES[dtype]
        self.M, self.N, self.K, self.u, self.t, self.dt = M, N, K, U[dtype], T[dtype], dt
        self.x, self.dh = r(M, K).to(dt), r(M, N).to(dt)
        self.wg, self.wu = ((r(N, K) / K ** 0.5).to(dt) for _ in range(2))


def near(got, want, tol, what):
    bad = (got.double() - want).abs() - tol
    assert bool(torch.isfinite(got).all()) and bool((bad <= 0).all()), (what, float(bad.max()))


def sums(c):
    """g, u in 64 bits and how far fp32 sums may be off."""
    x, wg, wu = c.x.double(), c.wg.double(), c.wu.double()
    s = depth(c.K)
    return x @ wg.t(), x @ wu.t(), s * (x.abs() @ wg.abs().t()), s * (x.abs() @ wu.abs().t())


def check_forward(sg, c, name, **views):
    x, wg, wu = (views.get(k, getattr(c, k)) for k in ("x", "wg", "wu"))
    g, u, eg, eu = sums(c)
    a, _ = act(g, name)
    want = a * u
    tol = 1.13 * eg * (u.abs() + eu) + (a.abs() + 1.13 * eg) * eu + 2.0 ** -19 * want.abs()
    tol = tol * 1.01 + c.u * 1.01 * (want.abs() + tol) + c.t
    h = sg.gated_ff(x, wg, wu, activation=name)
    near(h, want, tol, "h")
    h1, (gate, up) = sg.gated_ff(x, wg, wu, activation=name, keep="full")
    assert torch.equal(h1, h)
    near(h1, want, tol, "h beside what is kept")
    near(gate, g, eg + c.u * 1.01 * (g.abs() + eg) + c.t, "gate")
    near(up, u, eu + c.u * 1.01 * (u.abs() + eu) + c.t, "up")
    h2, kept = sg.gated_ff(x, wg, wu, activation=name, keep="8bit")
    # (Up to 16 tokens, checkpoints in 8 bits take another kernel, which sums in another order.)
    assert torch.equal(h2, h1) or c.M <= 16
    near(h2, want, tol, "h beside what is kept in 8 bits")
    for q, v, ev in zip(kept, (g, u), (eg, eu)):
        # Half a step of the block's largest magnitude, and the fp32 roundings of the definition.
        top = torch.nn.functional.pad(v.abs() + ev, (0, -c.N % 64)).view(c.M, -1, 64).amax(2)
        step = (top / 127).repeat_interleave(64, 1)[:, :c.N]
        near(q.dequantize(), v, ev + step * (0.5 + 2.0 ** -14), "8 bits")
        assert not bool(q.codes[:, c.N:].any())
    return h


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forward(sg, M, N, K, dtype, name):
    check_forward(sg, Case(M, N, K, dtype), name)


def whole(c, seed=1):
    """Small integers, with gates of 32 to 127 where act(g) = g and act' = 1 to the last bit: x's
    first column is 1 and the gate weight's carries the offset."""
    g = torch.Generator("cuda").manual_seed(seed)
    r = lambda lo, hi, *s: torch.randint(lo, hi + 1, s, generator=g, device="cuda").to(c.dt)
    c.x, c.wg, c.wu = r(-1, 1, c.M, c.K), torch.zeros_like(c.wg), torch.zeros_like(c.wu)
    # Few nonzero weights a row, so that sums stay small: every column of x is in some output.
    for w in (c.wg, c.wu):
        for _ in range(8):
            at = torch.randint(0, c.K, (c.N, 1), generator=g, device="cuda")
            w.scatter_(1, at, r(-2, 2, c.N, 1))
    c.x[:, 0], c.wg[:, 0] = 1, 80
    c.dh = r(-1, 1, c.M, c.N)
    return c


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("M,N,K", SHAPES + MANY)
def test_forward_of_integers_is_exact(sg, M, N, K, dtype):
    c = whole(Case(M, N, K, dtype))
    x, wg, wu = c.x.double(), c.wg.double(), c.wu.double()
    g, u = x @ wg.t(), x @ wu.t()
    for name in ("silu", "gelu_tanh"):
        assert torch.equal(sg.gated_ff(c.x, c.wg, c.wu, activation=name), (g * u).to(c.dt))
        h, (gate, up) = sg.gated_ff(c.x, c.wg, c.wu, activation=name, keep="full")
        assert torch.equal(h, (g * u).to(c.dt))
        assert torch.equal(gate, g.to(c.dt)) and torch.equal(up, u.to(c.dt))
        h, kept = sg.gated_ff(c.x, c.wg, c.wu, activation=name, keep="8bit")
        for q, v in zip(kept, (g, u)):
            ref = sg.act8_quantize(v.float())
            assert torch.equal(q.codes, ref.codes) and torch.equal(q.scales, ref.scales)


def check_backward(sg, c, name, kept, x=None, return_h=False, views={}):
    if x is None:
        x = views.get("x", c.x)
    wg, wu, dh = (views.get(k, getattr(c, k)) for k in ("wg", "wu", "dh"))
    out = sg.gated_ff_backward(dh, x, wg, wu, kept, activation=name, return_h=return_h)
    g, u = (q.dequantize().double() if isinstance(q, sg.Act8) else q.double() for q in kept)
    x64 = x.dequantize().double() if isinstance(x, sg.Act8) else c.x.double()
    dh, wg, wu = c.dh.double(), c.wg.double(), c.wu.double()
    a, slope = act(g, name)
    dg, du = dh * u * slope, dh * a
    # The terms' own errors: the activation's and the rounding to the operands' type.  The
    # slope is a difference of terms of at most 1 + |g| / 4 (silu) or 2 (gelu).
    edg = c.u * 1.01 * dg.abs() + 2.0 ** -19 * 4 * (dh * u).abs() + c.t
    edu = c.u * 1.01 * du.abs() + 2.0 ** -19 * du.abs() + c.t
    ex = c.u * 1.01 * x64.abs() + c.t if isinstance(x, sg.Act8) else torch.zeros_like(x64)
    want = dg @ wg + du @ wu
    tol = edg @ wg.abs() + edu @ wu.abs() + depth(2 * c.N) * (dg.abs() @ wg.abs() + du.abs() @ wu.abs())
    near(out[0], want, tol * 1.01 + c.u * 1.01 * (want.abs() + tol) + c.t, "dx")
    for got, d, ed, what in ((out[1], dg, edg, "dw_gate"), (out[2], du, edu, "dw_up")):
        want = d.t() @ x64
        tol = ed.t() @ (x64.abs() + ex) + d.abs().t() @ ex + depth(c.M) * (d.abs().t() @ x64.abs())
        near(got, want, tol * 1.01 + c.u * 1.01 * (want.abs() + tol) + c.t, what)
    if return_h:
        near(out[3], a * u, (c.u * 1.01 + 2.0 ** -19) * (a * u).abs() + c.t, "h again")
    return out


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_backward(sg, M, N, K, dtype, name):
    c = Case(M, N, K, dtype)
    _, kept = sg.gated_ff(c.x, c.wg, c.wu, activation=name, keep="full")
    first = check_backward(sg, c, name, kept)
    second = check_backward(sg, c, name, kept, return_h=True)
    assert all(torch.equal(a, b) for a, b in zip(first, second))
    _, kept = sg.gated_ff(c.x, c.wg, c.wu, activation=name, keep="8bit")
    check_backward(sg, c, name, kept, return_h=True)
    check_backward(sg, c, name, kept, sg.act8_quantize(c.x))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("M,N,K", SHAPES + MANY)
def test_backward_of_integers_is_exact(sg, M, N, K, dtype):
    c = whole(Case(M, N, K, dtype))
    x, wg, wu, dh = (t.double() for t in (c.x, c.wg, c.wu, c.dh))
    gen = torch.Generator("cuda").manual_seed(5)
    g = torch.randint(0, 2, (M, N), generator=gen, device="cuda").double() * 32 + 32
    u = torch.randint(-2, 3, (M, N), generator=gen, device="cuda").double()
    kept = (g.to(c.dt), u.to(c.dt))
    dg, du = dh * u, dh * g
    for name in ("silu", "gelu_tanh"):
        dx, dwg, dwu, h = sg.gated_ff_backward(c.dh, c.x, c.wg, c.wu, kept, activation=name, return_h=True)
        assert torch.equal(dx, (dg @ wg + du @ wu).to(c.dt))
        assert torch.equal(dwg, (dg.t() @ x).to(c.dt)) and torch.equal(dwu, (du.t() @ x).to(c.dt))
        assert torch.equal(h, (g * u).to(c.dt))


def test_gradient_against_differences(sg):
    """Central differences in 64 bits of the reference that the forward test ties to the kernels."""
    c = Case(3, 24, 16, "fp16")
    _, kept = sg.gated_ff(c.x, c.wg, c.wu, keep="full")
    grads = sg.gated_ff_backward(c.dh, c.x, c.wg, c.wu, kept)
    at = [c.x.double(), c.wg.double(), c.wu.double()]
    loss = lambda x, wg, wu: (act(x @ wg.t(), "silu")[0] * (x @ wu.t()) * c.dh.double()).sum()
    for which, got in enumerate(grads):
        scale = float(got.abs().max())
        for i in range(0, at[which].numel(), 5):
            step = torch.zeros_like(at[which])
            step.view(-1)[i] = 1e-4
            up, down = list(at), list(at)
            up[which], down[which] = at[which] + step, at[which] - step
            want = float(loss(*up) - loss(*down)) / 2e-4
            # Kept g and u, their gradients and the result: four roundings of 2^-11 of terms whose
            # magnitudes add up to a few times the result's.
            assert abs(float(got.view(-1)[i]) - want) < 2.0 ** -7 * scale


@pytest.mark.parametrize("offset,pad", [(0, 8), (1, 0), (1, 3), (3, 5), (2, 6), (8, 0)])
@pytest.mark.parametrize("M,N,K", [(5, 72, 200), (300, 200, 136)])
def test_strides_and_alignment(sg, M, N, K, offset, pad):
    c = Case(M, N, K, "bf16")

    def strided(t):
        rows, cols = t.shape
        flat = torch.full((offset + rows * (cols + pad) + 8,), float("nan"), dtype=t.dtype, device="cuda")
        view = flat[offset:offset + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        view.copy_(t)
        return view

    views = {k: strided(getattr(c, k)) for k in ("x", "wg", "wu", "dh")}
    check_forward(sg, c, "silu", **views)
    check_forward(sg, c, "silu", wu=views["wu"])
    _, kept = sg.gated_ff(c.x, c.wg, c.wu, keep="full")
    want = check_backward(sg, c, "silu", kept)
    for some in (views, {"x": views["x"]}, {"wg": views["wg"]}, {"dh": views["dh"], "wu": views["wu"]}):
        got = check_backward(sg, c, "silu", kept, views=some)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = check_backward(sg, c, "silu", tuple(strided(t) for t in kept))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("M,N,K", [(1, 72, 200), (5, 72, 200), (13, 71, 133), (300, 200, 136), (200, 129, 77)])
@pytest.mark.parametrize("keep", [1, 2])
def test_nothing_outside_the_outputs_is_written(sg, M, N, K, keep):
    """Outputs in larger buffers through the C entry, and a workspace of exactly the size asked for."""
    import ctypes
    lib, c, s = sg.load(), Case(M, N, K, "bf16"), torch.cuda.current_stream().cuda_stream
    for off, pad in ((0, 8), (1, 5)):
        bufs = []

        def out(rows, cols):
            flat = torch.full((off + rows * (cols + pad) + 64,), 7.0, dtype=c.dt, device="cuda")
            view = flat[off:off + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
            bufs.append((flat, view))
            return view

        def ws(backward, packed):
            n = ctypes.c_size_t(0)
            assert lib.sgemm_gated_ff_workspace(M, N, K, backward, packed, ctypes.byref(n)) == 0
            t = torch.full((n.value + 256,), 9, dtype=torch.uint8, device="cuda")
            return t, n.value

        h, dx, dwg, dwu, h2 = out(M, N), out(M, K), out(N, K), out(N, K), out(M, N)
        packed = 7 if K % 8 else 0
        if keep == 1:
            gate, up = out(M, N), out(M, N)
            k_at = (gate.data_ptr(), up.data_ptr(), N + pad, None, None)
        else:
            qs = [sg.act8_quantize(torch.zeros(M, N, device="cuda")) for _ in range(2)]
            k_at = (qs[0].codes.data_ptr(), qs[1].codes.data_ptr(), 0, qs[0].scales.data_ptr(),
                    qs[1].scales.data_ptr())
        # (Up to 16 tokens without 8-bit checkpoints: every matrix is read in place.)
        w, n = ws(0, 0 if M <= 16 and keep == 1 else packed)
        args = (M, N, K, 1, 0, c.x.data_ptr(), K, c.wg.data_ptr(), K, c.wu.data_ptr(), K, h.data_ptr(), N + pad,
                keep, *k_at)
        if n:
            assert lib.sgemm_gated_ff_forward(*args, None, n, s) == -6
            assert lib.sgemm_gated_ff_forward(*args, w.data_ptr(), n - 1, s) == -6
            assert lib.sgemm_gated_ff_forward(*args, w.data_ptr() + 16, n, s) == -6
        assert lib.sgemm_gated_ff_forward(*args, w.data_ptr(), n, s) == 0
        w2, n2 = ws(1, packed)
        args = (M, N, K, 1, 0, c.dh.data_ptr(), N, c.x.data_ptr(), K, None, None, c.wg.data_ptr(), K,
                c.wu.data_ptr(), K, keep, *k_at, dx.data_ptr(), K + pad, dwg.data_ptr(), K + pad,
                dwu.data_ptr(), K + pad, h2.data_ptr(), N + pad)
        assert lib.sgemm_gated_ff_backward(*args, w2.data_ptr(), n2 - 1, s) == -6
        assert lib.sgemm_gated_ff_backward(*args, None, n2, s) == -6
        assert lib.sgemm_gated_ff_backward(*args, w2.data_ptr(), n2, s) == 0
        torch.cuda.synchronize()
        assert bool((w[n:] == 9).all()) and bool((w2[n2:] == 9).all())
        want = sg.gated_ff(c.x, c.wg, c.wu, keep=("full", "8bit")[keep - 1])
        assert torch.equal(h, want[0])
        for got, ref in zip((dx, dwg, dwu, h2), sg.gated_ff_backward(c.dh, c.x, c.wg, c.wu, want[1],
                                                                    return_h=True)):
            assert torch.equal(got, ref)
        for flat, view in bufs:
            rest = flat.clone()
            rest[off:off + view.shape[0] * (view.shape[1] + pad)].view(
                view.shape[0], view.shape[1] + pad)[:, :view.shape[1]] = 7.0
            assert bool((rest == 7.0).all())


@pytest.mark.parametrize("M", [3, 300])
def test_odd_numbers_stay_in_their_row(sg, M):
    c = Case(M, 200, 136, "bf16")
    h0, kept0 = sg.gated_ff(c.x, c.wg, c.wu, keep="8bit")
    x = c.x.clone()
    x[1, 5], x[2, 100] = float("nan"), float("inf")
    h, kept = sg.gated_ff(x, c.wg, c.wu, keep="8bit")
    good = [i for i in range(M) if i not in (1, 2)]
    assert torch.equal(h[good], h0[good]) and bool(h[1].isnan().all())
    for a, b in zip(kept, kept0):
        assert torch.equal(a.codes[good], b.codes[good]) and bool(a.scales[1].isnan().all())
    dh = c.dh.clone()
    dh[1, 3] = float("nan")
    full = sg.gated_ff(c.x, c.wg, c.wu, keep="full")[1]
    got = sg.gated_ff_backward(dh, c.x, c.wg, c.wu, full)
    want = sg.gated_ff_backward(c.dh, c.x, c.wg, c.wu, full)
    assert torch.equal(got[0][good], want[0][good]) and bool(got[0][1].isnan().all())
    others = [i for i in range(200) if i != 3]
    assert torch.equal(got[1][others], want[1][others]) and bool(got[1][3].isnan().all())


def test_far_pre_activations(sg):
    """Gates of 10^3 and more, of either sign, and the largest numbers of the type: act is g or
    0 and its slope 1 or 0, without NaN."""
    for dt, top in ((torch.bfloat16, 1e30), (torch.float16, 6e4)):
        g = torch.tensor([[-top, -1000.0, -100.0, -30.0, 0.0, 30.0, 100.0, 1000.0]], device="cuda").to(dt)
        u, dh = torch.ones_like(g), torch.ones_like(g)
        eye = torch.zeros(8, 8, device="cuda", dtype=dt)
        x = torch.ones(1, 8, device="cuda", dtype=dt)
        for name in ("silu", "gelu_tanh"):
            dx, dwg, dwu, h = sg.gated_ff_backward(dh, x, eye, eye, (g, u), activation=name, return_h=True)
            want = torch.where(g > 0, g, torch.zeros_like(g)).float()
            assert bool(((h.float() - want).abs() <= 1e-11).all())
            slope = torch.tensor([0, 0, 0, 0, 0.5, 1, 1, 1], device="cuda")
            assert bool(((dwg.float() - slope[:, None]).abs() <= 1e-9).all())
            assert bool(torch.isfinite(dx).all()) and bool(torch.isfinite(dwu).all())


def test_no_tokens(sg):
    c = Case(4, 24, 40, "bf16")
    x, dh = c.x[:0], c.dh[:0]
    assert sg.gated_ff(x, c.wg, c.wu).shape == (0, 24)
    for keep in ("full", "8bit"):
        h, kept = sg.gated_ff(x, c.wg, c.wu, keep=keep)
        dx, dwg, dwu, h2 = sg.gated_ff_backward(dh, x, c.wg, c.wu, kept, return_h=True)
        assert dx.shape == (0, 40) and h2.shape == (0, 24)
        assert dwg.shape == (24, 40) and not bool(dwg.any()) and not bool(dwu.any())


def test_refusals(sg):
    c = Case(8, 24, 40, "bf16")
    x, wg, wu, dh = c.x, c.wg, c.wu, c.dh
    _, kept = sg.gated_ff(x, wg, wu, keep="full")
    _, k8 = sg.gated_ff(x, wg, wu, keep="8bit")
    for args in ((x.float(), wg, wu), (x, wg.half(), wu), (x, wg, wu[:23]), (x[:, :39], wg, wu), (x.t(), wg, wu),
                 (x, wg.t(), wu.t()), (x.cpu(), wg, wu), (x, wg.cpu(), wu), (x, wg[:0], wu[:0]),
                 (x[:, :0], wg[:, :0], wu[:, :0]), (x[0], wg, wu), (None, wg, wu)):
        with pytest.raises((TypeError, ValueError)):
            sg.gated_ff(*args)
    for kw in (dict(activation="relu"), dict(keep="fp8"), dict(activation=None)):
        with pytest.raises(ValueError):
            sg.gated_ff(x, wg, wu, **kw)
    q = sg.act8_quantize(x)
    for args in ((dh.half(), x, wg, wu, kept), (dh[:7], x, wg, wu, kept), (dh, x[:7], wg, wu, kept),
                 (dh[:, :23], x, wg, wu, kept), (dh, x, wg, wu, kept[:1]), (dh, x, wg, wu, None),
                 (dh, x, wg, wu, (kept[0], k8[1])), (dh, x, wg, wu, (k8[0], kept[1])), (dh, k8[0], wg, wu, kept),
                 (dh, x, wg, wu, (kept[0], kept[1].float())), (dh, x, wg, wu, (q, q)),
                 (dh, x, wg, wu, (kept[0], kept[1].clone(memory_format=torch.contiguous_format)[:7]))):
        with pytest.raises((TypeError, ValueError)):
            sg.gated_ff_backward(*args)
    # Checkpoints of another width whose padded rows are the same.
    wide = sg.act8_quantize(torch.zeros(8, 41, device="cuda"))
    for args in ((dh, wide, wg, wu, kept), (dh, x, wg, wu, (wide, wide))):
        with pytest.raises(ValueError):
            sg.gated_ff_backward(*args)


@pytest.mark.parametrize("M,N,K", [(140000, 16384, 64), (270000, 64, 8191)])
def test_long_offsets(sg, M, N, K):
    """More than 2^31 numbers in h, dh and what is kept, or in an x and a dx of unaligned rows: the
    last rows are their own.  Integers, so that every sum is exact in any order up to the result."""
    c = whole(Case(64, N, K, "bf16"))
    x, dh = torch.zeros(M, K, dtype=c.dt, device="cuda"), torch.zeros(M, N, dtype=c.dt, device="cuda")
    x[-64:], dh[-64:] = c.x, c.dh
    for keep in ("full", "8bit"):
        h, kept = sg.gated_ff(x, c.wg, c.wu, keep=keep)
        h0, kept0 = sg.gated_ff(c.x, c.wg, c.wu, keep=keep)
        assert torch.equal(h[-64:], h0) and not bool(h[:-64].any())
        for a, b in zip(kept, kept0):
            if keep == "full":
                assert torch.equal(a[-64:], b) and not bool(a[:-64].any())
            else:
                assert torch.equal(a.codes[-64:], b.codes) and torch.equal(a.scales[-64:], b.scales)
        del h
        got = sg.gated_ff_backward(dh, x, c.wg, c.wu, kept, return_h=True)
        want = sg.gated_ff_backward(c.dh, c.x, c.wg, c.wu, kept0, return_h=True)
        assert torch.equal(got[3][-64:], want[3]) and not bool(got[0][:-64].any())
        # (What is not an integer, slopes and numbers of 8 bits, makes sums that depend on their order:
        # both sides are within depth() of the magnitudes, and rounded once.)
        g, u = (q.dequantize().double() if keep == "8bit" else q.double() for q in kept0)
        a, slope = act(g, "silu")
        dg, du = (c.dh.double() * u * slope).abs() * 1.01, (c.dh.double() * a).abs() * 1.01
        bounds = ((got[0][-64:], want[0], depth(2 * N) * (dg @ c.wg.double().abs() + du @ c.wu.double().abs())),
                  (got[1], want[1], depth(M) * (dg.t() @ c.x.double().abs())),
                  (got[2], want[2], depth(M) * (du.t() @ c.x.double().abs())))
        for a, b, sum_off in bounds:
            b = b.double()
            tol = 2 * sum_off + 2 * c.u * 1.01 * (b.abs() + 2 * sum_off) + c.t
            assert bool(((a.double() - b).abs() <= tol).all())
        del kept, got


@pytest.mark.parametrize("M,N,K", [(300, 200, 136), (64, 8100, 72), (64, 8200, 72), (400, 2501, 72), (400, 2496, 72),
                                   (70, 7168, 64), (1300, 2560, 64), (7, 333, 72)])
def test_forward_alone_writes_its_result_only(sg, M, N, K):
    """h in a larger buffer through the C entry: tiles of every width, at the row's end and short of it."""
    lib, s = sg.load(), torch.cuda.current_stream().cuda_stream
    c = whole(Case(M, N, K, "bf16"))
    g, u = c.x.double() @ c.wg.double().t(), c.x.double() @ c.wu.double().t()
    for off, pad in ((0, 0), (0, 8), (1, 5)):
        flat = torch.full((off + M * (N + pad) + 64,), 7.0, dtype=c.dt, device="cuda")
        view = flat[off:off + M * (N + pad)].view(M, N + pad)[:, :N]
        assert lib.sgemm_gated_ff_forward(M, N, K, 1, 0, c.x.data_ptr(), K, c.wg.data_ptr(), K, c.wu.data_ptr(), K,
                                          view.data_ptr(), N + pad, 0, None, None, N, None, None, None, 0, s) == 0
        torch.cuda.synchronize()
        assert torch.equal(view, (g * u).to(c.dt))
        view.fill_(7.0)
        assert bool((flat == 7.0).all())
