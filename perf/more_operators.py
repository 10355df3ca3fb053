"""Measured cases of the operators of a pre-norm feed-forward block and of what its training
keeps.

* ``ln``: layer norm, its gradient with the sums for weight and bias, and both with the
  norm's input kept in 8 bits in between.
* ``act8``: a matrix to 8-bit codes with one scale per 64 columns of a row, and back.
* ``ff``: the gated feed-forward block act(x Wg^T) * (x Wu^T), its gradient, and both
  with the block's input and pre-activations kept in 8 bits in between.

``run`` computes each case from plain tensor operations in 32 bits, or, where ``own`` is
true, through the library's entry points.
"""
import math

import torch

own = False

BLOCK = 64
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}
EPS = 1e-5


def listed():
    return [
        # One token between two layers: latency.
        dict(name="ln_token", op="ln", rows=1, cols=4096, dtype="bf16"),
        # A long prompt, bandwidth.
        dict(name="ln_large", op="ln", rows=16384, cols=8192, dtype="bf16"),
        # Training: the norm's gradient, joined with the residual's.
        dict(name="ln_grad", op="ln_grad", rows=8192, cols=4096, dtype="bf16"),
        # Odd sizes in fp32: forward, input kept in 8 bits, backward from that.
        dict(name="ln_train_ragged", op="ln_train", rows=3001, cols=2047, dtype="fp32"),
        # A checkpoint of odd sizes, written and read.
        dict(name="act8_ragged", op="act8", rows=3001, cols=1999, dtype="fp32"),
        # A layer's activations of a large batch, written and read.
        dict(name="act8_large", op="act8", rows=16384, cols=8192, dtype="bf16"),
        # One token: both weights are read once.
        dict(name="ff_token", op="ff", M=1, K=4096, N=8192, dtype="bf16", act="silu"),
        # 16 sequences decoding.
        dict(name="ff_decode", op="ff", M=16, K=4096, N=16384, dtype="fp16", act="silu"),
        # Nothing a multiple of a tile, rows that are not 16-byte aligned.
        dict(name="ff_ragged", op="ff", M=3001, K=2047, N=1999, dtype="fp16", act="gelu_tanh"),
        # A long prompt.
        dict(name="ff_prompt", op="ff", M=8192, K=4096, N=16384, dtype="bf16", act="silu"),
        # A small training step, pre-activations kept as they are.
        dict(name="ff_train_small", op="ff_train", M=500, K=1024, N=4096, dtype="bf16",
             act="gelu_tanh", keep="full"),
        # A large one with everything kept in 8 bits.
        dict(name="ff_train", op="ff_train", M=8192, K=4096, N=8192, dtype="bf16", act="silu",
             keep="8bit"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _width(rng, hi):
    n = _log(rng, 16, hi)
    return max(64, n // 64 * 64) if rng.random() < 0.6 else n    # mostly multiples of 64


def draw(rng):
    op = rng.choice(["ln", "ln_grad", "ln_train", "act8", "ff", "ff", "ff", "ff_train",
                     "ff_train"])
    if op.startswith("ff"):
        M, K, N = _log(rng, 1, 16384), _width(rng, 8192), _width(rng, 16384)
        while M * N * K > (1 << 39 if op == "ff" else 1 << 38):
            M = (M + 1) // 2
        case = dict(op=op, M=M, K=K, N=N, dtype=rng.choice(["bf16", "bf16", "fp16"]),
                    act=rng.choice(["silu", "gelu_tanh"]))
        if op == "ff_train":
            case["keep"] = rng.choice(["full", "8bit"])
        return case
    cols = _width(rng, 16384)
    rows = _log(rng, 1, max(1, min(16384, (1 << 27) // cols)))
    return dict(op=op, rows=rows, cols=cols, dtype=rng.choice(["fp32", "bf16", "bf16", "fp16"]))


def work(case):
    """Bytes and operations of one pass: inputs read once, outputs written once."""
    op = case["op"]
    if op.startswith("ff"):
        M, K, N = case["M"], case["K"], case["N"]
        if op == "ff":                  # x and both weights in, h out
            return {"bytes": 2.0 * (M * K + 2 * N * K + M * N), "flops": 4.0 * M * N * K}
        # Weights and x in, h out; dh in; dx and both gradients out (and h once more).
        again = M * N if case["keep"] == "8bit" else 0
        return {"bytes": 2.0 * (2 * M * K + 4 * N * K + 2 * M * N + again),
                "flops": 12.0 * M * N * K}
    n, s, D = case["rows"] * case["cols"], SIZE[case["dtype"]], case["cols"]
    if op == "act8":                    # values in; codes and scales out; values back out
        return {"bytes": n * (2 * s + 1 + 4 / BLOCK), "flops": 4.0 * n}
    if op == "ln":
        return {"bytes": 2.0 * n * s + 8 * D, "flops": 8.0 * n}
    if op == "ln_grad":                 # dh, x, dy in; dx out
        return {"bytes": 4.0 * n * s + 12 * D, "flops": 14.0 * n}
    # x in, y out; dh and dy in, dx out
    return {"bytes": 5.0 * n * s + 20 * D, "flops": 26.0 * n}


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _activations(g, rows, cols, dtype):
    """Normal numbers with a mean, a spread of channel sizes and a few large channels."""
    x = _normal(g, rows, cols)
    c = _normal(g, cols).mul_(0.5).exp_()
    c = torch.where(torch.rand((cols,), generator=g, device="cuda") < 0.01, c * 8, c)
    return x.mul_(c).add_(_normal(g, cols).mul_(0.3).add_(0.5)).to(dtype)


def _moments(x):
    x = x.double()
    m = x.mean(dim=1)
    return m.float(), ((x - m.unsqueeze(1)).square().mean(dim=1) + EPS).rsqrt().float()


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    op, dt = case["op"], DTYPES[case["dtype"]]
    if op.startswith("ff"):
        M, K, N = case["M"], case["K"], case["N"]
        st["x"] = _normal(g, M, K).to(dt)
        st["wg"] = _normal(g, N, K).mul_(1 / math.sqrt(K)).to(dt)
        st["wu"] = _normal(g, N, K).mul_(1 / math.sqrt(K)).to(dt)
        if op == "ff_train":
            st["dh"] = _normal(g, M, N).to(dt)
        return st
    rows, cols = case["rows"], case["cols"]
    st["x"] = _activations(g, rows, cols, dt)
    if op == "act8":
        return st
    st["w"] = _normal(g, cols).mul_(0.2).add_(1.0)
    st["b"] = _normal(g, cols).mul_(0.2)
    if op != "ln":
        st["dh"] = _normal(g, rows, cols).to(dt)
        st["dy"] = _normal(g, rows, cols).to(dt)
    if op == "ln_grad":
        st["mean"], st["rstd"] = _moments(st["x"])
    return st


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------
def run(st):
    return _own(st) if own else _plain(st)


def _own(st):
    import dense_fp32_gemm_09_gb300 as sg
    op, x = st["op"], st["x"]
    if op == "ln":
        return sg.layer_norm(x, st["w"], st["b"], eps=EPS)
    if op == "ln_grad":
        return sg.layer_norm_backward(st["dh"], x, st["mean"], st["rstd"], st["w"], dy=st["dy"])
    if op == "ln_train":
        y, mean, rstd, kept = sg.layer_norm(x, st["w"], st["b"], eps=EPS, keep="8bit")
        return (y, mean, rstd) + sg.layer_norm_backward(st["dh"], kept, mean, rstd, st["w"],
                                                        dy=st["dy"])
    if op == "act8":
        return sg.act8_dequantize(sg.act8_quantize(x), DTYPES[st["dtype"]])
    if op == "ff":
        return sg.gated_ff(x, st["wg"], st["wu"], activation=st["act"])
    if st["keep"] == "full":
        h, kept = sg.gated_ff(x, st["wg"], st["wu"], activation=st["act"], keep="full")
        return (h,) + sg.gated_ff_backward(st["dh"], x, st["wg"], st["wu"], kept,
                                           activation=st["act"])
    h, kept = sg.gated_ff(x, st["wg"], st["wu"], activation=st["act"], keep="8bit")
    return (h,) + sg.gated_ff_backward(st["dh"], sg.act8_quantize(x), st["wg"], st["wu"], kept,
                                       activation=st["act"], return_h=True)


def _kept(x):
    """The fp32 values that 8 bits hold: codes rint(x * (127 / amax)) of blocks along a row,
    times amax / 127; zeros where amax is under 2^-100."""
    rows, cols = x.shape
    v = torch.nn.functional.pad(x.float(), (0, -cols % BLOCK)).view(rows, -1, BLOCK)
    amax = v.abs().amax(dim=2, keepdim=True)
    top = torch.full_like(amax, 127.0)
    live = amax >= 2.0 ** -100
    code = torch.round(v * torch.where(live, top / amax, torch.zeros_like(amax)))
    scale = torch.where(live, amax / top, torch.zeros_like(amax))
    bad = ~torch.isfinite(amax)
    scale = torch.where(bad, torch.full_like(scale, float("nan")), scale)
    code = torch.where(bad, torch.zeros_like(code), code)
    return (code * scale).view(rows, -1)[:, :cols]


def _norm(x):
    """(rows less their mean, mean, rstd)."""
    m = x.mean(dim=1, keepdim=True)
    d = x - m
    return d, m, torch.rsqrt(d.square().mean(dim=1, keepdim=True) + EPS)


def _norm_grad(dh, x, m, r, w, dy, dt):
    n = (x - m) * r
    g = dh.float() * w
    dx = (g - g.mean(dim=1, keepdim=True) - n * (g * n).mean(dim=1, keepdim=True)) * r + dy.float()
    return dx.to(dt), (dh.float() * n).sum(dim=0), dh.float().sum(dim=0)


def _act(g, name):
    """(act(g), its derivative)."""
    if name == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    c = math.sqrt(2 / math.pi)
    s = 1 / (1 + torch.exp(-2 * c * (g + 0.044715 * g * g * g)))
    return g * s, s + g * s * (1 - s) * 2 * c * (1 + 3 * 0.044715 * g * g)


def _plain(st):
    op, dt = st["op"], DTYPES[st["dtype"]]
    if op == "act8":
        return _kept(st["x"]).to(dt)
    if op in ("ln", "ln_train"):
        x = st["x"].float()
        d, m, r = _norm(x)
        y = (d * r * st["w"] + st["b"]).to(dt)
        out = (y, m.squeeze(1), r.squeeze(1))
        if op == "ln":
            return out
        return out + _norm_grad(st["dh"], _kept(x), m, r, st["w"], st["dy"], dt)
    if op == "ln_grad":
        return _norm_grad(st["dh"], st["x"].float(), st["mean"].unsqueeze(1),
                          st["rstd"].unsqueeze(1), st["w"], st["dy"], dt)
    x, wg, wu = st["x"].float(), st["wg"].float(), st["wu"].float()
    g, u = x @ wg.t(), x @ wu.t()
    a, _ = _act(g, st["act"])
    h = (a * u).to(dt)
    if op == "ff":
        return h
    if st["keep"] == "full":
        g, u = g.to(dt).float(), u.to(dt).float()
    else:
        g, u, x = _kept(g), _kept(u), _kept(x)
    dh = st["dh"].float()
    a, slope = _act(g, st["act"])
    dg, du = dh * u * slope, dh * a
    out = (h, (dg @ wg + du @ wu).to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt))
    return out + ((a * u).to(dt),) if st["keep"] == "8bit" else out


# ----------------------------------------------------------------------------
# The definitions in 64 bits
# ----------------------------------------------------------------------------
def _exact_kept(x):
    """Block by block of columns: scale and reciprocal are fp32 numbers of the definition, and
    a code is the nearest integer to an fp32 product."""
    x = x.double()
    out = torch.empty_like(x)
    for c in range(0, x.shape[1], BLOCK):
        part = x[:, c:c + BLOCK]
        amax = part.abs().max(dim=1, keepdim=True).values.float().double()
        inverse = (127 / amax.clamp(min=2.0 ** -100)).float().double()
        q = torch.round((part * inverse).float().double())
        out[:, c:c + BLOCK] = torch.where(amax < 2.0 ** -100, 0.0, 1.0) * q * (amax / 127).float()
    return out


def _exact_act(g, name):
    """(act(g), its derivative) through tanh: sigmoid(t) = (1 + tanh(t / 2)) / 2."""
    if name == "silu":
        th = torch.tanh(g / 2)
        return g / 2 * (1 + th), (1 + th) / 2 + g / 4 * (1 - th * th)
    c = math.sqrt(2 / math.pi)
    th = torch.tanh(c * (g + 0.044715 * g ** 3))
    return g / 2 * (1 + th), (1 + th) / 2 + g / 2 * (1 - th * th) * c * (1 + 0.134145 * g ** 2)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    x = st["x"].double()
    if op == "act8":
        return _exact_kept(x)
    if op in ("ln", "ln_grad", "ln_train"):
        R, D = x.shape
        w, b = st["w"].double(), st["b"].double()
        out = ()
        if op == "ln_grad":
            m, r = st["mean"].double(), st["rstd"].double()
        else:
            m = x.sum(dim=1) / D
            r = 1 / torch.sqrt((x - m.view(R, 1)).pow(2).sum(dim=1) / D + EPS)
            out = (torch.addcmul(b - w * (m * r).view(R, 1), x, w * r.view(R, 1)), m, r)
            if op == "ln":
                return out
            x = _exact_kept(x)
        # dx_j = r w_j dh_j - r / D sum_i w_i dh_i - (x_j - m) r^3 / D sum_i w_i dh_i (x_i - m)
        dh, x = st["dh"].double(), x - m.view(R, 1)
        one = torch.einsum("rd,d->r", dh, w)
        two = torch.einsum("rd,d,rd->r", dh, w, x)
        dx = dh * w * r.view(R, 1) - (r * one / D).view(R, 1) - x * (r ** 3 * two / D).view(R, 1)
        return out + (dx + st["dy"].double(), torch.einsum("rd,rd,r->d", dh, x, r), dh.sum(dim=0))
    wg, wu = st["wg"].double(), st["wu"].double()
    g, u = torch.einsum("mk,nk->mn", x, wg), torch.einsum("mk,nk->mn", x, wu)
    h = _exact_act(g, st["act"])[0].mul_(u)
    if op == "ff":
        return h
    if st["keep"] == "full":            # kept in the type of x
        g, u = (t.to(st["x"].dtype).double() for t in (g, u))
    else:
        g, u, x = _exact_kept(g), _exact_kept(u), _exact_kept(x)
    a, slope = _exact_act(g, st["act"])
    dh = st["dh"].double()
    du, dg = dh * a, dh * slope * u
    out = (h, torch.einsum("mn,nk->mk", dg, wg) + torch.einsum("mn,nk->mk", du, wu),
           torch.einsum("mn,mk->nk", dg, x), torch.einsum("mn,mk->nk", du, x))
    return out + (a * u,) if st["keep"] == "8bit" else out
