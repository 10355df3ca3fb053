"""Measured cases of the 4-bit and norm operators: what a gated residual block with
4-bit linear layers runs around the library's products.

* ``quantize``: rows of fp32 / bf16 / fp16 numbers to 4-bit codes (e2m1) with one 8-bit
  scale per block of 16 (``nvfp4``: e4m3 scales) or 32 (``mxfp4``: powers of two)
  along a row, and back; also for the transpose of the stored matrix.
* ``matmul``: C[m, n] = alpha * sum_k A[m, k] B[n, k] of two quantised matrices.
* ``before``: the norm before a block, quantised in the same pass and multiplied by a
  4-bit weight; and the norm's gradient.
* ``after``: the norm after a block with its gate and residual scale, together with the
  norm before the next block; and the gradient of both.

``run`` computes each case from plain tensor operations in 32 bits, or, where ``own`` is
true, through the library's entry points.
"""
import math

import torch

own = False

BLOCK = {"nvfp4": 16, "mxfp4": 32}
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}
EPS = 1e-6


def listed():
    return [
        # One token's activations on the way into a 4-bit linear layer: latency.
        dict(name="quantize_token", op="quantize", rows=1, cols=4096, dtype="bf16", fmt="nvfp4",
             transposed=False, scaled=False),
        # A ragged fp32 matrix read transposed: the weight-gradient operand of odd sizes.
        dict(name="quantize_ragged_t", op="quantize", rows=3001, cols=1999, dtype="fp32",
             fmt="mxfp4", transposed=True, scaled=False),
        # A long prompt's activations, bandwidth.
        dict(name="quantize_large", op="quantize", rows=16384, cols=8192, dtype="bf16",
             fmt="nvfp4", transposed=False, scaled=True),
        # One token through a square layer: the weight is read once.
        dict(name="matmul_token", op="matmul", M=1, N=4096, K=4096, fmt="nvfp4", out="bf16"),
        # Many rows, few columns.
        dict(name="matmul_tall", op="matmul", M=16384, N=64, K=4096, fmt="mxfp4", out="fp32"),
        # Nothing a multiple of a tile.
        dict(name="matmul_ragged", op="matmul", M=3001, N=2047, K=1999, fmt="nvfp4", out="fp32"),
        # The large square product.
        dict(name="matmul_8192", op="matmul", M=8192, N=8192, K=8192, fmt="nvfp4", out="bf16"),
        # 16 sequences decoding: norm, quantise, multiply.
        dict(name="before_decode", op="before", rows=16, cols=4096, N=8192, dtype="bf16",
             fmt="nvfp4"),
        # Training: gradient of the norm before a block, joined with the residual's.
        dict(name="before_grad", op="before_grad", rows=8192, cols=4096, dtype="bf16"),
        # One token between two blocks.
        dict(name="after_token", op="after", rows=1, cols=4096, dtype="bf16", gate="rows"),
        # A training batch between two blocks.
        dict(name="after_large", op="after", rows=8192, cols=8192, dtype="bf16", gate="rows"),
        # Its gradient at odd sizes, in fp32, with one gate for all rows.
        dict(name="after_grad_ragged", op="after_grad", rows=3001, cols=2047, dtype="fp32",
             gate="shared"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["quantize", "quantize", "matmul", "matmul", "matmul", "before",
                     "before_grad", "after", "after_grad"])
    fmt = rng.choice(["nvfp4", "mxfp4"])
    dtype = rng.choice(["fp32", "bf16", "bf16", "fp16"])
    gate = rng.choice(["none", "rows", "shared"])
    if op == "matmul":
        M, N, K = _log(rng, 1, 16384), _log(rng, 16, 16384), _log(rng, 16, 16384)
        while M * N * K > 8192 ** 3:
            M = (M + 1) // 2
        return dict(op=op, M=M, N=N, K=K, fmt=fmt, out=rng.choice(["fp32", "bf16", "fp16"]))
    cols = _log(rng, 16, 16384)
    if rng.random() < 0.6:          # hidden sizes are mostly multiples of 64
        cols = max(64, cols // 64 * 64)
    rows = _log(rng, 1, max(1, min(16384, (1 << 26) // cols)))
    if op == "quantize":
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, fmt=fmt,
                    transposed=rng.random() < 0.4, scaled=fmt == "nvfp4" and rng.random() < 0.5)
    if op == "before":
        rows = min(rows, 4096)
        return dict(op=op, rows=rows, cols=cols, N=_log(rng, 16, 8192),
                    dtype=rng.choice(["bf16", "fp16"]), fmt=fmt)
    if op == "before_grad":
        return dict(op=op, rows=rows, cols=cols, dtype=dtype)
    return dict(op=op, rows=rows, cols=cols, dtype=dtype, gate=gate)


def _up(n, m):
    return -(-n // m) * m


def work(case):
    """Bytes and operations of one pass: inputs read once, outputs written once."""
    op = case["op"]
    if op == "matmul":
        M, N, K = case["M"], case["N"], case["K"]
        per = 0.5 + 1 / BLOCK[case["fmt"]]
        return {"bytes": (M + N) * K * per + M * N * SIZE[case["out"]], "flops": 2.0 * M * N * K}
    n, s = case["rows"] * case["cols"], SIZE[case["dtype"]]
    if op == "quantize":            # values in; codes and scales out; values back out
        return {"bytes": n * (s + 0.5 + 1 / BLOCK[case["fmt"]] + 2), "flops": 4.0 * n}
    if op == "before":
        per = 0.5 + 1 / BLOCK[case["fmt"]]
        return {"bytes": n * s + case["cols"] * 4 + case["N"] * case["cols"] * per
                + case["rows"] * case["N"] * 2,
                "flops": 2.0 * n * case["N"] + 6.0 * n}
    if op == "before_grad":         # dh, x, dy in; dx out
        return {"bytes": 4.0 * n * s + 8 * case["cols"], "flops": 12.0 * n}
    full = 1 if case["gate"] == "rows" else 0
    if op == "after":               # block, residual (and gate) in; y and h out
        return {"bytes": n * s * (4.0 + full) + 8 * case["cols"], "flops": 12.0 * n}
    # dy, dh, block, y (and gate) in; dresidual, dblock (and dgate) out
    return {"bytes": n * s * (6.0 + 2 * full) + 20 * case["cols"], "flops": 28.0 * n}


# ----------------------------------------------------------------------------
# The 4-bit format in plain tensor operations
# ----------------------------------------------------------------------------
def _levels(v):
    """v rounded to the e2m1 values (0, .5, 1, 1.5, 2, 3, 4, 6), ties to even."""
    a = v.abs()
    r = torch.where(a < 2, torch.round(a * 2) / 2,
                    torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2))
    return torch.copysign(r.clamp(max=6.0), v)


def _plain_quantize(x, fmt, ts):
    """(e2m1 values, scales as fp32) of the rows of x, padded to whole blocks."""
    B = BLOCK[fmt]
    x = x.float()
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, _up(cols, B) - cols)).view(rows, -1, B)
    amax = x.abs().amax(dim=2)
    bad = ~torch.isfinite(amax)
    if fmt == "mxfp4":
        e = (torch.frexp(amax).exponent - 3).clamp(-127, 127)
        e = torch.where(amax > 0, e, torch.full_like(e, -127))
        s = torch.ldexp(torch.ones_like(amax, dtype=torch.float64), e).float()
        v = x / s.unsqueeze(2)
    else:
        t = amax / (6.0 * ts) if ts is not None else amax / 6.0
        s = t.clamp(max=448.0).to(torch.float8_e4m3fn).float()
        d = s * ts if ts is not None else s
        v = x / d.unsqueeze(2)
        v = torch.where((d == 0).unsqueeze(2), torch.zeros_like(v), v)
    s = torch.where(bad, torch.full_like(s, float("nan")), s)
    return _levels(v), s


def _plain_values(q, s, ts, cols):
    v = q * s.unsqueeze(2)
    if ts is not None:
        v = v * ts
    return v.reshape(v.shape[0], -1)[:, :cols]


def _encode(q, s, fmt):
    """The stored form: codes (row blocks of 128, chunks of 32 columns, 128 rows, 16 bytes)
    and scales (row blocks, groups of 4, row % 32, row / 32, 4), zero where padded."""
    rows, nb, B = q.shape
    K = nb * B
    a = q.abs()
    code = torch.where(a <= 2, (a * 2).round(),
                       torch.where(a <= 4, a + 2, torch.full_like(a, 7.0))).to(torch.uint8)
    code = code + 8 * torch.signbit(q).to(torch.uint8)
    R, Kp = _up(rows, 128), _up(K, 128)
    full = torch.zeros((R, Kp), dtype=torch.uint8, device=q.device)
    full[:rows, :K] = code.view(rows, K)
    byte = full[:, 0::2] | (full[:, 1::2] << 4)
    codes = byte.view(R // 128, 128, Kp // 32, 16).transpose(1, 2).contiguous()
    if fmt == "nvfp4":
        sb = s.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        sb = (torch.frexp(s.double()).exponent + 126).to(torch.uint8)
    sf = torch.zeros((R, Kp // B), dtype=torch.uint8, device=q.device)
    sf[:rows, :nb] = sb
    sf = sf.view(R // 128, 4, 32, Kp // B // 4, 4).permute(0, 3, 2, 1, 4).contiguous()
    return codes, sf


def _decode(codes, sf, rows, cols, fmt, ts):
    """fp32 values of the stored form."""
    B = BLOCK[fmt]
    R, Kp = codes.shape[0] * 128, codes.shape[1] * 32
    byte = codes.transpose(1, 2).reshape(R, Kp // 2)[:rows]
    code = torch.stack((byte & 15, byte >> 4), dim=2).view(rows, Kp)
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                         device=codes.device)
    q = table[code.int()]
    sb = sf.permute(0, 3, 2, 1, 4).reshape(R, Kp // B)[:rows]
    s = sb.view(torch.float8_e4m3fn).float() if fmt == "nvfp4" else \
        torch.pow(2.0, sb.double() - 127).float()
    return _plain_values(q.view(rows, -1, B), s, ts, cols)


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    return g


def _activations(g, rows, cols, dtype):
    """Normal numbers with a spread of channel sizes and a few large channels."""
    x = torch.randn((rows, cols), generator=g, device="cuda")
    c = torch.randn((cols,), generator=g, device="cuda").mul_(0.5).exp_()
    c = torch.where(torch.rand((cols,), generator=g, device="cuda") < 0.01, c * 8, c)
    return x.mul_(c).to(dtype)


def _norm_weight(g, cols):
    return torch.randn((cols,), generator=g, device="cuda").mul_(0.2).add_(1.0)


def _weight(g, n, k, fmt):
    """A layer's weight, quantised once, with its scale over the whole tensor."""
    w = torch.randn((n, k), generator=g, device="cuda").mul_(1 / math.sqrt(k))
    ts = (w.abs().amax() / (6 * 448)).view(1) if fmt == "nvfp4" else None
    q, s = _plain_quantize(w, fmt, ts)
    codes, sf = _encode(q, s, fmt)
    return codes, sf, ts


def _rstd(x):
    return torch.rsqrt(x.float().square().mean(dim=1) + EPS)


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    op = case["op"]
    if op == "matmul":
        x = _activations(g, case["M"], case["K"], torch.bfloat16)
        q, s = _plain_quantize(x, case["fmt"], None)
        st["a"] = _encode(q, s, case["fmt"]) + (None,)
        st["b"] = _weight(g, case["N"], case["K"], case["fmt"])
        return st
    rows, cols, dt = case["rows"], case["cols"], DTYPES[case["dtype"]]
    if op == "quantize":
        # Transposed: the matrix is stored (cols, rows) and read through its transpose.
        shape = (cols, rows) if case["transposed"] else (rows, cols)
        x = _activations(g, *shape, dt)
        st["x"] = x.t() if case["transposed"] else x
        if case["scaled"]:          # calibrated on other data: near this tensor's own
            near = torch.rand((1,), generator=g, device="cuda").mul_(0.4).add_(0.8)
            st["ts"] = x.float().abs().amax() * near / (6 * 448)
        else:
            st["ts"] = None
        return st
    st["w"] = _norm_weight(g, cols)
    if op == "before":
        st["x"] = _activations(g, rows, cols, dt)
        st["lin"] = _weight(g, case["N"], cols, case["fmt"])
        return st
    if op == "before_grad":
        st["x"] = _activations(g, rows, cols, dt)
        st["rstd"] = _rstd(st["x"])
        st["dh"] = torch.randn((rows, cols), generator=g, device="cuda").to(dt)
        st["dy"] = torch.randn((rows, cols), generator=g, device="cuda").to(dt)
        return st
    st["block"] = _activations(g, rows, cols, dt)
    st["next_w"] = _norm_weight(g, cols)
    shape = {"none": None, "rows": (rows, cols), "shared": (cols,)}[case["gate"]]
    st["gate"] = None if shape is None else \
        torch.randn(shape, generator=g, device="cuda").sigmoid_().to(dt)
    st["scale"] = 0.5
    if op == "after":
        st["residual"] = _activations(g, rows, cols, dt)
        return st
    st["y"] = _activations(g, rows, cols, dt)
    st["rstd"], st["next_rstd"] = _rstd(st["block"]), _rstd(st["y"])
    st["dy"] = torch.randn((rows, cols), generator=g, device="cuda").to(dt)
    st["dh"] = torch.randn((rows, cols), generator=g, device="cuda").to(dt)
    return st


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------
def run(st):
    return _own(st) if own else _plain(st)


def _own(st):
    import dense_fp32_gemm_09_gb300 as sg
    op = st["op"]
    if op == "quantize":
        q = sg.mx4_quantize(st["x"], st["fmt"], tensor_scale=st["ts"])
        return sg.mx4_dequantize(q, torch.bfloat16)
    if op == "matmul":
        a = sg.Mx4(*st["a"][:2], st["M"], st["K"], st["fmt"], st["a"][2])
        b = sg.Mx4(*st["b"][:2], st["N"], st["K"], st["fmt"], st["b"][2])
        return sg.mx4_matmul(a, b, dtype=DTYPES[st["out"]])
    if op == "before":
        w = sg.Mx4(*st["lin"][:2], st["N"], st["cols"], st["fmt"], st["lin"][2])
        h, rstd = sg.norm_before(st["x"], st["w"], eps=EPS, quantize=st["fmt"])
        return sg.mx4_matmul(h, w, dtype=torch.bfloat16), rstd
    if op == "before_grad":
        return sg.norm_before_backward(st["dh"], st["x"], st["rstd"], st["w"], dy=st["dy"])
    if op == "after":
        return sg.norm_after(st["block"], st["residual"], st["w"], gate=st["gate"],
                             scale=st["scale"], eps=EPS, next_weight=st["next_w"])
    return sg.norm_after_backward(st["dy"], st["block"], st["rstd"], st["w"], gate=st["gate"],
                                  scale=st["scale"], dh=st["dh"], y=st["y"],
                                  next_rstd=st["next_rstd"], next_weight=st["next_w"])


def _norm_grad(dh, x, rstd, w):
    """(gradient of x, gradient of w) of h = x * rstd * w, rstd a function of x."""
    n = x * rstd.unsqueeze(1)
    g = dh * w
    return (g - n * (g * n).mean(dim=1, keepdim=True)) * rstd.unsqueeze(1), (dh * n).sum(dim=0)


def _plain(st):
    op = st["op"]
    if op == "quantize":
        q, s = _plain_quantize(st["x"], st["fmt"], st["ts"])
        return _plain_values(q, s, st["ts"], st["cols"]).to(torch.bfloat16)
    if op == "matmul":
        a = _decode(*st["a"][:2], st["M"], st["K"], st["fmt"], st["a"][2])
        b = _decode(*st["b"][:2], st["N"], st["K"], st["fmt"], st["b"][2])
        return (a @ b.t()).to(DTYPES[st["out"]])
    dt = DTYPES[st["dtype"]]
    if op == "before":
        x = st["x"].float()
        rstd = _rstd(x)
        q, s = _plain_quantize(x * rstd.unsqueeze(1) * st["w"], st["fmt"], None)
        h = _plain_values(q, s, None, st["cols"])
        w = _decode(*st["lin"][:2], st["N"], st["cols"], st["fmt"], st["lin"][2])
        return (h @ w.t()).to(torch.bfloat16), rstd
    if op == "before_grad":
        dx, dw = _norm_grad(st["dh"].float(), st["x"].float(), st["rstd"], st["w"])
        return (dx + st["dy"].float()).to(dt), dw
    b = st["block"].float()
    gate = 1.0 if st["gate"] is None else st["gate"].float()
    if op == "after":
        rstd = _rstd(b)
        y = st["residual"].float() + st["scale"] * gate * (b * rstd.unsqueeze(1) * st["w"])
        next_rstd = _rstd(y)
        h = y * next_rstd.unsqueeze(1) * st["next_w"]
        return y.to(dt), rstd, h.to(dt), next_rstd
    dx, dnext_w = _norm_grad(st["dh"].float(), st["y"].float(), st["next_rstd"], st["next_w"])
    dx = dx + st["dy"].float()
    db, dw = _norm_grad(st["scale"] * gate * dx, b, st["rstd"], st["w"])
    dgate = None
    if st["gate"] is not None:
        dgate = st["scale"] * dx * (b * st["rstd"].unsqueeze(1) * st["w"])
        dgate = dgate.sum(dim=0) if st["gate"].dim() == 1 else dgate.to(dt)
    return dx.to(dt), db.to(dt), dw, dgate, dnext_w


# ----------------------------------------------------------------------------
# The definitions in 64 bits
# ----------------------------------------------------------------------------
def _e4m3_table():
    v = [m * 2.0 ** -9 for m in range(8)]
    v += [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64, device="cuda")


def _nearest(v, table):
    """The entry of the ascending table nearest to v >= 0; halfway, the even index."""
    mid = (table[1:] + table[:-1]) / 2
    low, high = torch.bucketize(v, mid), torch.bucketize(v, mid, right=True)
    return table[torch.where(high > low, torch.where(low % 2 == 0, low, high), low)]


def _exact_quantized(x, fmt, ts):
    """The values that quantising the rows of x leaves, in 64 bits."""
    B = BLOCK[fmt]
    x = x.double()
    rows, cols = x.shape
    blocks = torch.zeros((rows, _up(cols, B)), dtype=torch.float64, device=x.device)
    blocks[:, :cols] = x
    blocks = blocks.view(rows, -1, B)
    amax = blocks.abs().max(dim=2, keepdim=True).values
    whole = 1.0 if ts is None else ts.double()
    if fmt == "nvfp4":
        s = _nearest(amax / (6 * whole), _e4m3_table()) * whole
    else:
        s = torch.exp2((torch.floor(torch.log2(amax.clamp(min=1e-300))) - 2).clamp(min=-127))
    e2m1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    q = _nearest(torch.where(s > 0, blocks.abs() / s, torch.zeros_like(blocks)), e2m1)
    return (q * blocks.sign() * s).view(rows, -1)[:, :cols]


def _exact_stored(stored, rows, cols, fmt):
    """The values of a stored matrix, element by element from its layout, in 64 bits."""
    codes, sf, ts = stored
    r = torch.arange(rows, device="cuda").unsqueeze(1)
    k = torch.arange(cols, device="cuda").unsqueeze(0)
    byte = codes[r // 128, k // 32, r % 128, k % 32 // 2]
    code = torch.where(k % 2 == 1, byte >> 4, byte & 15).long()
    e2m1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")
    v = torch.where(code > 7, -1.0, 1.0) * e2m1[code & 7]
    del byte, code
    g = k // BLOCK[fmt]
    b = sf[r // 128, g // 4, r % 32, r % 128 // 32, g % 4].long()
    v = v * (_e4m3_table()[b] if fmt == "nvfp4" else torch.exp2(b.double() - 127))
    return v if ts is None else v * ts.double()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = st["x"]
        step = max(1, (1 << 24) // case["cols"])
        return torch.cat([_exact_quantized(x[i:i + step], case["fmt"], st["ts"]).float()
                          for i in range(0, case["rows"], step)])
    if op == "matmul":
        a = _exact_stored(st["a"], case["M"], case["K"], case["fmt"])
        b = _exact_stored(st["b"], case["N"], case["K"], case["fmt"])
        return torch.einsum("mk,nk->mn", a, b)
    rows = st["x" if "x" in st else "block"].shape[0]
    if op == "before":
        x = st["x"].double()
        rstd = 1 / torch.sqrt((x * x).sum(dim=1) / x.shape[1] + EPS)
        # The quantised numbers follow from the 32-bit norm of the definition.
        h = _exact_quantized(x * rstd.view(rows, 1) * st["w"].double(), case["fmt"], None)
        w = _exact_stored(st["lin"], case["N"], case["cols"], case["fmt"])
        return torch.einsum("mk,nk->mn", h, w), rstd
    D = case["cols"]

    def grad(dh, x, r, w):
        """By the formula: dx_j = r w_j dh_j - x_j r^3 / D sum_i w_i dh_i x_i."""
        r = r.double().view(rows, 1)
        dot = torch.einsum("rd,d,rd->r", dh, w, x).view(rows, 1)
        return r * w * dh - x * r ** 3 * dot / D, torch.einsum("rd,rd->d", dh, x * r)

    if op == "before_grad":
        dx, dw = grad(st["dh"].double(), st["x"].double(), st["rstd"], st["w"].double())
        return dx + st["dy"].double(), dw
    b, w, nw = st["block"].double(), st["w"].double(), st["next_w"].double()
    gate = torch.ones(D, dtype=torch.float64, device="cuda") if st["gate"] is None \
        else st["gate"].double()
    if op == "after":
        r = 1 / torch.sqrt((b * b).sum(dim=1) / D + EPS)
        y = st["residual"].double() + st["scale"] * gate * b * w * r.view(rows, 1)
        nr = 1 / torch.sqrt((y * y).sum(dim=1) / D + EPS)
        return y, r, y * nw * nr.view(rows, 1), nr
    dx, dnw = grad(st["dh"].double(), st["y"].double(), st["next_rstd"], nw)
    dx = dx + st["dy"].double()
    db, dw = grad(dx * gate * st["scale"], b, st["rstd"], w)
    dgate = None
    if st["gate"] is not None:
        dgate = dx * b * w * st["rstd"].double().view(rows, 1) * st["scale"]
        dgate = dgate.sum(dim=0) if st["gate"].dim() == 1 else dgate
    return dx, db, dw, dgate, dnw
