"""The 4-bit formats restated with numpy, element by element (test infrastructure).

Quotients are fp32 divisions as the format defines them; everything after is exact."""
import numpy as np

BLOCK = {"nvfp4": 16, "mxfp4": 32}
E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] +
                [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)])[:127]


def nearest(v, table):
    """Index of the entry of an ascending table nearest to v >= 0, ties to even."""
    mid = (table[1:] + table[:-1]) / 2
    lo, hi = np.searchsorted(mid, v, "left"), np.searchsorted(mid, v, "right")
    return np.where((hi > lo) & (lo % 2 == 1), hi, lo)


def quantize(x, fmt, ts=None):
    """(codes 0..15 and scale bytes) of the rows of x, padded to whole blocks."""
    B = BLOCK[fmt]
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    nb = -(-cols // B)
    v = np.zeros((rows, nb * B), np.float32)
    v[:, :cols] = x
    v = v.reshape(rows, nb, B)
    bad = ~np.isfinite(v).all(axis=2)
    a = np.abs(np.where(np.isfinite(v), v, 0))
    amax = a.max(axis=2, initial=0).astype(np.float32)
    t = np.float32(1 if ts is None else ts)
    with np.errstate(all="ignore"):
        if fmt == "nvfp4":
            sb = nearest((amax / (np.float32(6) * t)).astype(np.float64), E4M3)
            d = (E4M3[sb].astype(np.float32) * t)[..., None]
            q = np.where(d == 0, np.float32(0), a / np.where(d == 0, np.float32(1), d))
            v = np.where(d == 0, np.float32(0), v)      # a scale of 0: codes 0, without signs
            sb = np.where(bad, 0x7F, sb)
        else:
            e = np.maximum(np.frexp(amax)[1] - 3, -127)
            e = np.where(amax == 0, -127, e)
            q = a.astype(np.float64) * 2.0 ** (-e[..., None].astype(np.float64))
            sb = np.where(bad, 255, e + 127)
    code = nearest(q.astype(np.float64), E2M1) + 8 * np.signbit(v)
    return code.reshape(rows, nb * B).astype(np.uint8), sb.astype(np.uint8)


def values(code, sb, fmt, cols, ts=None):
    """fp64 numbers that codes and scale bytes stand for."""
    B = BLOCK[fmt]
    v = np.where(code > 7, -1.0, 1.0) * E2M1[code & 7]
    if fmt == "nvfp4":
        s = np.append(E4M3, np.nan)[np.minimum(sb, 127)]
    else:
        s = np.where(sb == 255, np.nan, 2.0 ** (sb.astype(np.float64) - 127))
    v = (v.reshape(len(code), -1, B) * s[..., None]).reshape(len(code), -1)[:, :cols]
    return v if ts is None else v * float(np.float32(ts))


def store(code, sb, fmt, fill=0):
    """The two buffers' bytes; padded rows hold `fill` (they are not data)."""
    B = BLOCK[fmt]
    rows, cols = code.shape
    R, K = -(-rows // 128) * 128, -(-cols // 128) * 128
    codes = np.full((R // 128, K // 32, 128, 16), fill, np.uint8)
    nib = np.zeros((rows, K), np.uint8)
    nib[:, :cols] = code
    byte = nib[:, 0::2] | nib[:, 1::2] << 4
    for r in range(rows):
        codes[r // 128, :, r % 128] = byte[r].reshape(-1, 16)
    scales = np.full((R // 128, K // B // 4, 32, 4, 4), fill, np.uint8)
    pad = np.zeros((rows, K // B), np.uint8)
    pad[:, :sb.shape[1]] = sb
    for r in range(rows):
        scales[r // 128, :, r % 32, r % 128 // 32] = pad[r].reshape(-1, 4)
    return codes, scales
