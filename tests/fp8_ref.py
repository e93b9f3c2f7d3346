"""Reference for the 8-bit block-scaled operators, in 64 bits on the CPU.

Values of an 8-bit type come from decoding all 256 bytes; rounding picks the
nearest of them, ties to the byte with an even last bit.  Scales follow from
comparing a block's largest finite magnitude with multiples of the type's
largest value.
"""
import numpy as np

BLOCK = 128


def decode_table(fmt):
    """The values of bytes 0 .. 127 in increasing order, finite ones only."""
    eb, mb, bias = (4, 3, 7) if fmt == "e4m3" else (5, 2, 15)
    out = []
    for v in range(128):
        e, m = v >> mb, v & ((1 << mb) - 1)
        if fmt == "e5m2" and e == 31 or fmt == "e4m3" and v == 127:
            break
        out.append((1 + m / (1 << mb)) * 2.0 ** (e - bias) if e else m / (1 << mb) * 2.0 ** (1 - bias))
    return np.array(out)


TABLE = {f: decode_table(f) for f in ("e4m3", "e5m2")}


def round8(y, fmt):
    """Nearest values of the type to y (float64), ties to even."""
    t = TABLE[fmt]
    a = np.abs(np.where(np.isfinite(y), y, 0.0))
    hi = np.clip(np.searchsorted(t, a), 1, len(t) - 1)
    lo = hi - 1
    dl, dh = a - t[lo], t[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    v = np.where(up, t[hi], t[lo])
    v = np.copysign(v, y)
    if fmt == "e5m2":
        v = np.where(np.isinf(y), y, v)
    else:
        v = np.where(np.isinf(y), np.nan, v)
    return np.where(np.isnan(y), np.nan, v)


def quantize(x, fmt="e4m3", block="row"):
    """(values of Q, exponents of S as (blocks, rows)) of a float64 matrix."""
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    top = TABLE[fmt][-1]
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    amax = np.zeros((rows, nb))
    for b in range(nb):
        amax[:, b] = a[:, b * BLOCK:(b + 1) * BLOCK].max(axis=1)
    if block == "square":
        for r in range(0, rows, BLOCK):
            amax[r:r + BLOCK] = amax[r:r + BLOCK].max(axis=0)
    e = np.zeros(amax.shape, dtype=np.int64)
    for i, v in np.ndenumerate(amax):
        if v > 0:
            k = -127
            if v > top * 2.0 ** -127:
                k = int(np.frexp(v / top)[1]) - 2
                while top * 2.0 ** k < v:
                    k += 1
            e[i] = k
    wide = np.repeat(e, BLOCK, axis=1)[:, :cols]
    return round8(np.ldexp(x, -wide), fmt), e.T


def values(q, e):
    """What (Q, S) stands for: q (rows, cols), e exponents (blocks, rows)."""
    return np.ldexp(q, np.repeat(e.T, BLOCK, axis=1)[:, :q.shape[1]])


def product(a, b):
    """(a b^T, |a| |b|^T) in 64 bits."""
    return a @ b.T, np.abs(a) @ np.abs(b).T


def gemm_bound(ref, mag, k):
    """How far a bfloat16 result may be: half a step of bfloat16 (2^-8 of the
    value, plus what the sum was off by), and what the sum may be off by.  The
    matrix instruction aligns the products of a group of eight to the largest
    of them and keeps 13 bits below it (tests of the GPU pin that), so a group
    loses at most 7 2^-13 of its largest product, below 2^-10 of its sum of
    magnitudes; adding the groups, and the K / 64 instructions, in float
    loses at most (K / 8 + 16) 2^-24."""
    off = (2.0 ** -10 + (k / 8 + 16) * 2.0 ** -24) * mag
    return 2.0 ** -8 * (np.abs(ref) + off) + off
