"""Block-scaled 4-bit floating point in float64 numpy: the formats' definitions, written without the library's code.

A block's scale and codes come from nearest-value searches over the two formats' value tables (exact ties to the even
code); products are float64 matrix products of the decoded values. Every function also bounds what an fp32
implementation may differ by, so that the tests' tolerances follow from the formulas.
"""
from __future__ import annotations

import numpy as np

BLOCK = {"nv": 16, "mx": 32}
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(b & 7) / 8 * 2.0**-6 if b < 8 else (1 + (b & 7) / 8) * 2.0 ** ((b >> 3) - 7) for b in range(127)])


def nearest(v, table):
    """Index of the nearest entry of the rising `table` to each v >= 0, ties to the even index, the last entry above."""
    hi = np.clip(np.searchsorted(table, v), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = v - table[lo], table[hi] - v
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def quantize(x, fmt):
    """x [rows, K] float64 -> (code magnitudes' index [rows, K] with bit 3 the sign, scale bytes [rows, blocks])."""
    x = np.asarray(x, np.float64)
    rows, K = x.shape
    b = BLOCK[fmt]
    nb = -(-K // b)
    v = np.zeros((rows, nb * b))
    v[:, :K] = x
    v = v.reshape(rows, nb, b)
    bad = np.isnan(v).any(-1)
    w = np.where(np.isnan(v), 0.0, v)
    amax = np.abs(w).max(-1)
    if fmt == "nv":
        byte = nearest(np.minimum(amax / 6, 448.0), E4M3)
        s = E4M3[byte]
    else:
        _, e = np.frexp(np.where(np.isfinite(amax), amax, 2.0**128))
        byte = np.where(amax > 0, np.clip(e - 1 - 2 + 127, 0, 254), 0)
        s = 2.0 ** (byte - 127.0)
    with np.errstate(invalid="ignore", over="ignore"):
        q = np.abs(w) / np.where(s > 0, s, 1.0)[..., None]
    code = nearest(np.minimum(np.where(s[..., None] > 0, q, 0.0), 6.0), E2M1)
    code = code | (np.signbit(w) & (code > 0)).astype(np.int64) << 3
    code[bad] = 0
    byte = np.where(bad, 127 if fmt == "nv" else 255, byte)
    return code.reshape(rows, nb * b)[:, :K], byte.astype(np.int64)


def scale_of(byte, fmt):
    byte = np.asarray(byte, np.int64)
    if fmt == "nv":
        return np.where(byte == 127, np.nan, E4M3[np.minimum(byte, 126)])
    return np.where(byte == 255, np.nan, 2.0 ** (byte - 127.0))


def dequantize(code, byte, fmt):
    v = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    return v * np.repeat(scale_of(byte, fmt), BLOCK[fmt], 1)[:, : code.shape[1]]


def unpack_codes(packed, K):
    """Bytes [rows, pitch] -> codes [rows, K], -0 as 0."""
    p = np.asarray(packed, np.int64)
    c = np.stack([p & 15, p >> 4], -1).reshape(p.shape[0], -1)
    assert (c[:, K:] == 0).all(), "codes past K are 0"
    return np.where(c == 8, 0, c)[:, :K]


#: One tcgen05.mma adds 64 products to an fp32 accumulator. Each such step is allowed four units in the last place of
#: the magnitudes summed (alignment and rounding of the partial sums): 2^-22 relative to sum |a b|.
STEP = 2.0**-22


def product_bound(a, w, y, half_step):
    """Elementwise bound of |fp32 result - y| for y = a @ w.T, rounded once to a type of `half_step` (= eps / 2)."""
    steps = -(-a.shape[1] // 64)
    return (steps + 4) * STEP * (np.abs(a) @ np.abs(w).T) + half_step * np.abs(y) + 1e-30


def swiglu_bound(g, eg, u, eu):
    """act = silu(g) u and a bound of its fp32 error, given the bounds of g and u (|silu'| < 1.1; the exponential and the
    quotient within 2^-18)."""
    sg = g / (1 + np.exp(-g))
    act = sg * u
    return act, 1.1 * eg * (np.abs(u) + eu) + np.abs(sg) * eu + 2.0**-18 * np.abs(act) + 1e-30


def requantized(act, err, fmt):
    """(Q(act), bound of the difference an error of `err` in act can make): zero unless a value comes within its error
    of a tie, then the whole step; where a block's scale can turn, every value of the block by what the next scale
    changes."""
    rows, K = act.shape
    b = BLOCK[fmt]
    code, byte = quantize(act, fmt)
    q = dequantize(code, byte, fmt)
    pad = -K % b
    a = np.pad(np.abs(act), ((0, 0), (0, pad))).reshape(rows, -1, b)
    e = np.pad(err, ((0, 0), (0, pad))).reshape(rows, -1, b)
    s = scale_of(byte, fmt)
    lo, hi = quantize((a - e).clip(0).reshape(rows, -1), fmt), quantize((a + e).reshape(rows, -1), fmt)
    with np.errstate(invalid="ignore"):
        turn = ((lo[1] != hi[1]))[..., None] & np.ones_like(a, bool)
        step = np.where(a < 2 * s[..., None], 0.5, np.where(a < 4 * s[..., None], 1.0, 2.0)) * s[..., None]
        mid = (E2M1[1:] + E2M1[:-1]) / 2
        near = (np.abs(a[..., None] - mid * s[..., None, None]) <= e[..., None]).any(-1) & (s[..., None] > 0)
    bound = np.where(turn, 2 * step + 0.5 * a, np.where(near, step, 0.0))
    return q, bound.reshape(rows, -1)[:, :K]
