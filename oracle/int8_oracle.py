"""8-bit integers under fp32 scales in float64: rows, blocks of a checkpoint, grouped products and the expert FFN."""
import numpy as np

TINY = 2.0**-96


def quantize(x):
    """(codes int64, scales float64 of fp32 numbers) of the rows of x [..., K] (values of a 32-bit type or narrower): x * 127 and amax
    are exact in float64, and their quotient comes no nearer to a border than 2^-33 of it, so its rounding crosses none."""
    x = np.asarray(x, np.float64)
    bad = ~np.isfinite(x).all(axis=-1)
    amax = np.abs(np.where(np.isfinite(x), x, 0.0)).max(axis=-1)
    live = (amax >= TINY) & ~bad
    codes = np.rint(np.where(live[..., None], x, 0.0) * 127.0 / np.where(live, amax, 1.0)[..., None]).astype(np.int64)
    scales = np.where(live, (amax.astype(np.float32) / np.float32(127.0)).astype(np.float64), np.where(bad, np.nan, 0.0))
    return codes, scales


def linear(codes, scales, offsets, w, w_scales):
    """[rows, N] of codes [rows, K], w [G, N, K], w_scales [G, N] (NaN where a row belongs to no group)."""
    out = np.full((codes.shape[0], w.shape[1]), np.nan)
    for g in range(w.shape[0]):
        lo, hi = offsets[g], offsets[g + 1]
        acc = codes[lo:hi].astype(np.float64) @ w[g].astype(np.float64).T      # whole numbers below 2^53: exact
        out[lo:hi] = acc * scales[lo:hi, None] * w_scales[g][None]
    return out


def act(x, offsets, gate, gate_scales, up, up_scales):
    c, s = quantize(x)
    g, u = linear(c, s, offsets, gate, gate_scales), linear(c, s, offsets, up, up_scales)
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u
