"""fp64 oracle of the 4-bit key/value cache and of attention over it.

Per group of 32 channels: m = the largest bf16 <= (min + max) / 2, s = the
smallest bf16 >= max(max - m, m - min) / 7.5, code = floor((x - m) / s) + 8,
value m + s (code - 7.5); s = 0 when every value equals m.  A group that holds a
non-finite value stands for NaN.
"""

import numpy as np

GROUP = 32


def bf16_floor(x):
    """Largest bf16 not above each finite fp64 value (subnormal bf16 are multiples of 2^-133)."""
    x = np.asarray(x, np.float64)
    unit = np.ldexp(1.0, np.maximum(np.frexp(x)[1] - 8, -133))
    return np.floor(x / unit) * unit


def floor_ratio(x, mid, step):
    """floor((x - mid) / step), 0 where step is 0, exact where the fp64 difference
    is not (x a subnormal fp32 beside mid, say): the difference is carried as a sum
    of two fp64 numbers, and k step (a few bits) is compared with it."""
    d = x - mid
    back = d - x
    rest = (x - (d - back)) + (-mid - back)  # x - mid = d + rest exactly
    safe = np.where(step > 0, step, 1.0)
    k = np.floor(d / safe)
    for _ in range(2):
        k -= (k * safe > d) | ((k * safe == d) & (rest < 0))
        up = (k + 1) * safe
        k += (up < d) | ((up == d) & (rest >= 0))
    return np.where(step > 0, k, 0.0)


def quantise(x):
    """(codes, steps, midpoints) of x [..., d]; groups on the second to last axis."""
    g = np.asarray(x, np.float64).reshape(*np.shape(x)[:-1], -1, GROUP)
    lo, hi = g.min(-1, keepdims=True), g.max(-1, keepdims=True)
    bad = ~np.isfinite(g).all(-1, keepdims=True)
    lo, hi = np.where(bad, 0.0, lo), np.where(bad, 0.0, hi)
    mid = bf16_floor((lo + hi) / 2)
    step = -bf16_floor(-np.maximum(hi - mid, mid - lo) / 7.5)
    code = np.where(bad, 8, floor_ratio(np.where(bad, 0.0, g), mid, step) + 8)
    return code, np.where(bad, np.nan, step), np.where(bad, np.nan, mid)


def values(x):
    """What the cache stands for after x [..., d] has been written."""
    code, step, mid = quantise(x)
    return (mid + step * (code - 7.5)).reshape(np.shape(x))


def decode(q, k, v, lengths, window, sinks):
    """Attention of the last token: q [batch, heads, d] over the fp64 keys and
    values [batch, kv_heads, n, d] that the cache stands for; returns (o, lse)."""
    batch, heads, d = q.shape
    group = heads // k.shape[1]
    o, lse = np.zeros(q.shape), np.full((batch, heads), -np.inf)
    for b in range(batch):
        n = int(min(max(lengths[b], 0), k.shape[2]))
        at = np.arange(n)
        at = at[(at >= n - window) | (at < sinks)]
        if not at.size:
            continue
        for h in range(heads):
            s = k[b, h // group, at] @ q[b, h] / np.sqrt(d)
            top = s.max()
            p = np.exp(s - top)
            o[b, h] = p @ v[b, h // group, at] / p.sum()
            lse[b, h] = top + np.log(p.sum())
    return o, lse
