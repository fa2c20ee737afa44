"""fp64 oracle of causal attention with a sliding window and visible first tokens:
query q sees key k when k <= q < L and (q - k < window or k < sinks).  Query head
h reads key/value head h // (heads // kv_heads)."""

import numpy as np


def visible(n, length, window, sinks):
    q, k = np.arange(n)[:, None], np.arange(n)[None]
    return (k <= q) & (q < length) & ((q - k < window) | (k < sinks))


def _weights(q, k, mask):
    """(P, lse) of one head; rows without a visible key get 0 and -inf."""
    s = np.where(mask, q @ k.T / np.sqrt(q.shape[-1]), -np.inf)
    top = s.max(-1, keepdims=True)
    seen = np.isfinite(top)
    e = np.exp(s - np.where(seen, top, 0.0))
    total = e.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = np.where(seen, top + np.log(total), -np.inf)
    return e / np.where(seen, total, 1.0), lse[:, 0]


def fwd(q, k, v, window, sinks, lengths=None):
    batch, heads, n, _ = q.shape
    group = heads // k.shape[1]
    o, lse = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
    for b in range(batch):
        mask = visible(n, n if lengths is None else lengths[b], window, sinks)
        for h in range(heads):
            p, lse[b, h] = _weights(q[b, h], k[b, h // group], mask)
            o[b, h] = p @ v[b, h // group]
    return o, lse


def bwd(q, k, v, do, window, sinks, lengths=None, rounding=0.0):
    """(dQ, dK, dV) and, for each, a bound on what a relative `rounding` of P, dS,
    O and the result changes: sums of absolute values of the terms rounded."""
    batch, heads, n, d = q.shape
    group = heads // k.shape[1]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    bq, bk, bv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for b in range(batch):
        length = n if lengths is None else lengths[b]
        mask = visible(n, length, window, sinks)
        for h in range(heads):
            kk, vv = k[b, h // group], v[b, h // group]
            g = np.where(np.arange(n)[:, None] < length, do[b, h], 0.0)
            p, _ = _weights(q[b, h], kk, mask)
            o = p @ vv
            row = (g * o).sum(-1, keepdims=True)
            ds = p * (g @ vv.T - row) / np.sqrt(d)
            dq[b, h] = ds @ kk
            dk[b, h // group] += ds.T @ q[b, h]
            dv[b, h // group] += p.T @ g
            # O is off by the rounding of P's terms and its own; so is the row term
            row_off = (np.abs(g) * (p @ np.abs(vv) + np.abs(o))).sum(-1, keepdims=True)
            ds_off = rounding * (np.abs(ds) + p * row_off / np.sqrt(d))
            bq[b, h] = ds_off @ np.abs(kk)
            bk[b, h // group] += ds_off.T @ np.abs(q[b, h])
            bv[b, h // group] += rounding * (p.T @ np.abs(g))
    return (dq, dk, dv), tuple(x + rounding * np.abs(y)
                               for x, y in ((bq, dq), (bk, dk), (bv, dv)))
