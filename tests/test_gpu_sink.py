"""GPU parity of the attention with a sliding window and sinks (nb_attn_sink_fwd,
nb_attn_sink_bwd) against the fp64 oracle.

Tolerances.  A rounding to bf16 is off by at most 2^-8 of the value.  O: each P
term is rounded once and the result once: 2^-8 (sum_j p_j |v_j| + |o|), bounded by
2^-8 (max |v| + |o|).  Gradients: P, dS and the results are rounded, and the row
term takes the rounded O; the oracle adds up the absolute values of those terms.
fp32 arithmetic (sums of at most a few thousand terms, ex2.approx) stays below
1e-4 of the same sums and of the largest value; 1e-4 absolute on the log-sum-exp,
whose inputs are exact products added in fp32.
"""

import numpy as np
import pytest
import torch

import block_sparse_local_nb_b200 as nb
from oracle import sink
from tests.gpu_util import f64

pytestmark = pytest.mark.gpu

HALF_STEP = 2.0 ** -8


def inputs(batch, heads, kv_heads, n, d, seed):
    g = torch.Generator().manual_seed(seed)

    def t(h):
        return torch.randn((batch, h, n, d), generator=g).bfloat16()

    return t(heads), t(kv_heads), t(kv_heads), t(heads)


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")


def run_fwd(q, k, v, lengths, window, sinks, with_lse=True):
    batch, heads, n, d = q.shape
    o = torch.full_like(q, 9.0)
    lse = torch.full((batch, heads, n), 9.0, device="cuda") if with_lse else None
    nb.nb_attn_sink_fwd(q, k, v, o, lse, lengths, batch, heads, k.shape[1], n, d, window, sinks,
                        nb.NB_BF16)
    return o, lse


def run_bwd(q, k, v, o, do, lse, lengths, window, sinks):
    batch, heads, n, d = q.shape
    shape = (batch, heads, k.shape[1], n, d, window, sinks, nb.NB_BF16)
    size = nb.attn_sink_bwd_workspace_size(*shape)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    dq, dk, dv = (torch.full_like(x, 9.0) for x in (q, k, v))
    nb.nb_attn_sink_bwd(q, k, v, o, do, lse, lengths, dq, dk, dv, ws, size, *shape)
    return dq, dk, dv


def check(q, k, v, do, lengths, window, sinks, backward=True, device_inputs=None):
    n = q.shape[2]
    qd, kd, vd, dod = device_inputs or (x.cuda() for x in (q, k, v, do))
    o, lse = run_fwd(qd, kd, vd, i32(lengths), window, sinks)
    args = [f64(x) for x in (q, k, v)]
    want, want_lse = sink.fwd(*args, window, sinks, lengths)
    got = f64(o)
    top = np.abs(args[2]).max()
    assert (np.abs(got - want) <= HALF_STEP * (np.abs(want) + top) + 1e-4 * top).all()
    got_lse, pad = f64(lse), np.isinf(want_lse)
    assert np.array_equal(np.isneginf(got_lse), pad)
    assert np.abs(got_lse[~pad] - want_lse[~pad]).max(initial=0) <= 1e-4
    lens = [n] * q.shape[0] if lengths is None else lengths
    for b, L in enumerate(lens):
        assert (got[b, :, L:] == 0).all()
    if not backward:
        return
    grads = run_bwd(qd, kd, vd, o, dod, lse, i32(lengths), window, sinks)
    wants, bounds = sink.bwd(*args, f64(do), window, sinks, lengths, HALF_STEP)
    for name, g, w, tol in zip(("dq", "dk", "dv"), grads, wants, bounds):
        off = np.abs(f64(g) - w)
        limit = tol * (1 + 1e-4 / HALF_STEP) + 1e-4 * np.abs(w).max()
        assert (off <= limit).all(), (name, float((off / limit).max()))
        for b, L in enumerate(lens):
            assert (g[b, :, L:] == 0).all(), name


CASES = [  # heads, kv_heads, n, lengths, window, sinks
    (1, 1, 1, [1], 1, 0), (2, 2, 61, [61], 32, 4), (2, 1, 64, [64, 1], 64, 0),
    (4, 2, 129, [129, 0], 5, 1), (3, 3, 128, [127, 128], 1, 0), (3, 1, 333, [333, 97], 100, 1),
    (2, 2, 500, [500, 385], 64, 128), (4, 1, 700, [700, 641], 200, 33),
    (2, 1, 640, None, 2147483647, 7), (1, 1, 1000, [999, 513], 129, 65), (2, 2, 900, [900, 130], 1, 4)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv_heads,n,lengths,window,sinks", CASES)
def test_fwd(heads, kv_heads, n, lengths, window, sinks, d):
    batch = 1 if lengths is None else len(lengths)
    check(*inputs(batch, heads, kv_heads, n, d, n + d), lengths, window, sinks, backward=False)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv_heads,n,lengths,window,sinks", CASES)
def test_fwd_bwd(heads, kv_heads, n, lengths, window, sinks, d):
    batch = 1 if lengths is None else len(lengths)
    check(*inputs(batch, heads, kv_heads, n, d, n + d), lengths, window, sinks)
