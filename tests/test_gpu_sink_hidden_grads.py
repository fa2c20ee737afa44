"""GPU checks that a NaN or an infinity in Q, K, V or dO reaches the gradients that
depend on it and no other, in the backward of the attention with a sliding window and
sinks.  The others come from the fp64 oracle on the same inputs with zeros in their
place, in the tolerances of test_gpu_sink."""

import numpy as np
import pytest
import torch

from oracle import sink
from tests.gpu_util import f64
from tests.test_gpu_sink import HALF_STEP, i32, inputs, run_bwd, run_fwd

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
CASES = [  # heads, kv_heads, n, lengths, window, sinks, bad tokens
    (2, 1, 700, None, 64, 4, [10]),                 # beside the sinks, long before the windows
    (2, 2, 700, [700, 512], 64, 70, [127, 400]),
    (4, 2, 500, None, 160, 4, [200]),               # inside a tile, and at a window's edge
    (2, 2, 500, [500, 290], 2147483647, 0, [289]),  # plain causal
    (3, 1, 300, None, 1, 0, [0, 128, 299]),         # every row sees itself alone
    (2, 1, 640, [513, 640], 33, 0, [480]),
    (2, 1, 420, None, 5, 128, [128, 300]),          # the token behind the last sink
    (1, 1, 200, None, 100, 30, [30, 150]),          # the sinks' block is the window's too
    (8, 1, 1500, [1437], 1000, 3, [300, 1436])]     # key tiles in parts


def spoil(x, tokens, seed, values):
    """Two channels of the tokens' rows in the first head of each sequence."""
    g = np.random.default_rng(seed)
    bad = np.zeros(x.shape, bool)
    y = x.clone()
    for t in tokens:
        for b in range(x.shape[0]):
            for c in g.choice(x.shape[3], 2, replace=False):
                bad[b, 0, t, c] = True
                y[b, 0, t, c] = values[g.integers(len(values))]
    return y, bad


def reached(what, bad, heads, kv_heads, n, lengths, window, sinks):
    """Which elements of dQ, dK, dV depend on the bad elements of `what`."""
    batch, d = bad.shape[0], bad.shape[3]
    group = heads // kv_heads
    dq = np.zeros((batch, heads, n, d), bool)
    dk, dv = np.zeros((batch, kv_heads, n, d), bool), np.zeros((batch, kv_heads, n, d), bool)
    for b in range(batch):
        mask = sink.visible(n, n if lengths is None else lengths[b], window, sinks)
        mask &= np.arange(n)[None] < (n if lengths is None else lengths[b])
        for h in range(heads):
            kv = h // group
            if what in "kv":
                rows = (mask & bad[b, kv].any(1)[None]).any(1)  # queries that see a bad token
            else:
                rows = mask.any(1) & bad[b, h].any(1)
            keys = mask[rows].any(0)
            dq[b, h, rows] = True
            dk[b, kv, keys] = True
            if what in "qk":
                dv[b, kv, keys] = True
            elif what == "do":
                dv[b, kv] |= mask.T.astype(float) @ (bad[b, h] & rows[:, None]) > 0
    return dq, dk, dv


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", ["q", "k", "v", "do"])
@pytest.mark.parametrize("heads,kv_heads,n,lengths,window,sinks,tokens", CASES)
def test_gradients(heads, kv_heads, n, lengths, window, sinks, tokens, what, d):
    batch = 1 if lengths is None else len(lengths)
    clean = dict(zip(("q", "k", "v", "do"), inputs(batch, heads, kv_heads, n, d, n + d)))
    # (an infinite score may be a weight of 0, so Q and K take NaN alone)
    dirty = dict(clean)
    dirty[what], bad = spoil(clean[what], tokens, n, (NAN,) if what in "qk" else (NAN, INF, -INF))
    clean[what] = torch.where(torch.from_numpy(bad), torch.zeros_like(clean[what]), clean[what])
    q, k, v, do = (dirty[x].cuda() for x in ("q", "k", "v", "do"))
    o, lse = run_fwd(q, k, v, i32(lengths), window, sinks)
    grads = run_bwd(q, k, v, o, do, lse, i32(lengths), window, sinks)
    wants, bounds = sink.bwd(*(f64(clean[x]) for x in ("q", "k", "v", "do")), window, sinks,
                             lengths, HALF_STEP)
    hits = reached(what, bad, heads, kv_heads, n, lengths, window, sinks)
    for name, g, w, tol, hit in zip(("dq", "dk", "dv"), grads, wants, bounds, hits):
        g = f64(g)
        assert not np.isfinite(g[hit]).any(), name
        limit = tol * (1 + 1e-4 / HALF_STEP) + 1e-4 * np.abs(w).max()
        assert (np.abs(g - w) <= limit)[~hit].all(), name
        assert hit.any() or (what, name) == ("v", "dv")
    again = run_bwd(q, k, v, o, do, lse, i32(lengths), window, sinks)
    for x, y in zip(grads, again):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))


@pytest.mark.parametrize("d", [64, 128])
def test_other_heads_and_sequences_keep_their_bits(d):
    q, k, v, do = (x.cuda() for x in inputs(2, 4, 2, 700, d, 4))

    def both():
        o, lse = run_fwd(q, k, v, None, 90, 3)
        return run_bwd(q, k, v, o, do, lse, None, 90, 3)

    want = both()
    k[0, 1, 300], do[0, 3, 17] = NAN, INF
    got = both()
    for x, y in zip(got, want):
        half = x.shape[1] // 2
        assert torch.equal(x[1], y[1]) and torch.equal(x[0, :half], y[0, :half])
        assert not torch.isfinite(x[0, half:]).all()


def test_more_sequences_than_the_work_table_holds():
    batch, n = 1030, 40
    q, k, v, do = inputs(batch, 2, 1, n, 64, 9)
    lengths = [b % (n + 1) for b in range(batch)]
    do[:, 1, 20, 3] = NAN
    q, k, v, do = (x.cuda() for x in (q, k, v, do))
    o, lse = run_fwd(q, k, v, i32(lengths), 6, 1)
    dq, dk, dv = run_bwd(q, k, v, o, do, lse, i32(lengths), 6, 1)
    bad = np.zeros((batch, 2, n, 64), bool)
    bad[:, 1, 20, 3] = True
    for x, hit in zip((dq, dk, dv), reached("do", bad, 2, 1, n, lengths, 6, 1)):
        assert np.array_equal(~torch.isfinite(x).cpu().numpy(), hit)


@pytest.mark.parametrize("what", ["q", "k", "v", "do"])
def test_nothing_but_nan(what):
    """Every gradient that depends on it is none; the backward ends all the same."""
    x = dict(zip(("q", "k", "v", "do"), (t.cuda() for t in inputs(1, 4, 2, 1000, 64, 2))))
    x[what] = torch.full_like(x[what], NAN)
    o, lse = run_fwd(x["q"], x["k"], x["v"], None, 200, 4)
    grads = run_bwd(x["q"], x["k"], x["v"], o, x["do"], lse, None, 200, 4)
    for name, g in zip(("dq", "dk", "dv"), grads):
        if (what, name) == ("v", "dv"):
            assert torch.isfinite(g).all()
        else:
            assert g.isnan().all()
