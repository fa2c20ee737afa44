"""GPU checks that a NaN or an infinity reaches the rows that see it and no other, in
the attention with a sliding window and sinks.  What a row is without it comes from the
fp64 oracle on the same inputs with zeros in their place, in the tolerances of
test_gpu_sink."""

import numpy as np
import pytest
import torch

from oracle import sink
from tests.gpu_util import f64
from tests.test_gpu_sink import HALF_STEP, i32, inputs, run_fwd

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
CASES = [  # heads, kv_heads, n, lengths, window, sinks, bad tokens
    (2, 1, 700, None, 64, 4, [10]),             # beside the sinks, long before the windows
    (2, 2, 700, [700, 512], 64, 70, [71, 127]),   # two blocks of sinks
    (4, 2, 500, None, 160, 4, [200]),           # inside a tile, and at a window's edge
    (2, 2, 500, [500, 290], 2147483647, 0, [130, 255, 289]),  # plain causal
    (3, 1, 300, None, 1, 0, [0, 128, 299]),     # every row sees itself alone
    (2, 1, 640, [513, 640], 33, 0, [479, 480, 512]),
    (2, 1, 420, None, 5, 128, [127, 128, 300]),  # the last sink, and the token behind it
    (1, 1, 200, None, 100, 30, [29, 30, 99, 100])]  # the sinks' block is the window's too


def sees(n, length, window, sinks, tokens):
    """Rows of a sequence that see one of the tokens."""
    return sink.visible(n, length, window, sinks)[:, tokens].any(1)


def spoil(x, tokens, seed):
    """Some channels of the tokens' rows of each head become NaN, inf or -inf."""
    g = np.random.default_rng(seed)
    bad = np.zeros(x.shape, bool)
    y = x.clone()
    for t in tokens:
        for b in range(x.shape[0]):
            for h in range(x.shape[1]):
                for c in g.choice(x.shape[3], 3, replace=False):
                    bad[b, h, t, c] = True
                    y[b, h, t, c] = (NAN, INF, -INF)[g.integers(3)]
    return y, bad


def close(got, want, top):
    return np.abs(got - want) <= HALF_STEP * (np.abs(want) + top) + 1e-4 * top


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv_heads,n,lengths,window,sinks,tokens", CASES)
def test_values(heads, kv_heads, n, lengths, window, sinks, tokens, d):
    batch = 1 if lengths is None else len(lengths)
    q, k, v, _ = inputs(batch, heads, kv_heads, n, d, n + d)
    dirty, bad = spoil(v, tokens, n)
    clean = torch.where(torch.from_numpy(bad), torch.zeros_like(v), v)
    o, lse = run_fwd(q.cuda(), k.cuda(), dirty.cuda(), i32(lengths), window, sinks)
    want, want_lse = sink.fwd(f64(q), f64(k), f64(clean), window, sinks, lengths)
    got = f64(o)
    top = np.abs(f64(clean)).max()
    lens = lengths or [n] * batch
    for b, L in enumerate(lens):
        mask = sink.visible(n, L, window, sinks)
        for h in range(heads):
            hit = mask.astype(float) @ bad[b, h // (heads // kv_heads)] > 0  # [row, channel]
            assert not np.isfinite(got[b, h][hit]).any()
            assert close(got[b, h][~hit], want[b, h][~hit], top).all()
    seen = np.isfinite(want_lse)
    assert np.abs(f64(lse)[seen] - want_lse[seen]).max() <= 1e-4
    again, _ = run_fwd(q.cuda(), k.cuda(), dirty.cuda(), i32(lengths), window, sinks)
    assert torch.equal(o.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("d", [64, 128])
def test_a_token_beside_the_sinks_changes_no_later_bit(d):
    """Past its window, and past the tiles that hold it, a bad token leaves every bit."""
    n, window, sinks, t = 1500, 64, 4, 10
    q, k, v, _ = (x.cuda() for x in inputs(2, 4, 2, n, d, 3))
    want, want_lse = run_fwd(q, k, v, None, window, sinks)
    v[0, 1, t] = NAN
    k[0, 1, t] = INF
    o, lse = run_fwd(q, k, v, None, window, sinks)
    assert torch.equal(o[1], want[1]) and torch.equal(o[0, :2], want[0, :2])
    assert torch.equal(o[0, :, 256:], want[0, :, 256:])
    seen = torch.zeros(n, dtype=torch.bool, device="cuda")
    seen[t:t + window] = True
    assert torch.equal(lse[0, :, ~seen], want_lse[0, :, ~seen])
    assert o[0, 2:, seen].isnan().all() and not o[0, :, ~seen].isnan().any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", ["all", "channel", "infinite channel"])
def test_values_that_are_no_numbers_at_all(what, d):
    """Every row sees one of them (itself), so every row keeps them."""
    n = 900
    q, k, v, _ = inputs(1, 2, 2, n, d, 5)
    clean = v.clone()
    at = slice(None) if what == "all" else 7
    v[..., at] = INF if what == "infinite channel" else NAN
    clean[..., at] = 0
    o, _ = run_fwd(q.cuda(), k.cuda(), v.cuda(), None, 200, 4)
    want, _ = sink.fwd(f64(q), f64(k), f64(clean), 200, 4)
    assert not torch.isfinite(o[..., at]).any()
    if what != "all":
        rest = [c for c in range(d) if c != 7]
        assert close(f64(o)[..., rest], want[..., rest], np.abs(f64(clean)).max()).all()


def test_more_sequences_than_the_work_table_holds():
    batch, n = 1030, 40
    q, k, v, _ = inputs(batch, 2, 1, n, 64, 9)
    lengths = [b % (n + 1) for b in range(batch)]
    v[:, :, 20] = NAN
    o, _ = run_fwd(q.cuda(), k.cuda(), v.cuda(), i32(lengths), 6, 1)
    hit = np.zeros((batch, 2, n), bool)
    for b, L in enumerate(lengths):
        hit[b] = sees(n, L, 6, 1, [20])
    assert np.array_equal(o.isnan().any(-1).cpu().numpy(), hit)


def test_replayed_in_a_graph():
    """One captured call, on clean values, on spoiled ones, and on clean ones again."""
    n, d, window, sinks = 600, 64, 90, 2
    q, k, v, _ = (x.cuda() for x in inputs(1, 4, 2, n, d, 8))
    spoiled, _ = spoil(v.cpu(), [17, 300], 1)
    o, lse = torch.empty_like(q), torch.empty(1, 4, n, device="cuda")
    import block_sparse_local_nb_b200 as nb

    def step(x):
        nb.nb_attn_sink_fwd(q, k, x, o, lse, None, 1, 4, 2, n, d, window, sinks, nb.NB_BF16)
        return o.clone()

    wants = [step(x).view(torch.int16) for x in (v, spoiled.cuda(), v)]
    assert torch.equal(wants[0], wants[2]) and not torch.equal(wants[0], wants[1])
    held = v.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        nb.nb_attn_sink_fwd(q, k, held, o, lse, None, 1, 4, 2, n, d, window, sinks, nb.NB_BF16)
    for x, want in zip((v, spoiled.cuda(), v), wants):
        held.copy_(x)
        graph.replay()
        assert torch.equal(o.view(torch.int16), want)
