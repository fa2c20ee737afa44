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


@pytest.mark.parametrize("d", [64, 128])
def test_what_lies_past_the_length_does_not_matter(d):
    """NaN and infinities in Q, K, V, O and dO past the length change no bit."""
    q, k, v, do = inputs(2, 4, 2, 300, d, 5)
    lengths, window, sinks = [213, 64], 90, 5
    clean = [x.cuda() for x in (q, k, v, do)]
    dirty = [x.clone() for x in clean]
    for x in dirty:
        x[0, :, 213:] = float("nan")
        x[1, :, 64:] = float("inf")
    out = []
    for qd, kd, vd, dod in (clean, dirty):
        o, lse = run_fwd(qd, kd, vd, i32(lengths), window, sinks)
        if qd is dirty[0]:
            o[0, :, 213:] = float("nan")
            lse[1, :, 64:] = float("nan")
        out.append((o, lse, *run_bwd(qd, kd, vd, o, dod, lse, i32(lengths), window, sinks)))
    for b, L in enumerate(lengths):
        for x, y in zip(*out):
            assert torch.equal(x[b, :, :L], y[b, :, :L])
    for x in out[1][2:]:
        assert torch.isfinite(x.float()).all()


@pytest.mark.parametrize("d,n,window,sinks", [(64, 2000, 300, 4), (128, 1500, 4000, 128)])
def test_results_repeat_bit_for_bit(d, n, window, sinks):
    q, k, v, do = (x.cuda() for x in inputs(2, 6, 2, n, d, 6))
    runs = []
    for _ in range(3):
        o, lse = run_fwd(q, k, v, i32([n, n - 77]), window, sinks)
        runs.append((o, lse, *run_bwd(q, k, v, o, do, lse, i32([n, n - 77]), window, sinks)))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], r))


def test_split_key_tiles():
    """Few key/value heads and a wide window: every key tile is cut into parts."""
    q, k, v, do = inputs(1, 8, 1, 1500, 64, 7)
    check(q, k, v, do, [1437], 1000, 3)


def test_large_scores_and_far_apart_maxima():
    """Scores of a few hundred that grow along the sequence: the running maximum
    rises by more than 2^8 again and again."""
    q, k, v, do = inputs(1, 2, 2, 400, 64, 8)
    ramp = torch.linspace(0.1, 6, 400)[None, None, :, None]
    check((q * ramp).bfloat16(), (k * ramp).bfloat16(), v, do, [400], 350, 2, backward=False)


def test_more_sequences_than_the_work_table_holds():
    batch, n = 1030, 5
    q, k, v, do = inputs(batch, 2, 1, n, 64, 9)
    lengths = [b % (n + 1) for b in range(batch)]
    check(q, k, v, do, lengths, 2, 1)


def test_lse_is_optional_and_lengths_are_clamped():
    q, k, v, _ = (x.cuda() for x in inputs(2, 2, 2, 130, 64, 10))
    o, lse = run_fwd(q, k, v, None, 50, 1)
    o2, none = run_fwd(q, k, v, i32([1000, 130]), 50, 1, with_lse=False)
    assert none is None and torch.equal(o, o2)
    o3, lse3 = run_fwd(q, k, v, i32([-4, 130]), 50, 1)
    assert (o3[0] == 0).all() and torch.isneginf(lse3[0]).all() and torch.equal(o3[1], o[1])


def test_other_stream_and_graph_replay():
    """A forward and backward captured once and replayed on new inputs, and the same
    on a side stream, give the bits of the plain calls."""
    batch, heads, n, d, window, sinks = 2, 4, 500, 64, 120, 4
    shape = (batch, heads, 2, n, d, window, sinks, nb.NB_BF16)
    q, k, v, do = (x.cuda() for x in inputs(batch, heads, 2, n, d, 11))
    lengths = i32([500, 390])
    o, lse = torch.empty_like(q), torch.empty(batch, heads, n, device="cuda")
    dq, dk, dv = (torch.empty_like(x) for x in (q, k, v))
    size = nb.attn_sink_bwd_workspace_size(*shape)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def step():
        nb.nb_attn_sink_fwd(q, k, v, o, lse, lengths, *shape)
        nb.nb_attn_sink_bwd(q, k, v, o, do, lse, lengths, dq, dk, dv, ws, size, *shape)
        return o, lse, dq, dk, dv

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    first = [x.clone() for x in (o, lse, dq, dk, dv)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (11, 12):
        for x, y in zip((q, k, v, do), inputs(batch, heads, 2, n, d, seed)):
            x.copy_(y)
        want = [x.clone() for x in step()]
        for x in (o, lse, dq, dk, dv, ws):
            x.fill_(7)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((o, lse, dq, dk, dv), want):
            assert torch.equal(x, y)
        if seed == 11:
            assert all(torch.equal(x, y) for x, y in zip(want, first))


def test_layer_captured_with_its_gradients():
    """The layer's function and its backward in one graph, replayed on new inputs."""
    from block_sparse_local_nb_b200.layer import sink_attention

    q, k, v, do = (x.cuda() for x in inputs(2, 4, 1, 300, 64, 21))
    lengths = i32([300, 77])
    leaves = [x.requires_grad_(True) for x in (q, k, v)]

    def step():
        o = sink_attention(*leaves, lengths, 90, 2)
        return [o.detach(), *torch.autograd.grad(o, leaves, do)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for x, y in zip((q, k, v, do), inputs(2, 4, 1, 300, 64, 22)):
        with torch.no_grad():
            x.copy_(y)
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in held]
    for x, y in zip(got, step()):
        assert torch.equal(x, y)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,window", [(1, 1), (300, 50), (1000, 400)])
def test_what_is_not_a_number_reaches_the_rows_that_see_it(n, window, d):
    q, k, v, _ = (x.cuda() for x in inputs(1, 2, 2, n, d, 0))
    want, _ = run_fwd(q, k, v, None, window, 0)
    at = n // 2
    q[0, 0, at, 3] = float("nan")
    k[0, 1, at, 5] = float("nan")
    o, lse = run_fwd(q, k, v, None, window, 0)
    seen = torch.zeros(2, n, dtype=torch.bool, device="cuda")
    seen[0, at] = True
    seen[1, at:at + window] = True
    assert torch.equal(o[0].isnan(), seen[..., None].expand(-1, -1, d))
    assert torch.equal(lse[0].isnan(), seen)
    assert torch.equal(o[0][~seen], want[0][~seen])


def test_autograd_on_strided_inputs():
    """The layer's function on [batch, n, heads, d] storage, against the direct calls."""
    from block_sparse_local_nb_b200.layer import sink_attention

    q, k, v, do = inputs(2, 4, 2, 200, 64, 13)
    L = torch.tensor([200, 150])
    leaves = [x.transpose(1, 2).contiguous().cuda().requires_grad_(True) for x in (q, k, v)]
    o = sink_attention(*(x.transpose(1, 2) for x in leaves), L.cuda(), 60, 4)
    o.backward(do.cuda())
    qd, kd, vd, dod = (x.cuda() for x in (q, k, v, do))
    want, lse = run_fwd(qd, kd, vd, i32([200, 150]), 60, 4)
    grads = run_bwd(qd, kd, vd, want, dod, lse, i32([200, 150]), 60, 4)
    assert torch.equal(o, want)
    for leaf, g in zip(leaves, grads):
        assert torch.equal(leaf.grad.transpose(1, 2), g)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv_heads,n,window,sinks", [
    (8, 8, 3, 3, 0), (4, 2, 40, 40, 1), (2, 1, 700, 2, 0), (2, 1, 700, 1, 4), (2, 2, 500, 31, 1),
    (3, 1, 300, 2, 30)])
def test_rows_of_few_keys_lose_nothing_to_the_rounded_output(heads, kv_heads, n, window, sinks, d):
    """dQ and dK are off by two roundings, of dS and of the result.  One is uniform within
    half a step of a value whose mantissa is spread over its logarithm: 2^-8 / sqrt(3)
    times the root mean square of 1 / m, sqrt(3 / (8 ln 2)), is 1.66e-3 of the norm, two
    independent ones 2.35e-3; the allowance for a finite sample is a fifth, 2.8e-3, and
    two fifths for the few hundred elements of the shortest.  (With D from the rounded
    O it is 3.7e-3 at window 2 and 1e-2 at n = 3.)"""
    q, k, v, do = inputs(4, heads, kv_heads, n, d, n + window)
    qd, kd, vd, dod = (x.cuda() for x in (q, k, v, do))
    o, lse = run_fwd(qd, kd, vd, None, window, sinks)
    grads = run_bwd(qd, kd, vd, o, dod, lse, None, window, sinks)
    wants, _ = sink.bwd(*(f64(x) for x in (q, k, v, do)), window, sinks)
    for g, w in zip(grads[:2], wants[:2]):
        assert np.linalg.norm(f64(g) - w) <= (2.8e-3 if n > 3 else 3.3e-3) * np.linalg.norm(w)


def test_gradients_against_differences():
    """Directional differences of the kernel's own fp32-summed loss.  The step h moves
    the bf16 inputs exactly (multiples of 2^-6 times +-1); the output's rounding enters the
    loss as noise of at most 2^-8 |o| per element, each of random sign."""
    n, d = 96, 64
    q, k, v, do = inputs(1, 2, 1, n, d, 14)
    h = 2.0 ** -4
    q, k, v = ((x.float() * 2 ** 5).round() / 2 ** 5 for x in (q, k, v))  # exact in bf16 with the step
    args = [x.clamp(-2, 2).bfloat16().cuda() for x in (q, k, v)]
    dod = do.cuda()
    o, lse = run_fwd(*args, None, 40, 3)
    grads = run_bwd(*args, o, dod, lse, None, 40, 3)
    g = torch.Generator().manual_seed(1)
    for i in range(3):
        way = (torch.randint(0, 2, args[i].shape, generator=g) * 2 - 1).float().cuda()
        moved = []
        for sign in (1, -1):
            a = list(args)
            a[i] = (args[i].float() + sign * h * way).bfloat16()
            assert torch.equal(a[i].float(), args[i].float() + sign * h * way)
            moved.append(f64(run_fwd(*a, None, 40, 3)[0]))
        want = ((moved[0] - moved[1]) * f64(do)).sum() / (2 * h)
        got = (f64(grads[i]) * f64(way)).sum()
        exact, bounds = sink.bwd(*(f64(a) for a in args), f64(do), 40, 3, None, HALF_STEP)
        # noise of 2 n heads d roundings of 2^-8 |o dO|, at four of their standard deviations,
        # and the central difference's own h^2 term, bounded by the same differences in fp64
        noise = 4 * HALF_STEP * np.sqrt((f64(o) ** 2 * f64(do) ** 2).sum() * 2) / (2 * h)
        wide = [sink.fwd(*(f64(x) if j != i else f64(x) + s * h * f64(way) for j, x in enumerate(args)),
                         40, 3)[0] for s in (1, -1)]
        curve = abs(((wide[0] - wide[1]) * f64(do)).sum() / (2 * h) - (exact[i] * f64(way)).sum())
        assert abs(got - want) <= noise + curve + bounds[i].sum()
