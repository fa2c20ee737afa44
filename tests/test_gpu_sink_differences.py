"""GPU checks of the windowed attention's gradients against differences of its own
forward, in directions where a wrong gradient shows, and of the backward at large scores.

Differences: the loss is sum(O dO), the direction the sign of the fp64 gradient, so that the
derivative is the sum of all its absolute values, and the step 2^-6 moves inputs that are
multiples of it exactly.  Three things part the central difference from the gradient:
  - O's roundings.  Its own and that of each weight, at most 2^-8 of the term and of random
    sign, enter the loss with dO: four of their standard deviations, of two passes, over
    the double step;
  - the difference's own h^2 term: what the fp64 oracle has of it, the oracle being off by
    nothing else;
  - the gradient's roundings, random in sign too: four times the root of their squares.
The sum has to stay below a quarter of the derivative, and the check must turn away a
gradient of 0, its negative and its double."""

import numpy as np
import pytest
import torch

from oracle import sink
from tests.gpu_util import f64
from tests.test_gpu_sink import HALF_STEP, i32, inputs, run_bwd, run_fwd

pytestmark = pytest.mark.gpu

H = 2.0 ** -6


def squared_roundings(q, k, v, do, window, sinks, lengths):
    """Sum over O's elements of dO^2 (o^2 + sum_j (p_j v_j)^2)."""
    total = 0.0
    group = q.shape[1] // k.shape[1]
    for b in range(q.shape[0]):
        mask = sink.visible(q.shape[2], lengths[b], window, sinks)
        for h in range(q.shape[1]):
            p, _ = sink._weights(q[b, h], k[b, h // group], mask)
            vv = v[b, h // group]
            total += (do[b, h] ** 2 * ((p @ vv) ** 2 + p ** 2 @ vv ** 2)).sum()
    return total


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv_heads,n,lengths,window,sinks", [
    (2, 1, 96, [96], 40, 3), (4, 2, 300, [300, 171], 64, 4), (3, 3, 200, [200], 1000, 0)])
def test_gradients_against_differences(heads, kv_heads, n, lengths, window, sinks, d):
    q, k, v, do = inputs(len(lengths), heads, kv_heads, n, d, n + d)
    # multiples of 2^-6 below 2, and so are they a step further: exact in bf16
    q, k, v = ((x.float().clamp(-1.5, 1.5) / H).round() * H for x in (q, k, v))
    args, dod = [x.bfloat16().cuda() for x in (q, k, v)], do.cuda()
    exact_args = [f64(a) for a in args]
    o, lse = run_fwd(*args, i32(lengths), window, sinks)
    grads = run_bwd(*args, o, dod, lse, i32(lengths), window, sinks)
    wants, bounds = sink.bwd(*exact_args, f64(do), window, sinks, lengths, HALF_STEP)
    rounding = 4 * HALF_STEP * np.sqrt(
        2 * squared_roundings(*exact_args, f64(do), window, sinks, lengths)) / (2 * H)
    for i, name in enumerate("qkv"):
        way = np.where(wants[i] >= 0, 1.0, -1.0)
        loss, exact_loss = [], []
        for sign in (1, -1):
            moved = list(exact_args)
            moved[i] = exact_args[i] + sign * H * way
            on = [torch.from_numpy(x).bfloat16() for x in moved]
            assert np.array_equal(f64(on[i]), moved[i])
            loss.append((f64(run_fwd(*(x.cuda() for x in on), i32(lengths), window, sinks)[0])
                         * f64(do)).sum())
            exact_loss.append((sink.fwd(*moved, window, sinks, lengths)[0] * f64(do)).sum())
        want = (loss[0] - loss[1]) / (2 * H)
        exact = (wants[i] * way).sum()
        curve = abs((exact_loss[0] - exact_loss[1]) / (2 * H) - exact)
        limit = rounding + curve + 4 * np.sqrt((bounds[i] ** 2).sum())
        got = (f64(grads[i]) * way).sum()
        assert limit < abs(want) / 4, (name, limit, want)
        assert abs(got - want) <= limit, (name, got, want, limit)
        for wrong in (0.0, -got, 2 * got):
            assert abs(wrong - want) > limit, (name, wrong)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lengths,window,sinks", [([400], 350, 2), ([391], 20, 4)])
def test_backward_at_large_scores(lengths, window, sinks, d):
    """Scores of a few hundred.  Their sums before the factor 1 / sqrt(d) pass through 2^12,
    in fp32 off by up to 2^-12 at each of d / 16 steps: 2^-12 of a weight after the
    factor, and as much again in the log-sum-exp: every weight is off by 2^-11 more."""
    q, k, v, do = inputs(1, 2, 2, 400, d, 8)
    ramp = torch.linspace(0.1, 9.5, 400)[None, None, :, None]
    q, k = (q * ramp).bfloat16(), (k * ramp).bfloat16()
    assert 200 < (f64(q)[0, 0] @ f64(k)[0, 0].T).max() / np.sqrt(d) and \
        np.abs(f64(q)[0, 0] @ f64(k)[0, 0].T).max() < 2 ** 12
    o, lse = run_fwd(q.cuda(), k.cuda(), v.cuda(), i32(lengths), window, sinks)
    grads = run_bwd(q.cuda(), k.cuda(), v.cuda(), o, do.cuda(), lse, i32(lengths), window, sinks)
    args = [f64(x) for x in (q, k, v, do)]
    wants, bounds = sink.bwd(*args, window, sinks, lengths, HALF_STEP + 2.0 ** -11)
    for name, g, w, tol in zip(("dq", "dk", "dv"), grads, wants, bounds):
        limit = tol * (1 + 1e-4 / HALF_STEP) + 1e-4 * np.abs(w).max()
        assert (np.abs(f64(g) - w) <= limit).all(), name
        # a wrong gradient is not within these bounds
        assert (np.abs(w) > limit).any() and (np.abs(2 * f64(g) - w) > limit).any()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv_heads,n,window,sinks", [
    (4, 2, 700, 160, 4), (2, 1, 900, 2147483647, 0), (8, 1, 600, 300, 33)])
def test_gradients_in_the_norm(heads, kv_heads, n, window, sinks, d):
    """Each is off by two independent roundings to bf16, of P or dS and of the result:
    2.35e-3 of the norm (test_gpu_sink has the arithmetic).  D of rows of many keys takes O's
    rounding in, 1.66e-3 over the root of the row's effective number of keys, 12 or more: in
    quadrature 2.4e-3.  The allowance for a finite sample brings 2.8e-3, and a gradient that is
    off by a hundredth is turned away."""
    q, k, v, do = inputs(2, heads, kv_heads, n, d, n)
    qd, kd, vd, dod = (x.cuda() for x in (q, k, v, do))
    o, lse = run_fwd(qd, kd, vd, None, window, sinks)
    grads = run_bwd(qd, kd, vd, o, dod, lse, None, window, sinks)
    wants, _ = sink.bwd(*(f64(x) for x in (q, k, v, do)), window, sinks)
    for g, w in zip(grads, wants):
        limit = 2.8e-3 * np.linalg.norm(w)
        assert np.linalg.norm(f64(g) - w) <= limit
        assert np.linalg.norm(1.01 * f64(g) - w) > limit
