"""GPU checks of the single-token attention over the 4-bit cache at the ends of its
range, against the fp64 oracle, in the tolerances of test_gpu_kv4."""

import pytest
import torch

from oracle import kv4
from tests.test_gpu_kv4 import PAGE, Cache, check_decode, i32, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [4, 18])  # one set of heads a block, and two
@pytest.mark.parametrize("up", [110, 112, 113, 120, 123, 124, 125, 126, 127])
def test_decode_of_the_largest_queries(up, heads, d):
    """Queries up to the largest bf16, keys as small, so that the scores are moderate.

    A score is a sum in units of 2^-(7 + e), 2^e the largest power of two in the query's
    row; with e = 127 the smallest float, 2^-149, is 2^-15 / sqrt(d) <= 2^-18 of a score.  The
    sums over the groups of channels round at most 2 d / 32 + 3 <= 11 times by half of that:
    2.1e-5, within the 1e-4 of the log-sum-exp."""
    n, lengths, window, sinks = 160, [160, 33], 120, 3
    c = Cache(2, 2, d, n // PAGE)
    k = (rows((2, 2, n, d), 5, torch.float32) * 2.0 ** -up).bfloat16()
    v = rows((2, 2, n, d), 6, torch.bfloat16)
    c.write(k.cuda(), v.cuda(), None, i32(lengths))
    g = torch.Generator().manual_seed(up)
    q = (torch.rand(2, heads, d, generator=g).double() * 1.99).bfloat16().double()
    q *= torch.randint(0, 2, q.shape, generator=g) * 2 - 1
    q[:, 1] *= 0.25  # a head that is not as large beside those that are
    q = q * 2.0 ** up
    assert torch.isfinite(q.bfloat16()).all() and torch.equal(q.bfloat16().double(), q)
    check_decode(c, q.bfloat16(), kv4.values(k.double().numpy()), kv4.values(v.double().numpy()),
                 lengths, window, sinks)
