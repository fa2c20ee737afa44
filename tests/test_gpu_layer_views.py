"""GPU checks of the layer's windowed attention and 4-bit cache on contiguous views that
begin between two 16-byte boundaries, as a gradient that is a piece of a larger one does."""

import pytest
import torch

from block_sparse_local_nb_b200.layer import KV4Cache, sink_attention
from tests.test_gpu_sink import inputs

pytestmark = pytest.mark.gpu


def odd(x):
    """The same values in a contiguous view three elements into its storage."""
    y = torch.empty(x.numel() + 3, dtype=x.dtype, device=x.device)
    y[3:] = x.flatten()
    y = y[3:].view(x.shape)
    assert y.is_contiguous() and y.data_ptr() % 16 != 0
    return y


def test_attention_and_its_gradients():
    q, k, v, do = (x.cuda() for x in inputs(2, 4, 2, 130, 64, 3))
    leaves = [x.clone().requires_grad_(True) for x in (q, k, v)]
    want = sink_attention(*leaves, None, 40, 2)
    grads = torch.autograd.grad(want, leaves, do)
    held = [odd(x).requires_grad_(True) for x in (q, k, v)]
    o = sink_attention(*held, None, 40, 2)
    assert torch.equal(o, want)
    for x, y in zip(torch.autograd.grad(o, held, odd(do)), grads):
        assert torch.equal(x, y)


def test_a_gradient_that_is_a_piece_of_another():
    """The backward of a concatenation hands out views."""
    q, k, v, do = (x.cuda() for x in inputs(1, 2, 1, 70, 64, 4))
    leaves = [x.clone().requires_grad_(True) for x in (q, k, v)]
    want = torch.autograd.grad(sink_attention(*leaves, None, 20, 1), leaves, do)
    o = sink_attention(*leaves, None, 20, 1)
    lead = torch.zeros(3, dtype=o.dtype, device="cuda", requires_grad=True)
    whole = torch.cat([lead, o.flatten()])
    got = torch.autograd.grad(whole, leaves, torch.cat([lead.detach(), do.flatten()]))
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_cache():
    q, k, v, _ = (x.cuda() for x in inputs(2, 4, 2, 33, 128, 5))
    a, b = KV4Cache(2, 2, 128, 40), KV4Cache(2, 2, 128, 40)
    a.append(k, v)
    b.append(odd(k), odd(v))
    assert torch.equal(a.pool, b.pool)
    last = q[:, :, -1].contiguous()
    assert torch.equal(a.attend(last, 20, 2), b.attend(odd(last), 20, 2))
