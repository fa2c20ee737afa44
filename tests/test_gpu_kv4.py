"""GPU parity of the 4-bit cache (nb_kv4_write, nb_kv4_read) and of the
single-token attention over it (nb_attn_kv4_decode) against the fp64 oracle.

Tolerances.  The cache's values are exact in fp64; reading rounds once, so fp32
read-back equals the oracle's fp32 value and bf16 read-back is within half a
step, 2^-8 relative.  The attention output adds to that final rounding (2^-8 of
|o|) the rounding of each p s to bf16 (2^-8 of the term): its sum over the terms
is at most 2^-8 sum_j p_j s_j 7.5 <= 2^-8 max_j |v_j - m_j|, in all
2^-8 (|o| + R) with R the largest |value - midpoint| (bounded below by the value
range); fp32 arithmetic adds less than 1e-4 of R.  The log-sum-exp has no bf16
rounding: fp32 sums of d products, ex2.approx (2 ulp): 1e-4.
"""

import numpy as np
import pytest
import torch

import block_sparse_local_nb_b200 as nb
from oracle import kv4

pytestmark = pytest.mark.gpu

PAGE = 32


def code_of(dtype):
    return nb.NB_F32 if dtype == torch.float32 else nb.NB_BF16


def rows(shape, seed, dtype):
    """Rows with channel offsets and a few large channels, as keys have."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    size = 0.5 + torch.rand(shape[-1], generator=g)
    size[::16] *= 4
    return (x * size + torch.randn(shape[-1], generator=g)).to(dtype)


class Cache:
    """A pool with a shuffled block table, filled with 0xa5 (NaN-free but odd)."""

    def __init__(self, batch, kv_heads, d, max_pages, seed=0, spare=3, fill=0xA5):
        g = torch.Generator().manual_seed(seed)
        self.num = batch * max_pages + spare
        order = torch.randperm(self.num, generator=g)[:batch * max_pages]
        self.table = order.reshape(batch, max_pages).to(torch.int32).cuda()
        self.pool = torch.full((self.num, kv_heads, nb.kv4_page_bytes(d)), fill,
                               dtype=torch.uint8, device="cuda")
        self.batch, self.kv_heads, self.d, self.max_pages = batch, kv_heads, d, max_pages

    def write(self, k, v, starts=None, counts=None, **kw):
        n = k.shape[2]
        nb.nb_kv4_write(k, v, self.pool, self.table, starts, counts, self.batch, self.kv_heads, n,
                        self.d, self.max_pages, self.num, code_of(k.dtype), **kw)

    def read(self, n, dtype, starts=None, counts=None):
        k = torch.full((self.batch, self.kv_heads, n, self.d), 7.0, dtype=dtype, device="cuda")
        v = k.clone()
        nb.nb_kv4_read(self.pool, self.table, starts, counts, k, v, self.batch, self.kv_heads, n,
                       self.d, self.max_pages, self.num, code_of(dtype))
        return k, v

    def decode(self, q, lengths, window, sinks, with_lse=True, splits_ws=None):
        heads = q.shape[1]
        size = nb.attn_kv4_decode_workspace_size(self.batch, heads, self.kv_heads, self.d,
                                                 self.max_pages, window, sinks, nb.NB_BF16)
        ws = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
        o = torch.full_like(q, 9.0)
        lse = torch.full(q.shape[:2], 9.0, dtype=torch.float32, device="cuda") if with_lse else None
        nb.nb_attn_kv4_decode(q, self.pool, self.table, lengths, o, lse, ws, size, self.batch,
                              heads, self.kv_heads, self.d, self.max_pages, self.num, window, sinks,
                              nb.NB_BF16)
        return o, lse


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,starts,counts", [(1, [0, 31], [1, 1]), (5, [30, 63], [5, 3]),
                                             (33, [0, 7], [33, 0]), (130, [1, 95], [129, 130])])
def test_write_then_read(n, starts, counts, dtype, d):
    c = Cache(2, 3, d, 8, seed=n)
    k, v = rows((2, 3, n, d), n + d, dtype), rows((2, 3, n, d), n + d + 1, dtype)
    c.write(k.cuda(), v.cuda(), i32(starts), i32(counts))
    for out in (torch.float32, torch.bfloat16):
        got = c.read(n, out, i32(starts), i32(counts))
        for x, y in zip((k, v), got):
            want = kv4.values(x.double().numpy())
            y = y.cpu()
            for b, m in enumerate(counts):
                if out == torch.float32:
                    assert np.array_equal(y[b, :, :m].numpy(), want[b, :, :m].astype(np.float32))
                else:
                    err = np.abs(y[b, :, :m].double().numpy() - want[b, :, :m])
                    assert (err <= 2.0 ** -8 * np.abs(want[b, :, :m])).all()
                assert (y[b, :, m:] == 0).all()


@pytest.mark.parametrize("d", [64, 128])
def test_only_listed_bytes_change(d):
    """Appending token 70 of one sequence and none of the other touches one slot of one page."""
    c = Cache(2, 2, d, 4)
    before = c.pool.clone()
    k = rows((2, 2, 1, d), 1, torch.bfloat16).cuda()
    c.write(k, k, i32([70, 5]), i32([1, 0]))
    changed = (c.pool != before).any(-1)  # [page, head]
    page = int(c.table[0, 70 // 32])
    assert changed[page].all()
    changed[page] = False
    assert not changed.any()
    # inside the page: a row of codes and a row of params of K and of V
    per_page = (c.pool[page] != before[page]).sum(-1)
    assert (per_page <= 2 * (d // 2 + d // 8)).all()
    nxt, _ = c.read(1, torch.float32, i32([71, 0]))
    c2 = Cache(2, 2, d, 4)
    same, _ = c2.read(1, torch.float32, i32([71, 0]))
    assert torch.equal(nxt[0].nan_to_num(), same[0].nan_to_num())  # the next slot is as it was


def test_token_by_token_equals_one_write():
    k, v = rows((2, 2, 70, 128), 3, torch.bfloat16).cuda(), rows((2, 2, 70, 128), 4, torch.bfloat16).cuda()
    a, b = Cache(2, 2, 128, 3, fill=0), Cache(2, 2, 128, 3, fill=0)
    a.write(k, v)
    for t in range(70):
        b.write(k[:, :, t:t + 1].contiguous(), v[:, :, t:t + 1].contiguous(), i32([t, t]))
    assert torch.equal(a.pool, b.pool)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_odd_groups(dtype):
    """Constant, zero, one-sided, huge, tiny and non-finite groups."""
    x = torch.zeros(1, 1, 12, 64)
    x[0, 0, 1] = 3.140625
    x[0, 0, 2, 5] = -7.0
    x[0, 0, 3] = torch.linspace(1e30, 3e30, 64)
    x[0, 0, 4] = torch.linspace(-2e-30, 1e-30, 64)
    x[0, 0, 5, 40] = float("nan")
    x[0, 0, 6, 2] = float("inf")
    x[0, 0, 7] = 100.0 + 0.5 * torch.arange(64)
    x[0, 0, 8] = torch.arange(64) - 31.5
    x[0, 0, 9] = -x[0, 0, 8]
    x[0, 0, 10] = torch.tensor([1.0, -1.0]).repeat(32) * 1e-3
    x[0, 0, 11, ::2] = float("-inf")
    x = x.to(dtype)
    c = Cache(1, 1, 64, 1)
    c.write(x.cuda(), x.cuda())
    k, v = c.read(12, torch.float32)
    with np.errstate(over="ignore"):
        want = kv4.values(x.double().numpy()).astype(np.float32)
    assert np.array_equal(k.cpu().numpy(), want, equal_nan=True)
    assert np.array_equal(v.cpu().numpy(), want, equal_nan=True)


def test_subnormal_groups_are_exact():
    """Extremes whose sum is odd in units of 2^-149: its half is no fp32 number, and a
    midpoint just below a bf16 must not be rounded up to it."""
    g = np.random.default_rng(8)
    units = g.integers(-2 ** 18, 2 ** 18, (1, 1, 200, 64))
    for t, base in enumerate((2 ** 17, 2 ** 16, 3 * 2 ** 16, -2 ** 16, -2 ** 17)):
        units[0, 0, t] = base - g.integers(0, 2, 64)
        units[0, 0, t, ::32], units[0, 0, t, 1::32] = base - 1, base
    x = (units * 2.0 ** -149).astype(np.float32)
    assert np.array_equal(x.astype(np.float64), units * 2.0 ** -149)
    c = Cache(1, 1, 64, 7)
    xd = torch.from_numpy(x).cuda()
    c.write(xd, xd)
    for y in c.read(200, torch.float32):
        want = kv4.values(x.astype(np.float64))
        assert np.array_equal(y.cpu().numpy().astype(np.float64), want)


def test_every_border_is_exact():
    """Values on, just below and just above code borders of awkward steps."""
    g = np.random.default_rng(5)
    x = np.zeros((1, 1, 400, 64), np.float32)
    for t in range(400):
        step = np.float32(2.0 ** g.integers(-20, 20) * (128 + g.integers(0, 128)) / 128)
        mid = np.float32(step * g.integers(-40, 40) / 8)
        border = (mid + step * g.integers(-7, 8, 64)).astype(np.float32)
        border = np.nextafter(border, np.float32(g.choice([-np.inf, np.inf])) if t % 3 else border)
        border[0], border[1] = mid - np.float32(7.5) * step, mid + np.float32(7.5) * step
        border[32], border[33] = border[0], border[1]
        x[0, 0, t] = border
    c = Cache(1, 1, 64, 13)
    xd = torch.from_numpy(x).cuda()
    c.write(xd, xd)
    k, _ = c.read(400, torch.float32)
    assert np.array_equal(k.cpu().numpy(), kv4.values(x.astype(np.float64)).astype(np.float32))


def check_decode(c, q, kq, vq, lengths, window, sinks):
    o, lse = c.decode(q.cuda(), None if lengths is None else i32(lengths), window, sinks)
    L = lengths if lengths is not None else [c.max_pages * PAGE] * c.batch
    want, want_lse = kv4.decode(q.double().numpy(), kq, vq, L, window, sinks)
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    span = np.abs(vq).max()
    assert (np.abs(o - want) <= 2.0 ** -8 * (np.abs(want) + span) + 1e-4 * span).all()
    empty = np.isinf(want_lse)
    assert np.array_equal(np.isneginf(lse), empty)
    assert (o[empty] == 0).all()
    assert np.abs(lse[~empty] - want_lse[~empty]).max(initial=0) <= 1e-4
    return o


DECODE = [  # heads, kv_heads, lengths, window, sinks
    (2, 2, [1, 301], 301, 0), (4, 2, [0, 33], 1000, 4), (3, 3, [64, 31], 7, 0),
    (10, 1, [95, 200], 50, 33), (16, 1, [127, 128], 1, 1), (36, 2, [255, 256], 60, 128),
    (8, 1, [5, 256], 3, 128), (5, 1, [256, 2], 2147483647, 0)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,kv_heads,lengths,window,sinks", DECODE)
def test_decode(heads, kv_heads, lengths, window, sinks, d):
    n = 256
    c = Cache(2, kv_heads, d, n // PAGE, seed=heads, fill=0xFF)  # unwritten params are NaN
    k, v = rows((2, kv_heads, n, d), heads, torch.bfloat16), rows((2, kv_heads, n, d), 7, torch.bfloat16)
    c.write(k.cuda(), v.cuda(), None, i32(lengths))
    q = torch.randn(2, heads, d, generator=torch.Generator().manual_seed(d)).bfloat16()
    check_decode(c, q, kv4.values(k.double().numpy()), kv4.values(v.double().numpy()), lengths,
                 window, sinks)


@pytest.mark.parametrize("d,batch,kv_heads,heads,n,window,sinks",
                         [(64, 1, 1, 4, 20000, 1 << 30, 0), (128, 3, 2, 2, 9001, 4096, 4),
                          (128, 1, 2, 16, 5000, 1 << 30, 0), (128, 1, 2, 16, 1000, 1 << 30, 0),
                          (64, 2, 1, 9, 700, 400, 33), (128, 40, 1, 3, 1500, 1 << 30, 0)])
def test_decode_long_in_shares(d, batch, kv_heads, heads, n, window, sinks):
    """Long sequences are cut into shares that are joined; twice gives the same bits."""
    pages = -(-n // PAGE) + 2
    c = Cache(batch, kv_heads, d, pages, fill=0xFF)
    k, v = (rows((batch, kv_heads, n, d), s, torch.bfloat16) for s in (1, 2))
    lengths = [n - 37 * b for b in range(batch)]
    c.write(k.cuda(), v.cuda(), None, i32(lengths))
    # rows of many shares go through the workspace, the others join in clusters
    assert bool(nb.attn_kv4_decode_workspace_size(batch, heads, kv_heads, d, pages, window, sinks,
                                                  nb.NB_BF16)) == (n >= 5000)
    q = torch.randn(batch, heads, d, generator=torch.Generator().manual_seed(3)).bfloat16()
    kq, vq = kv4.values(k.double().numpy()), kv4.values(v.double().numpy())
    a = check_decode(c, q, kq, vq, lengths, window, sinks)
    assert np.array_equal(a, check_decode(c, q, kq, vq, lengths, window, sinks))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("up,down", [(-130, 0), (-100, 0), (60, -60), (118, -118), (0, 40)])
def test_decode_of_queries_and_keys_of_any_size(up, down, d):
    """Queries by 2^up (subnormal ones too), keys by 2^down where the product stays
    moderate; (0, 40): the channels of a query 2^40 apart, one head's query 0.
    Subnormal fp32 sums keep 2^-18 of a score, well inside the 1e-4."""
    n, lengths = 192, [192, 70]
    wide = down > 0
    c = Cache(2, 2, d, n // PAGE)
    k = (rows((2, 2, n, d), 5, torch.float32) * 2.0 ** (0 if wide else down)).bfloat16()
    v = rows((2, 2, n, d), 6, torch.bfloat16)
    c.write(k.cuda(), v.cuda(), None, i32(lengths))
    q = torch.randn(2, 6, d, generator=torch.Generator().manual_seed(d)).double()
    if wide:
        q[..., ::2] *= 2.0 ** -down
        q[:, 1] = 0
    q = (q * 2.0 ** up).bfloat16()
    check_decode(c, q, kv4.values(k.double().numpy()), kv4.values(v.double().numpy()), lengths, 100, 3)


@pytest.mark.parametrize("n", [1, 100, 1000, 3000, 20000])  # one warp, a block, a cluster, the workspace
def test_decode_of_what_is_not_a_number(n):
    """A key that is no number, where it is visible, makes its head's outputs none; a
    value makes its group of channels none; where they are hidden nothing changes."""
    pages = -(-n // PAGE)
    c = Cache(1, 3, 64, pages)
    k, v = (rows((1, 3, n, 64), s, torch.bfloat16) for s in (1, 2))
    k[0, 1, n // 2, 5] = float("inf")
    v[0, 2, n // 2, 40] = float("nan")
    c.write(k.cuda(), v.cuda())
    q = torch.randn(1, 6, 64, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    o, lse = c.decode(q, i32([n]), n, 0)
    lse, o = lse.isnan()[0].tolist(), o.isnan()[0]
    assert lse == [False] * 2 + [True] * 2 + [False] * 2
    assert not o[:2].any() and o[2:4].all() and not o[4:, :32].any() and o[4:, 32:].all()
    if n > 1:
        o, lse = c.decode(q, i32([n]), n - 1 - n // 2, 0)
        assert not o.isnan().any() and not lse.isnan().any()


def test_decode_in_graphs_on_streams_and_at_once():
    """Shares through the workspace: captured and replayed on new inputs, and two calls
    at once on two streams with a workspace each, give the bits of plain calls."""
    n, heads = 20000, 4
    pages = -(-n // PAGE)
    shape = (1, heads, 1, 64, pages, pages + 3, 1 << 30, 0, nb.NB_BF16)
    caches, qs, lens, outs, spaces = [], [], [], [], []
    size = nb.attn_kv4_decode_workspace_size(1, heads, 1, 64, pages, 1 << 30, 0, nb.NB_BF16)
    assert size > 0
    for s in range(2):
        c = Cache(1, 1, 64, pages, seed=s)
        c.write(rows((1, 1, n, 64), s, torch.bfloat16).cuda(), rows((1, 1, n, 64), 5 + s, torch.bfloat16).cuda())
        caches.append(c)
        qs.append(torch.randn(1, heads, 64, generator=torch.Generator().manual_seed(s)).bfloat16().cuda())
        lens.append(i32([n - 1000 * s]))
        outs.append((torch.empty_like(qs[s]), torch.empty(1, heads, device="cuda")))
        spaces.append(torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda"))

    def step(s):
        nb.nb_attn_kv4_decode(qs[s], caches[s].pool, caches[s].table, lens[s], *outs[s], spaces[s],
                              size, *shape)

    want = [caches[s].decode(qs[s], lens[s], 1 << 30, 0) for s in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s in range(2):
            with torch.cuda.stream(streams[s]):
                step(s)
    torch.cuda.synchronize()
    for s in range(2):
        assert all(torch.equal(x, y) for x, y in zip(outs[s], want[s]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(0)
    for q, length in ((qs[0], n), (qs[1], 777), (qs[0], 0)):
        q, now = q.clone(), i32([length])
        want = caches[0].decode(q, now, 1 << 30, 0)
        qs[0].copy_(q)
        lens[0].copy_(now)
        spaces[0].fill_(0xFF)
        graph.replay()
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip(outs[0], want))


def test_decode_lengths_null_and_clamped():
    c = Cache(2, 1, 64, 2)
    k, v = (rows((2, 1, 64, 64), s, torch.bfloat16) for s in (1, 2))
    c.write(k.cuda(), v.cuda())
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(3)).bfloat16()
    kq, vq = kv4.values(k.double().numpy()), kv4.values(v.double().numpy())
    a = check_decode(c, q, kq, vq, None, 100, 0)
    o, lse = c.decode(q.cuda(), i32([1000, -5]), 100, 0)
    assert np.array_equal(o[0].double().cpu().numpy(), a[0])
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()
    o2, none = c.decode(q.cuda(), None, 100, 0, with_lse=False)
    assert none is None and np.array_equal(o2.double().cpu().numpy(), a)


def test_pages_outside_the_window_need_no_mapping():
    c = Cache(1, 1, 64, 8, fill=0xFF)
    k, v = (rows((1, 1, 256, 64), s, torch.bfloat16) for s in (1, 2))
    c.write(k.cuda(), v.cuda())
    c.table[0, 1:5] = -1  # tokens 32..159: neither sinks (< 4) nor in the window
    q = torch.randn(1, 2, 64, generator=torch.Generator().manual_seed(3)).bfloat16()
    check_decode(c, q, kv4.values(k.double().numpy()), kv4.values(v.double().numpy()), [256], 96, 4)


def test_unmapped_positions_are_skipped_and_reported():
    """Entries below zero and past the pool: nothing is written, rows read as 0, a
    page is not seen; each is reported once through nb_kernel_error."""
    c = Cache(1, 2, 64, 3, fill=0)
    good = c.table.clone()
    c.table[0, 1] = c.num
    k, v = (rows((1, 2, 96, 64), s, torch.bfloat16) for s in (1, 2))
    c.write(k.cuda(), v.cuda())
    assert nb.nb_kernel_error() == 0x51
    used = {int(good[0, 0]), int(good[0, 2])}
    for page in range(c.num):
        assert bool(c.pool[page].any()) == (page in used)
    kr, vr = c.read(96, torch.float32)
    assert nb.nb_kernel_error() == 0x52
    assert (kr[0, :, 32:64] == 0).all() and (vr[0, :, 32:64] == 0).all()
    kq, vq = kv4.values(k.double().numpy()), kv4.values(v.double().numpy())
    q = torch.randn(1, 2, 64, generator=torch.Generator().manual_seed(3)).bfloat16()
    keep = np.r_[0:32, 64:96]
    o, lse = c.decode(q.cuda(), i32([96]), 96, 0)
    assert nb.nb_kernel_error() == 0x53
    want, want_lse = kv4.decode(q.double().numpy(), kq[:, :, keep], vq[:, :, keep], [64], 64, 0)
    assert np.abs(lse.cpu().numpy() - want_lse).max() <= 1e-4
    c.table[0, 1] = -7
    c.write(k.cuda(), v.cuda(), i32([-3]))
    assert nb.nb_kernel_error() == 0x51
    c.write(k.cuda(), v.cuda(), i32([90]), i32([7]))
    assert nb.nb_kernel_error() == 0x51  # position 96 is past the table


def test_pool_offsets_past_32_bits():
    """Pages whose byte offsets pass 2^32, reached through the table."""
    num, d = 900_000, 128  # 4.6 GB
    pool = torch.empty((num, 1, nb.kv4_page_bytes(d)), dtype=torch.uint8, device="cuda")
    table = i32([[num - 1, 3, num - 2]])
    k, v = (rows((1, 1, 90, d), s, torch.bfloat16) for s in (1, 2))
    nb.nb_kv4_write(k.cuda(), v.cuda(), pool, table, None, None, 1, 1, 90, d, 3, num, nb.NB_BF16)
    ko, vo = torch.empty(1, 1, 90, d, device="cuda"), torch.empty(1, 1, 90, d, device="cuda")
    nb.nb_kv4_read(pool, table, None, None, ko, vo, 1, 1, 90, d, 3, num, nb.NB_F32)
    kq, vq = kv4.values(k.double().numpy()), kv4.values(v.double().numpy())
    assert np.array_equal(ko.cpu().numpy(), kq.astype(np.float32))
    assert np.array_equal(vo.cpu().numpy(), vq.astype(np.float32))
    q = torch.randn(1, 4, d, generator=torch.Generator().manual_seed(3)).bfloat16()
    o, lse = torch.empty(1, 4, d, dtype=torch.bfloat16, device="cuda"), torch.empty(1, 4, device="cuda")
    nb.nb_attn_kv4_decode(q.cuda(), pool, table, i32([90]), o, lse, None, 0, 1, 4, 1, d, 3, num, 90, 0,
                          nb.NB_BF16)
    want, want_lse = kv4.decode(q.double().numpy(), kq, vq, [90], 90, 0)
    span = np.abs(vq).max()
    assert (np.abs(o.double().cpu().numpy() - want) <= 2.0 ** -8 * (np.abs(want) + span) + 1e-4 * span).all()
    assert np.abs(lse.double().cpu().numpy() - want_lse).max() <= 1e-4


def test_no_pages_at_all():
    """A table without pages: rows read as 0 and are reported; a decode gives 0."""
    k = torch.ones(2, 1, 3, 64, dtype=torch.bfloat16, device="cuda")
    nb.nb_kv4_write(k, k, None, None, None, None, 2, 1, 3, 64, 0, 0, nb.NB_BF16)
    assert nb.nb_kernel_error() == 0x51
    out = torch.ones_like(k)
    nb.nb_kv4_read(None, None, None, None, out, out.clone(), 2, 1, 3, 64, 0, 0, nb.NB_BF16)
    assert nb.nb_kernel_error() == 0x52 and (out == 0).all()
    o = torch.ones(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    nb.nb_attn_kv4_decode(o.clone(), None, None, None, o, None, None, 0, 2, 2, 1, 64, 0, 0, 5, 0, nb.NB_BF16)
    assert (o == 0).all()


def test_serving_from_prompt_to_tokens():
    """The operators as a program uses them: a ragged prompt through the windowed
    attention and into the cache, then tokens one by one through a captured step; each
    token's output is the windowed attention's last row over what the cache reads back."""
    from block_sparse_local_nb_b200.layer import KV4Cache, sink_attention
    from oracle import sink

    batch, heads, kv_heads, d, window, sinks = 3, 8, 2, 64, 70, 4
    prompts, steps = [100, 33, 1], 40
    n = max(prompts) + steps
    g = torch.Generator().manual_seed(21)
    q = torch.randn(batch, heads, n, d, generator=g).bfloat16().cuda()
    k = rows((batch, kv_heads, n, d), 22, torch.bfloat16).cuda()
    v = rows((batch, kv_heads, n, d), 23, torch.bfloat16).cuda()
    L = i32(prompts)
    p = max(prompts)
    out = sink_attention(q[:, :, :p], k[:, :, :p], v[:, :, :p], L, window, sinks)
    assert all((out[b, :, m:] == 0).all() for b, m in enumerate(prompts))
    cache = KV4Cache(batch, kv_heads, d, n)
    cache.append(k[:, :, :p], v[:, :, :p], L)
    assert cache.lengths.tolist() == prompts
    # sequence b's next tokens are its own rows prompts[b], prompts[b] + 1, ...
    at = torch.tensor(prompts, device="cuda")
    step_k = torch.empty(batch, kv_heads, 1, d, dtype=torch.bfloat16, device="cuda")
    step_v, step_q = torch.empty_like(step_k), torch.empty(batch, heads, d, dtype=torch.bfloat16, device="cuda")
    seq = torch.arange(batch, device="cuda")

    def feed(i):
        step_q.copy_(q[seq, :, at + i])
        step_k.copy_(k[seq, :, at + i][:, :, None])
        step_v.copy_(v[seq, :, at + i][:, :, None])

    def step():
        cache.append(step_k, step_v)
        return cache.attend(step_q, window, sinks)

    feed(0)
    got = [step().clone()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = step()
    for i in range(1, steps):
        feed(i)
        graph.replay()
        got.append(static.clone())
    torch.cuda.synchronize()
    assert cache.lengths.tolist() == [m + steps for m in prompts]
    kq, vq = cache.read(n, dtype=torch.float32)
    ks, vs = kv4.values(k.double().cpu().numpy()), kv4.values(v.double().cpu().numpy())
    for b, m in enumerate(prompts):
        assert np.array_equal(kq[b, :, :m + steps].cpu().numpy(), ks[b, :, :m + steps].astype(np.float32))
    span = np.abs(vs).max()
    want, _ = sink.fwd(q.double().cpu().numpy(), ks, vs, window, sinks, [m + steps for m in prompts])
    for i in range(steps):
        for b, m in enumerate(prompts):
            w = want[b, :, m + i]
            off = np.abs(got[i][b].double().cpu().numpy() - w)
            assert (off <= 2.0 ** -8 * (np.abs(w) + span) + 1e-4 * span).all()
