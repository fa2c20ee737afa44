"""CPU checks of the windowed attention with sinks and of the 4-bit cache: the
host-side refusals of their entry points (these calls return before any CUDA
call), their sizes, the argument checks of the layer, and the fp64 oracles
against independent forms."""

import numpy as np
import pytest
import torch

from block_sparse_local_nb_b200 import layer
from oracle import attn_bwd_dense, attn_fwd_dense, kv4, sink

NB_OK, INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 0, -1, -2, -3, -5
F32, BF16 = 0, 1


def call(fn, names, defaults, kw):
    args = dict(defaults, **kw)
    return fn(*(args[n] for n in names), None)


SINK = dict(batch=1, heads=2, kv_heads=1, n=70, d=64, window=16, sinks=4, dtype=BF16)
SINK_BAD = [
    (dict(batch=-1), INVALID), (dict(heads=-2), INVALID), (dict(kv_heads=0), INVALID),
    (dict(heads=3, kv_heads=2), INVALID), (dict(n=-1), INVALID), (dict(window=0), INVALID),
    (dict(sinks=-1), INVALID), (dict(dtype=5), INVALID), (dict(sinks=129), UNSUPPORTED),
    (dict(d=96), UNSUPPORTED), (dict(dtype=F32), UNSUPPORTED), (dict(heads=70000, kv_heads=1), UNSUPPORTED),
    (dict(batch=70000), UNSUPPORTED), (dict(n=2147483647), UNSUPPORTED), (dict(q=None), INVALID),
    (dict(v=None), INVALID), (dict(o=None), INVALID), (dict(k=24), MISALIGNED), (dict(lse=20), MISALIGNED),
    (dict(lengths=18), MISALIGNED), (dict(batch=0), NB_OK), (dict(n=0), NB_OK), (dict(heads=0), NB_OK)]


@pytest.mark.parametrize("kw,status", SINK_BAD)
def test_sink_fwd_refusals(built_lib, kw, status):
    names = ["q", "k", "v", "o", "lse", "lengths", *SINK]
    assert call(built_lib.nb_attn_sink_fwd, names,
                dict(SINK, q=16, k=16, v=16, o=16, lse=None, lengths=None), kw) == status


@pytest.mark.parametrize("kw,status", [x for x in SINK_BAD if "lse" not in x[0]] + [
    (dict(lse=None), INVALID), (dict(dout=None), INVALID), (dict(dk=None), INVALID),
    (dict(dq=8), MISALIGNED), (dict(ws=None), WORKSPACE), (dict(ws=272), WORKSPACE),
    (dict(ws_bytes=100), WORKSPACE)])
def test_sink_bwd_refusals(built_lib, kw, status):
    names = ["q", "k", "v", "o", "dout", "lse", "lengths", "dq", "dk", "dv", "ws", "ws_bytes", *SINK]
    base = dict(SINK, lengths=None, ws=256, ws_bytes=1 << 40)
    base.update({n: 16 for n in ("q", "k", "v", "o", "dout", "lse", "dq", "dk", "dv")})
    assert call(built_lib.nb_attn_sink_bwd, names, base, kw) == status


KV = dict(batch=2, kv_heads=3, n=5, d=64, max_pages=4, num_pages=9, dtype=BF16)
KV_BAD = [
    (dict(batch=-1), INVALID), (dict(kv_heads=0), INVALID), (dict(n=-1), INVALID),
    (dict(max_pages=-1), INVALID), (dict(num_pages=-1), INVALID), (dict(dtype=2), INVALID),
    (dict(d=32), UNSUPPORTED), (dict(batch=70000), UNSUPPORTED), (dict(kv_heads=70000), UNSUPPORTED),
    (dict(max_pages=1 << 26), UNSUPPORTED), (dict(k=None), INVALID), (dict(table=None), INVALID),
    (dict(cache=None), INVALID), (dict(v=40), MISALIGNED), (dict(cache=24), MISALIGNED),
    (dict(table=18), MISALIGNED), (dict(starts=18), MISALIGNED), (dict(counts=18), MISALIGNED),
    (dict(batch=0), NB_OK), (dict(n=0), NB_OK)]


@pytest.mark.parametrize("kw,status", KV_BAD)
def test_kv4_refusals(built_lib, kw, status):
    base = dict(KV, k=16, v=16, cache=16, table=16, starts=None, counts=None)
    assert call(built_lib.nb_kv4_write, ["k", "v", "cache", "table", "starts", "counts", *KV], base,
                kw) == status
    assert call(built_lib.nb_kv4_read, ["cache", "table", "starts", "counts", "k", "v", *KV], base,
                kw) == status


DEC = dict(batch=2, heads=4, kv_heads=2, d=64, max_pages=4, num_pages=9, window=16, sinks=0, dtype=BF16)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), INVALID), (dict(heads=3), INVALID), (dict(kv_heads=0), INVALID),
    (dict(window=0), INVALID), (dict(sinks=-1), INVALID), (dict(dtype=9), INVALID),
    (dict(sinks=129), UNSUPPORTED), (dict(d=256), UNSUPPORTED), (dict(dtype=F32), UNSUPPORTED),
    (dict(max_pages=1 << 26), UNSUPPORTED), (dict(q=None), INVALID), (dict(o=None), INVALID),
    (dict(table=None), INVALID), (dict(cache=None), INVALID), (dict(q=24), MISALIGNED),
    (dict(lengths=18), MISALIGNED), (dict(lse=18), MISALIGNED),
    (dict(max_pages=100000, num_pages=100000, window=10**6, ws=None), WORKSPACE),
    (dict(max_pages=100000, num_pages=100000, window=10**6, ws=272), WORKSPACE),
    (dict(max_pages=100000, num_pages=100000, window=10**6, ws_bytes=64), WORKSPACE),
    (dict(batch=0), NB_OK), (dict(heads=0), NB_OK)])
def test_decode_refusals(built_lib, kw, status):
    names = ["q", "cache", "table", "lengths", "o", "lse", "ws", "ws_bytes", *DEC]
    base = dict(DEC, q=16, cache=16, table=16, lengths=None, o=16, lse=None, ws=256, ws_bytes=1 << 40)
    assert call(built_lib.nb_attn_kv4_decode, names, base, kw) == status


def test_sizes(built_lib):
    assert [built_lib.nb_kv4_page_bytes(d) for d in (64, 128, 96, 0)] == [2560, 5120, 0, 0]
    size = built_lib.nb_attn_sink_bwd_workspace_size
    assert size(1, 2, 3, 64, 64, 8, 0, BF16) == 0       # 2 heads over 3
    assert size(0, 2, 1, 64, 64, 8, 0, BF16) == 0
    one = size(1, 8, 2, 4096, 128, 256, 0, BF16)
    assert one >= 2 * 8 * 4096 * 4                       # row statistics
    assert size(1, 8, 2, 4096, 128, 256, 4, BF16) > one  # parts of the sinks' tile
    need = built_lib.nb_attn_kv4_decode_workspace_size
    assert need(1, 4, 2, 64, 8, 256, 0, BF16) == 0       # one share
    assert need(1, 4, 3, 64, 8, 256, 0, BF16) == 0       # invalid
    assert need(1, 4, 1, 128, 32768, 1 << 20, 0, BF16) > 0


def test_layer_checks_arguments(built_lib):
    q, k = torch.zeros(1, 4, 8, 64), torch.zeros(1, 2, 8, 64)
    with pytest.raises(ValueError):
        layer.sink_attention(q, k, k[:, :1])
    with pytest.raises(ValueError):
        layer.sink_attention(q, torch.zeros(1, 2, 9, 64), torch.zeros(1, 2, 9, 64))
    with pytest.raises(TypeError):
        layer.sink_attention(q, k.double(), k.double())
    for bad in ((1, 1, 96, 8), (0, 1, 64, 8), (1, 0, 64, 8), (1, 1, 64, 0)):
        with pytest.raises(ValueError):
            layer.KV4Cache(*bad, device="cpu")
    c = layer.KV4Cache(2, 3, 64, 70, device="cpu")
    assert c.max_pages == 3 and c.block_table.tolist() == [[0, 1, 2], [3, 4, 5]]
    with pytest.raises(ValueError):
        c.append(torch.zeros(2, 2, 1, 64), torch.zeros(2, 2, 1, 64))
    with pytest.raises(ValueError):
        c.append(torch.zeros(2, 3, 1, 64), torch.zeros(2, 3, 2, 64))
    with pytest.raises(ValueError):
        c.attend(torch.zeros(2, 3, 1, 64))


# ------------------------------------------------------------------- oracles
@pytest.mark.parametrize("extension", [True, False])
def test_binding_takes_tensors_addresses_and_none(built_lib, extension, monkeypatch):
    """The new entry points through the extension module, and through ctypes where it is missing."""
    import sys

    import block_sparse_local_nb_b200 as nb
    from block_sparse_local_nb_b200 import binding

    monkeypatch.setattr(binding, "_entries", {})
    if extension:
        import os

        from block_sparse_local_nb_b200 import build

        if not os.path.exists(build.CALL):
            build._build_call()
    else:
        monkeypatch.setitem(sys.modules, "block_sparse_local_nb_b200._call", None)
        monkeypatch.delattr(sys.modules["block_sparse_local_nb_b200"], "_call", raising=False)
    t = torch.empty(64)
    kv = dict(stream=0, check=False)

    def write(k=t, starts=None, d=64, n=1, cache=t):
        return nb.nb_kv4_write(k, t, cache, t, starts, None, 1, 1, n, d, 4, 9, BF16, **kv)

    assert write(d=63) == UNSUPPORTED and write(n=0) == NB_OK
    assert write(k=None) == INVALID and write(cache=24) == MISALIGNED
    assert write(starts=t[1:].data_ptr() + 1) == MISALIGNED
    assert write(cache=2 ** 63 + 8) == MISALIGNED  # an address takes all 64 bits
    with pytest.raises(nb.NbError):
        nb.nb_kv4_read(t, t, None, None, t, t, 1, 1, 1, 32, 4, 9, BF16, stream=0)
    with pytest.raises((TypeError, AttributeError)):
        write(k="a tensor")
    with pytest.raises((TypeError, AttributeError)):
        write(d=64.0)
    assert nb.nb_attn_sink_fwd(t, t, t, t, None, None, 1, 2, 1, 8, 96, 4, 0, BF16, **kv) == UNSUPPORTED
    assert nb.nb_attn_sink_bwd(t, t, t, t, t, t, None, t, t, t, 256, 2 ** 40, 1, 3, 2, 8, 64, 4, 0,
                               BF16, **kv) == INVALID
    assert nb.nb_attn_kv4_decode(t, t, t, None, t, None, None, 0, 1, 2, 1, 64, 4, 9, 0, 0, BF16,
                                 **kv) == INVALID
    if extension:
        assert isinstance(binding._entries["nb_kv4_write"], type(len))
        with pytest.raises(OverflowError):
            write(n=2 ** 31)
        with pytest.raises(TypeError):
            binding._entry("nb_kv4_write")(t, t)


def draw(batch, heads, kv_heads, n, d, seed=0):
    g = np.random.default_rng(seed)
    return (g.standard_normal((batch, heads, n, d)), g.standard_normal((batch, kv_heads, n, d)),
            g.standard_normal((batch, kv_heads, n, d)), g.standard_normal((batch, heads, n, d)))


@pytest.mark.parametrize("sinks", [0, 7])
def test_sink_oracle_is_causal_attention_when_the_window_holds_everything(sinks):
    q, k, v, do = draw(2, 2, 2, 64, 8)
    lengths = [64, 41]
    o, lse = sink.fwd(q, k, v, 64, sinks, lengths)
    want, want_lse = attn_fwd_dense(q, k, v, 9, lengths, causal=True)
    assert np.allclose(o, want, atol=1e-12)
    assert np.allclose(lse[np.isfinite(lse)], want_lse[np.isfinite(want_lse)], atol=1e-12)
    for a, b in zip(sink.bwd(q, k, v, do, 64, sinks, lengths)[0],
                    attn_bwd_dense(q, k, v, do, 9, lengths, causal=True)):
        assert np.allclose(a, b, atol=1e-12)


def test_sink_oracle_rows_by_hand():
    q, k, v, _ = draw(1, 2, 1, 30, 8, 1)
    window, sinks, length = 5, 3, 27
    o, lse = sink.fwd(q, k, v, window, sinks, [length])
    for h in range(2):
        for i in range(30):
            see = [j for j in range(i + 1) if j < length and i < length and (i - j < window or j < sinks)]
            if not see:
                assert (o[0, h, i] == 0).all() and lse[0, h, i] == -np.inf
                continue
            e = np.array([np.exp(q[0, h, i] @ k[0, 0, j] / np.sqrt(8)) for j in see])
            assert np.allclose(o[0, h, i], sum(w * v[0, 0, j] for w, j in zip(e, see)) / e.sum(), atol=1e-12)
            assert np.isclose(lse[0, h, i], np.log(e.sum()), atol=1e-12)


def test_sink_oracle_gradients_against_differences():
    q, k, v, do = draw(1, 2, 1, 12, 4, 2)
    window, sinks, lengths = 4, 2, [11]
    (dq, dk, dv), _ = sink.bwd(q, k, v, do, window, sinks, lengths)

    def loss():
        return (sink.fwd(q, k, v, window, sinks, lengths)[0] * do)[:, :, :11].sum()

    for x, g in ((q, dq), (k, dk), (v, dv)):
        for i in np.ndindex(x.shape):
            keep, h = x[i], 1e-6
            x[i] = keep + h
            up = loss()
            x[i] = keep - h
            down = loss()
            x[i] = keep
            assert abs((up - down) / (2 * h) - g[i]) <= 1e-7, i


def test_layer_refuses_what_it_cannot_see_through():
    """Shapes and devices that would send the kernels past a buffer."""
    from block_sparse_local_nb_b200 import layer

    q, k = torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="lengths"):
        layer.sink_attention(q, k, k, torch.zeros(1, dtype=torch.int32), 4)
    with pytest.raises(ValueError):  # not on a GPU
        layer.sink_attention(q, k, k, torch.zeros(2, dtype=torch.int32), 4)
    with pytest.raises(ValueError):
        layer.sink_attention(q, k[:1], k[:1], None, 4)
    with pytest.raises(TypeError):
        layer.sink_attention(q, k.float(), k.float(), None, 4)
    c = layer.KV4Cache(2, 2, 64, 100, device="cpu")
    with pytest.raises(ValueError, match="device"):
        c.append(k.to("meta"), k.to("meta"))
    with pytest.raises(ValueError, match="k must be"):
        c.append(k[:, :1], k)
    with pytest.raises(ValueError, match="share"):
        c.append(k, k[:, :, :4])
    with pytest.raises(ValueError, match="counts"):
        c.append(k, k, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="starts"):
        c.read(4, starts=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="counts"):
        c.read(4, counts=torch.zeros(2, 1, dtype=torch.int32))
    with pytest.raises(ValueError, match="q must be"):
        c.attend(torch.zeros(1, 4, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="device"):
        c.attend(torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="meta"))
    for call in (lambda: c.append(k, k), lambda: c.read(4), lambda: c.attend(q[:, :, 0])):
        with pytest.raises(ValueError):  # a cache that is not on a GPU
            call()
    for args in ((0, 1, 64, 1), (1, 0, 64, 1), (1, 1, 96, 1), (1, 1, 64, 0)):
        with pytest.raises(ValueError):
            layer.KV4Cache(*args, device="cpu")


def test_layer_windows_past_32_bits_are_the_largest():
    from block_sparse_local_nb_b200 import layer

    assert layer._c_int(10**12) == 2**31 - 1 and layer._c_int(7) == 7
    assert layer._c_int(-10**12) == -2**31


def test_kv4_oracle_cells():
    """Every value is one of 16 equally spaced ones, at most half a step from x, and
    the extremes of the group fit."""
    g = np.random.default_rng(3)
    x = (g.standard_normal((50, 64)) * 10.0 ** g.integers(-3, 4, (50, 1))).astype(np.float32).astype(np.float64)
    code, step, mid = kv4.quantise(x)
    y = kv4.values(x)
    assert ((code >= 0) & (code <= 15)).all() and (code == np.floor(code)).all()
    assert (np.abs(y - x).reshape(50, 2, 32) <= step / 2).all()
    for p in (step, mid):  # held in bf16
        assert (p.astype(np.float32).view(np.uint32) & 0xffff == 0).all()
    # no smaller bf16 step would do, and the midpoint is the one below the centre
    lo, hi = x.reshape(50, 2, 32).min(-1, keepdims=True), x.reshape(50, 2, 32).max(-1, keepdims=True)
    below = (step.astype(np.float32).view(np.uint32) - 0x10000).view(np.float32).astype(np.float64)
    assert (7.5 * below < np.maximum(hi - mid, mid - lo)).all() and (mid <= (lo + hi) / 2).all()


def test_kv4_oracle_rounds_to_the_grid_of_bf16():
    x = np.array([2.0 ** -133 * 1.75, -2.0 ** -133 * 0.5, 2.0 ** -126 * 1.999, 1.0 - 2.0 ** -30, -1.0 - 2.0 ** -30])
    want = np.array([2.0 ** -133, -2.0 ** -133, 2.0 ** -126 * (2 - 2.0 ** -7), 1.0 - 2.0 ** -8, -1.0 - 2.0 ** -7])
    assert np.array_equal(kv4.bf16_floor(x), want)


def test_kv4_oracle_constant_groups_are_kept():
    x = np.repeat(np.array([0.0, -1.5, 3.140625])[:, None], 64, 1)
    assert (kv4.values(x) == x).all()


def test_decode_oracle_is_the_last_row_of_the_sink_oracle():
    q, k, v, _ = draw(2, 4, 2, 50, 8, 4)
    for window, sinks in ((7, 0), (7, 3), (100, 5)):
        o, lse = sink.fwd(q, k, v, window, sinks, [50, 33])
        last = np.stack([q[b, :, L - 1] for b, L in enumerate((50, 33))])
        got, got_lse = kv4.decode(last, k, v, [50, 33], window, sinks)
        for b, L in enumerate((50, 33)):
            assert np.allclose(got[b], o[b, :, L - 1], atol=1e-12)
            assert np.allclose(got_lse[b], lse[b, :, L - 1], atol=1e-12)
