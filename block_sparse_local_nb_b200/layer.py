"""Training-layer glue around the C ABI (argument marshalling and buffer
allocation only; every step of the computation runs in ``libnb_b200.so``).

* :func:`collate` is the page's "Dynamic Ceiling Hardware Alignment" data path
  (NucleoByte page, section 2 item 2): a batch of DNA strings becomes one
  int64 ``[batch, n_pad]`` matrix of model input IDs, ``n_pad`` the smallest
  multiple of 32 that holds the longest sequence's k-mer windows, plus the
  per-sequence window counts that the attention takes as ``lengths``.  One
  kernel (``nb_tokenize_batch``) tokenizes, offsets and pads on the device.
* :class:`BlockSparseLocalAttention` is the page's ``torch.autograd.Function``
  integration (section 4 "Tech Stack"): forward through ``nb_attn_fwd``
  (keeping the log-sum-exp), backward through ``nb_attn_bwd`` (P recomputed
  from it).  Tensors are ``[batch, heads, n, d]``; the backward needs bf16.
* :class:`SinkAttention` is the same for the causal attention with a sliding
  window of tokens and visible first tokens (``nb_attn_sink_fwd`` and
  ``nb_attn_sink_bwd``), with key/value heads that query heads may share.
* :class:`KV4Cache` serves such a model token by token: a 4-bit key/value cache
  (``nb_kv4_write``, ``nb_kv4_read``) and the single-token form of the attention
  over it (``nb_attn_kv4_decode``).
"""

from __future__ import annotations

from typing import Sequence

import numpy as np
import torch

from . import binding as nb

BLOCK = 32
PAD_ID = 0


def ceiling_layout(base_counts: Sequence[int], k: int = 6) -> tuple[np.ndarray, int]:
    """Offsets (int64 [batch + 1]) of the concatenated sequences and the
    dynamic ceiling n_pad (computed by the library's nb_batch_ceiling) for
    sequences of the given base counts."""
    counts = np.asarray([int(c) for c in base_counts], dtype=np.int64)
    if (counts < 0).any():
        raise ValueError("base counts must be non-negative")
    offsets = np.zeros(counts.size + 1, dtype=np.int64)
    np.cumsum(counts, out=offsets[1:])
    return offsets, nb.nb_batch_ceiling(offsets, counts.size, k)


def collate(seqs: Sequence[bytes], k: int = 6, device=None, stream=None):
    """Model input IDs and lengths of a batch of DNA byte strings, on the device.

    Returns ``(input_ids, lengths)``: int64 ``[batch, n_pad]`` with ID 0 for
    padding, raw k-mer ID + 1 for a window of A/C/G/T and 4**k + 1 for a window
    holding any other byte; int32 ``[batch]`` window counts.  Asynchronous on
    ``stream`` (default: the current stream).
    """
    device = torch.device(device if device is not None else "cuda")
    offsets, n_pad = ceiling_layout([len(s) for s in seqs], k)
    blob = b"".join(bytes(s) for s in seqs)
    host = torch.frombuffer(bytearray(blob or b"\0"), dtype=torch.uint8).pin_memory()
    host_off = torch.from_numpy(offsets).pin_memory()
    s = stream if stream is not None else torch.cuda.current_stream(device)
    with torch.cuda.stream(s):
        dev_blob = host.to(device, non_blocking=True)
        dev_off = host_off.to(device, non_blocking=True)
        ids = torch.empty((len(seqs), n_pad), dtype=torch.int64, device=device)
        lengths = torch.empty(len(seqs), dtype=torch.int32, device=device)
    nb.nb_tokenize_batch(dev_blob, dev_off, len(seqs), k, ids, lengths, n_pad, s)
    return ids, lengths


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return nb.NB_BF16
    if t.dtype == torch.float32:
        return nb.NB_F32
    raise TypeError(f"unsupported dtype {t.dtype} (bf16 or fp32)")


class BlockSparseLocalAttention(torch.autograd.Function):
    """O = softmax(Q K^T / sqrt(d) restricted to the band |i - j| <= R of
    32-token blocks and to keys < lengths[b]) V, with its backward.  With
    ``causal`` the band is i - R <= j <= i and keys k <= q."""

    @staticmethod
    def forward(ctx, q, k, v, lengths, R: int, causal: bool = False):
        if not (q.shape == k.shape == v.shape and q.dim() == 4):
            raise ValueError("q, k, v must share one [batch, heads, n, d] shape")
        if not (q.dtype == k.dtype == v.dtype):
            raise TypeError("q, k, v must share one dtype")
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
        batch, heads, n, d = q.shape
        if lengths is not None:
            lengths = lengths.to(device=q.device, dtype=torch.int32).contiguous()
        o = torch.empty_like(q)
        lse = torch.empty((batch, heads, n), dtype=torch.float32, device=q.device)
        fwd = nb.nb_attn_fwd_causal if causal else nb.nb_attn_fwd
        fwd(q, k, v, o, lse, lengths, batch, heads, n, d, R, _dtype_code(q),
            torch.cuda.current_stream(q.device))
        ctx.save_for_backward(q, k, v, o, lse, lengths)
        ctx.R = R
        ctx.causal = causal
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse, lengths = ctx.saved_tensors
        batch, heads, n, d = q.shape
        do = do.to(q.dtype).contiguous()
        code = _dtype_code(q)
        ws_bytes = nb.attn_bwd_workspace_size(batch, heads, n, d, code)
        ws = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        bwd = nb.nb_attn_bwd_causal if ctx.causal else nb.nb_attn_bwd
        bwd(q, k, v, o, do, lse, lengths, dq, dk, dv, ws, ws_bytes, batch, heads, n, d, ctx.R, code,
            torch.cuda.current_stream(q.device))
        return dq, dk, dv, None, None, None


def block_sparse_local_attention(q, k, v, lengths=None, R: int = 1, causal: bool = False):
    """Differentiable banded block-sparse local attention (see the class)."""
    return BlockSparseLocalAttention.apply(q, k, v, lengths, R, causal)


def _dense(x):
    """x contiguous and 16-byte aligned, as the library takes it (a gradient or a cache row
    may be a contiguous view at an odd offset): itself, or a copy."""
    x = x.contiguous()
    return x if x.data_ptr() % 16 == 0 else x.clone()


def _c_int(x) -> int:
    """A Python integer as the library's 32-bit one: the nearest (a window or sinks
    beyond it mean the same, or are refused all the same)."""
    return max(-2**31, min(int(x), 2**31 - 1))


class SinkAttention(torch.autograd.Function):
    """O = softmax(Q K^T / sqrt(d)) V where query q sees key k when k <= q,
    k < lengths[b] and (q - k < window or k < sinks), with its backward.  q is
    [batch, heads, n, d], k and v [batch, kv_heads, n, d]; query head h reads
    key/value head h // (heads // kv_heads).

    A pass may be captured into a graph; its backward with ``torch.autograd.grad``, or
    with leaves that no earlier graph still holds (torch adds a leaf's gradient on
    the stream of the graph that lives, outside of the capture)."""

    @staticmethod
    def forward(ctx, q, k, v, lengths, window: int, sinks: int = 0):
        if q.dim() != 4 or k.shape != v.shape or k.dim() != 4:
            raise ValueError("q must be [batch, heads, n, d], k and v [batch, kv_heads, n, d]")
        batch, heads, n, d = q.shape
        if k.shape[0] != batch or k.shape[2:] != q.shape[2:]:
            raise ValueError("q, k, v must share batch, n and d")
        if not (q.dtype == k.dtype == v.dtype):
            raise TypeError("q, k, v must share one dtype")
        if not (q.device == k.device == v.device):
            raise ValueError("q, k, v must be on one device")
        window, sinks = _c_int(window), _c_int(sinks)
        q, k, v = _dense(q), _dense(k), _dense(v)
        if lengths is not None:
            if lengths.shape != (batch,):
                raise ValueError("lengths must be [batch]")
            lengths = lengths.to(device=q.device, dtype=torch.int32).contiguous()
        o = torch.empty_like(q)
        lse = torch.empty((batch, heads, n), dtype=torch.float32, device=q.device)
        with torch.cuda.device(q.device):
            nb.nb_attn_sink_fwd(q, k, v, o, lse, lengths, batch, heads, k.shape[1], n, d, window,
                                sinks, _dtype_code(q), torch.cuda.current_stream(q.device))
        ctx.save_for_backward(q, k, v, o, lse, lengths)
        ctx.window, ctx.sinks = window, sinks
        return o

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse, lengths = ctx.saved_tensors
        batch, heads, n, d = q.shape
        do = _dense(do.to(q.dtype))
        shape = (batch, heads, k.shape[1], n, d, ctx.window, ctx.sinks, _dtype_code(q))
        ws_bytes = nb.attn_sink_bwd_workspace_size(*shape)
        ws = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=q.device)
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        with torch.cuda.device(q.device):
            nb.nb_attn_sink_bwd(q, k, v, o, do, lse, lengths, dq, dk, dv, ws, ws_bytes, *shape,
                                torch.cuda.current_stream(q.device))
        return dq, dk, dv, None, None, None


def sink_attention(q, k, v, lengths=None, window: int = 1, sinks: int = 0):
    """Differentiable causal attention with a sliding window of tokens and visible
    first tokens (see :class:`SinkAttention`)."""
    return SinkAttention.apply(q, k, v, lengths, window, sinks)


class KV4Cache:
    """The 4-bit keys and values of a batch of sequences.

    ``max_tokens`` bounds a sequence; its pages are taken from the pool in order,
    so the block table is fixed.  ``lengths`` (int32 [batch], on the device) counts
    the tokens of each sequence; ``append`` adds to it on the current stream, so a
    captured step can be replayed.
    """

    def __init__(self, batch: int, kv_heads: int, d: int, max_tokens: int, device="cuda"):
        page_bytes = nb.kv4_page_bytes(d)
        if page_bytes == 0:
            raise ValueError("d must be 64 or 128")
        if batch < 1 or kv_heads < 1 or max_tokens < 1:
            raise ValueError("batch, kv_heads and max_tokens must be positive")
        self.batch, self.kv_heads, self.d = batch, kv_heads, d
        self.max_pages = -(-max_tokens // BLOCK)
        self.num_pages = batch * self.max_pages
        self.pool = torch.zeros((self.num_pages, kv_heads, page_bytes), dtype=torch.uint8,
                                device=device)
        self.device = self.pool.device  # with its index, whatever the current device is later
        self.block_table = torch.arange(self.num_pages, dtype=torch.int32,
                                        device=self.device).reshape(batch, self.max_pages)
        self.lengths = torch.zeros(batch, dtype=torch.int32, device=self.device)

    def _rows(self, x, name):
        if x.dim() != 4 or x.shape[0] != self.batch or x.shape[1] != self.kv_heads or x.shape[3] != self.d:
            raise ValueError(f"{name} must be [{self.batch}, {self.kv_heads}, n, {self.d}]")
        if x.device != self.device:
            raise ValueError(f"{name} must be on the cache's device, {self.device}")
        return _dense(x)

    def _per_sequence(self, x, name):
        if x.shape != (self.batch,):
            raise ValueError(f"{name} must be [{self.batch}]")
        return x.to(device=self.device, dtype=torch.int32).contiguous()

    def append(self, k, v, counts=None):
        """Quantise the first ``counts[b]`` (default: all n) tokens of k, v
        [batch, kv_heads, n, d] behind those of sequence b.  Tokens past the
        cache's end are dropped and reported by nb_kernel_error."""
        k, v = self._rows(k, "k"), self._rows(v, "v")
        if k.shape != v.shape or k.dtype != v.dtype:
            raise ValueError("k and v must share shape and dtype")
        n = k.shape[2]
        if counts is not None:
            counts = self._per_sequence(counts, "counts").clamp(0, n)
        with torch.cuda.device(self.device):
            nb.nb_kv4_write(k, v, self.pool, self.block_table, self.lengths, counts, self.batch,
                            self.kv_heads, n, self.d, self.max_pages, self.num_pages,
                            _dtype_code(k), torch.cuda.current_stream(self.device))
            self.lengths.add_(n if counts is None else counts)

    def read(self, n: int, starts=None, counts=None, dtype=torch.bfloat16):
        """Tokens starts[b] .. starts[b] + n - 1 (default: from 0) as the cache holds
        them, (k, v) [batch, kv_heads, n, d]; rows past counts[b] (default: the tokens
        that the cache has from there) are 0."""
        if starts is None:
            starts = torch.zeros_like(self.lengths)
        starts = self._per_sequence(starts, "starts")
        if counts is None:
            counts = (self.lengths.clamp(max=self.max_pages * BLOCK) - starts).clamp(0, n)
        counts = self._per_sequence(counts, "counts")
        k = torch.empty((self.batch, self.kv_heads, n, self.d), dtype=dtype, device=self.device)
        v = torch.empty_like(k)
        with torch.cuda.device(self.device):
            nb.nb_kv4_read(self.pool, self.block_table, starts, counts, k, v, self.batch,
                           self.kv_heads, n, self.d, self.max_pages, self.num_pages,
                           _dtype_code(k), torch.cuda.current_stream(self.device))
        return k, v

    def attend(self, q, window: int = 2**31 - 1, sinks: int = 0):
        """Attention of each sequence's last token, q [batch, heads, d] bf16, over its
        window of tokens and its first ``sinks``; [batch, heads, d]."""
        if q.dim() != 3 or q.shape[0] != self.batch or q.shape[2] != self.d:
            raise ValueError(f"q must be [{self.batch}, heads, {self.d}]")
        if q.device != self.device:
            raise ValueError(f"q must be on the cache's device, {self.device}")
        window, sinks = _c_int(window), _c_int(sinks)
        q = _dense(q)
        heads, code = q.shape[1], _dtype_code(q)
        o = torch.empty_like(q)
        size = nb.attn_kv4_decode_workspace_size(self.batch, heads, self.kv_heads, self.d,
                                                 self.max_pages, window, sinks, code)
        ws = torch.empty(size, dtype=torch.uint8, device=self.device) if size else None
        with torch.cuda.device(self.device):
            nb.nb_attn_kv4_decode(q, self.pool, self.block_table, self.lengths, o, None, ws, size,
                                  self.batch, heads, self.kv_heads, self.d, self.max_pages,
                                  self.num_pages, window, sinks, code,
                                  torch.cuda.current_stream(self.device))
        return o
