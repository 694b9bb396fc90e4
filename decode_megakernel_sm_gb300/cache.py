"""KVCache: one layer's KV cache with its operators -- append new tokens (rotated
on the way), attend with one new token per sequence (decode) or with many
(prefill).  Marshals torch CUDA tensors to the C ABI; no arithmetic here."""
from __future__ import annotations

import math

import torch

from . import _lib as L

_BF16 = torch.bfloat16


def _index(t, name, n, device):
    """A dense int32 vector of n entries on the cache's device, as a pointer."""
    if t.dtype != torch.int32 or t.dim() != 1 or t.shape[0] != n or t.device != device or \
            not t.is_contiguous():
        raise ValueError(f"{name}: expected {n} contiguous int32 values on {device}")
    return t.data_ptr()


class KVCache:
    """k, v: bf16 CUDA tensors.  With table (int32 [batch][stride], contiguous):
    pools [n_blocks][kv heads][block][head_dim], row p of sequence b in block
    table[b][p // block] at row p % block.  Without: [batch][kv heads][max_seq]
    [head_dim].  The tensors are used in place and kept alive.

    In every call, ``lens`` (int32 [batch]) is each sequence's number of cache
    rows, the new tokens' included, and ``cu`` (int32 [batch + 1]) the offsets of
    the sequences' new tokens in the rows of q, k, v and the outputs; cu None:
    one new token per sequence.  The new tokens are the last ones of their
    sequences.  Rows from cu[batch] on are padding, neither read nor written.

    Calls run asynchronously on ``stream`` (default: the current one), allocate
    their scratch, and their outputs unless given, from torch's allocator, and
    may be captured into a CUDA graph.  Outputs carry no gradients.  What the
    kernels find in lens, cu and table (a length the cache cannot hold, a block
    outside the pool) is kept for ``check``."""

    __slots__ = ("k", "v", "table", "device", "_view", "_ws")

    def __init__(self, k, v, table=None):
        if k.dim() != 4 or k.shape != v.shape or k.dtype != _BF16 or v.dtype != _BF16 or \
                not k.is_cuda or v.device != k.device:
            raise ValueError("k, v: expected two 4-dimensional bf16 CUDA tensors of one shape")
        if not (k.is_contiguous() and v.is_contiguous()):
            raise ValueError("k, v: expected contiguous tensors")
        self.k, self.v, self.table, self.device = k, v, table, k.device
        n_blocks, heads, block, dim = k.shape
        if table is None:
            tp, stride = None, 0
        else:
            if table.dtype != torch.int32 or table.dim() != 2 or table.device != k.device or \
                    not table.is_contiguous():
                raise ValueError("table: expected a contiguous int32 matrix on the cache's device")
            tp, stride = table.data_ptr(), table.shape[1]
        self._view = L.mk_kv_view(k.data_ptr(), v.data_ptr(), n_blocks, heads, block, dim, tp,
                                  stride)
        self._ws = {}

    # -- marshalling --------------------------------------------------------
    def _rows(self, t, name, dtype, n=None, heads=None):
        s = t.shape
        if len(s) != 3 or t.dtype != dtype or t.device != self.device or \
                s[2] != self._view.head_dim or t.stride(2) != 1 or \
                (n is not None and s[0] != n) or (heads is not None and s[1] != heads):
            raise ValueError(f"{name}: expected {dtype} [{'tokens' if n is None else n}]"
                             f"[{'heads' if heads is None else heads}][{self._view.head_dim}] on "
                             f"{self.device}, dense in the last dimension")
        if t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name}: the cache operators have no backward pass")
        # the stride of a dimension of one means nothing
        return L.mk_rows(t.data_ptr(), t.stride(0) if s[0] > 1 else 0,
                         t.stride(1) if s[1] > 1 else 0)

    def _batch(self, lens, cu, n):
        batch = lens.shape[0] if lens.dim() == 1 else -1
        held = self.k.shape[0] if self.table is None else self.table.shape[0]
        if batch > held:
            raise ValueError(f"lens: {batch} sequences in a cache of {held}")
        lp = _index(lens, "lens", batch, self.device)
        if cu is None:
            if n != batch:
                raise ValueError(f"{n} tokens for {batch} sequences: pass cu")
            return L.mk_kv_batch(batch, n, lp, None)
        return L.mk_kv_batch(batch, n, lp, _index(cu, "cu", batch + 1, self.device))

    def _on(self, stream, tensors, call):
        """call(raw stream) with the cache's device and `stream` current."""
        if stream is None and torch.cuda.current_device() == self.device.index:
            return call(torch.cuda.current_stream().cuda_stream)
        with torch.cuda.device(self.device):
            if stream is None:
                return call(torch.cuda.current_stream().cuda_stream)
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(getattr(stream, "value", stream) or 0)
            for t in tensors:  # their memory is not reused before the stream is done with it
                if t is not None:
                    t.record_stream(stream)
            with torch.cuda.stream(stream):
                return call(stream.cuda_stream)

    # -- operators ----------------------------------------------------------
    def append(self, q, k, v, lens, cu=None, *, theta, q_out=None, stream=None):
        """Write the new tokens' keys and values into the cache, queries and keys
        rotated by their positions: the pair (t, t + head_dim / 2) by the angle
        position * theta^(-2t / head_dim); theta 0: no rotation.

        q [tokens][query heads][head_dim] (None: no queries), k and v [tokens]
        [kv heads][head_dim]: all bf16 or all float32, any token and head strides
        that keep rows on 16-byte boundaries.  Returns the rotated queries, bf16
        (q_out if given; it may be q itself)."""
        view, heads = self._view, self._view.n_kv_heads
        n, src = k.shape[0], k.dtype
        if src is not _BF16 and src is not torch.float32:
            raise ValueError("k: expected bf16 or float32")
        kr, vr = self._rows(k, "k", src, None, heads), self._rows(v, "v", src, n, heads)
        bt = self._batch(lens, cu, n)
        hq, qr = 0, None
        if q is not None:
            qr, hq = self._rows(q, "q", src, n), q.shape[1]
            given = None if q_out is None else self._rows(q_out, "q_out", _BF16, n, hq)
        code = L.MK_SRC_F32 if src is torch.float32 else L.MK_SRC_BF16

        def call(raw):
            out, rows = q_out, None
            if q is not None:
                rows = given
                if rows is None:
                    out = torch.empty(q.shape, dtype=_BF16, device=self.device)
                    rows = L.mk_rows(out.data_ptr(), hq * view.head_dim, view.head_dim)
            L.mk_kv_append(view, bt, hq, qr, kr, vr, code, rows, theta, raw)
            return out

        return self._on(stream, (q, k, v, lens, cu, q_out, self.k, self.v, self.table), call)

    def _attend(self, decode, q, lens, cu, scale, out, return_lse, stream):
        view = self._view
        qr = self._rows(q, "q", _BF16)
        n, hq = q.shape[0], q.shape[1]
        bt = self._batch(lens, cu, n)
        given = None if out is None else self._rows(out, "out", _BF16, n, hq)
        if scale is None:
            scale = 1.0 / math.sqrt(view.head_dim)
        key = (decode, n, bt.batch, hq)
        need = self._ws.get(key)
        if need is None:
            need = L.mk_attn_workspace_bytes(decode, n, bt.batch, hq, view.n_kv_heads,
                                             view.head_dim)
            if len(self._ws) > 64:
                self._ws.clear()
            self._ws[key] = need

        def call(raw):
            o, rows = out, given
            if rows is None:
                o = torch.empty(q.shape, dtype=_BF16, device=self.device)
                rows = L.mk_rows(o.data_ptr(), hq * view.head_dim, view.head_dim)
            lse = torch.empty((n, hq), dtype=torch.float32, device=self.device) \
                if return_lse else None
            ws = torch.empty(need, dtype=torch.uint8, device=self.device) if need else None
            (L.mk_attn_decode if decode else L.mk_attn_prefill)(
                view, bt, hq, qr, scale, rows, lse.data_ptr() if return_lse else None,
                ws.data_ptr() if need else None, need, raw)
            return (o, lse) if return_lse else o

        return self._on(stream, (q, lens, cu, out, self.k, self.v, self.table), call)

    def decode(self, q, lens, *, scale=None, out=None, return_lse=False, stream=None):
        """Attention of one new token per sequence, q [batch][query heads][head_dim]
        (bf16, rotated), over all lens[b] rows of its sequence: softmax(scale q k^T) v
        with scale 1 / sqrt(head_dim) unless given; an empty sequence gives zeros.
        Returns out (bf16, q's shape), with return_lse also the logarithm of each
        row's sum of exponentials, float32 [batch][query heads] (-inf if empty)."""
        return self._attend(True, q, lens, None, scale, out, return_lse, stream)

    def prefill(self, q, lens, cu, *, scale=None, out=None, return_lse=False, stream=None):
        """As decode, for any number of new tokens per sequence: the token at position
        p attends to rows [0, p]."""
        if cu is None:
            raise ValueError("cu: expected the offsets of the new tokens")
        return self._attend(False, q, lens, cu, scale, out, return_lse, stream)

    def check(self, stream=None):
        """Wait for the stream and raise MkError if a kernel of any cache operator on
        this device has found bad contents (or run into a time limit) since the last
        check."""
        def call(raw):
            status = L.mk_kv_status(raw)
            if status != L.MK_OK:
                raise L.MkError(status, "KVCache")
        self._on(stream, (), call)
