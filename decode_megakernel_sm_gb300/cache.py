"""KVCache: one layer's KV cache with its operators -- append new tokens (rotated
on the way), attend with one new token per sequence (decode) or with many
(prefill).  Marshals torch CUDA tensors to the C ABI; no arithmetic here."""
from __future__ import annotations

import struct

import torch

from . import _lib as L

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
_empty = torch.empty
_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream

# The C structures as packed bytes, and the entry points that take them so.
_VIEW = struct.Struct("=QQiiiiQi4x")  # mk_kv_view
_BATCH = struct.Struct("=iiQQ")       # mk_kv_batch
_ROWS = struct.Struct("=Qqq")         # mk_rows
_entry = {}
_scratch = {}  # scratch bytes by device, operator and sizes


def _call(name):
    f = _entry[name] = L.packed(name)
    return f


class KVCache:
    """k, v: bf16 CUDA tensors.  With table (int32 [batch][stride], contiguous):
    pools [n_blocks][kv heads][block][head_dim], row p of sequence b in block
    table[b][p // block] at row p % block.  Without: [batch][kv heads][max_seq]
    [head_dim].  The tensors are used in place and kept alive.

    In every call, ``lens`` (int32 [batch]) is each sequence's number of cache
    rows, the new tokens' included, and ``cu`` (int32 [batch + 1]) the offsets of
    the sequences' new tokens in the rows of q, k, v and the outputs; cu None:
    one new token per sequence.  The new tokens are the last ones of their
    sequences.  Rows before cu[0] and from cu[batch] on are padding: not written,
    and what they hold has no effect.

    Calls run asynchronously on ``stream`` (default: the current one), allocate
    their scratch, and their outputs unless given, from torch's allocator, and
    may be captured into a CUDA graph.  Outputs carry no gradients.  What the
    kernels find in lens, cu and table (a length the cache cannot hold, offsets
    that fall, a block outside the pool) is kept for ``check``."""

    __slots__ = ("k", "v", "table", "device", "heads", "dim", "held", "_index", "_view", "_unusable",
                 "__weakref__")

    def __init__(self, k, v, table=None):
        shape, device = k.shape, k.device
        if len(shape) != 4 or v.shape != shape or k.dtype is not _BF16 or v.dtype is not _BF16 or \
                not k.is_cuda or v.device != device:
            raise ValueError("k, v: expected two 4-dimensional bf16 CUDA tensors of one shape")
        if not (k.is_contiguous() and v.is_contiguous()):
            raise ValueError("k, v: expected contiguous tensors")
        if k.requires_grad or v.requires_grad:
            raise ValueError("k, v: the cache operators have no backward pass")
        self.k, self.v, self.device, self._index = k, v, device, device.index
        self._read_as(table, shape)

    def _read_as(self, table, shape, unusable=None):
        """Read the tensors through `table` from now on; unusable: why they cannot be
        read so, for the calls to say."""
        n_blocks, self.heads, block, self.dim = shape
        self._unusable = unusable
        if unusable:
            self.table, self.held, self._view = None, -1, None
            return
        if table is None:
            self.held, tp, stride = n_blocks, 0, 0
        else:
            if table.dtype is not _I32 or table.dim() != 2 or table.device != self.device or \
                    not table.is_contiguous():
                raise ValueError("table: expected a contiguous int32 matrix on the cache's device")
            self.held, stride = table.shape
            tp = table.data_ptr()
        self.table = table
        self._view = _VIEW.pack(self.k.data_ptr(), self.v.data_ptr(), n_blocks, self.heads, block,
                                self.dim, tp, stride)

    # -- marshalling --------------------------------------------------------
    def _rows(self, t, name, dtype, n, heads):
        """mk_rows of t, which has to be [n][heads][dim] (None: any)."""
        try:
            a, b, c = t.shape
        except ValueError:
            a = b = c = -1
        if c != self.dim or t.dtype is not dtype or t.get_device() != self._index or \
                (n is not None and a != n) or (heads is not None and b != heads):
            raise ValueError(f"{name}: expected {dtype} [{'tokens' if n is None else n}]"
                             f"[{'heads' if heads is None else heads}][{self.dim}] on {self.device}")
        ts, hs, one = t.stride()
        if one != 1:
            raise ValueError(f"{name}: expected a dense last dimension")
        if t.requires_grad and torch.is_grad_enabled():
            raise ValueError(f"{name}: the cache operators have no backward pass")
        # the stride of a dimension of one means nothing
        return _ROWS.pack(t.data_ptr(), ts if a > 1 else 0, hs if b > 1 else 0)

    def _vector(self, t, name, n):
        if t.dtype is not _I32 or t.dim() != 1 or t.get_device() != self._index or \
                (n is not None and t.shape[0] != n) or not t.is_contiguous():
            raise ValueError(f"{name}: expected {'' if n is None else str(n) + ' '}contiguous int32 "
                             f"values on {self.device}")
        return t.data_ptr()

    def _batch(self, lens, cu, n):
        """(mk_kv_batch, batch)."""
        lp = self._vector(lens, "lens", None)
        batch = lens.shape[0]
        if batch > self.held:
            if self._unusable:
                raise ValueError(self._unusable)
            raise ValueError(f"lens: {batch} sequences in a cache of {self.held}")
        if cu is None:
            if n != batch:
                raise ValueError(f"{n} tokens for {batch} sequences: pass cu")
            return _BATCH.pack(batch, n, lp, 0), batch
        return _BATCH.pack(batch, n, lp, self._vector(cu, "cu", batch + 1)), batch

    def _on(self, stream, tensors, call, *args):
        """call(raw stream, *args) with the cache's device and `stream` current."""
        with torch.cuda.device(self.device):
            if stream is None:
                return call(_raw_stream(self._index), *args)
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(getattr(stream, "value", stream) or 0)
            if stream.device != self.device:
                raise ValueError(f"stream: expected one of {self.device}")
            for t in tensors:  # their memory is not reused before the stream is done with it
                if t is not None:
                    t.record_stream(stream)
            with torch.cuda.stream(stream):
                return call(stream.cuda_stream, *args)

    def _dense(self, n, heads):
        """A new bf16 [n][heads][dim] tensor and its mk_rows."""
        t = _empty((n, heads, self.dim), dtype=_BF16, device=self.device)
        return t, _ROWS.pack(t.data_ptr(), heads * self.dim, self.dim)

    # -- operators ----------------------------------------------------------
    def append(self, q, k, v, lens, cu=None, *, theta, q_out=None, stream=None):
        """Write the new tokens' keys and values into the cache, queries and keys
        rotated by their positions: the pair (t, t + head_dim / 2) by the angle
        position * theta^(-2t / head_dim); theta 0: no rotation.

        q [tokens][query heads][head_dim] (None: no queries), k and v [tokens]
        [kv heads][head_dim]: all bf16 or all float32, any token and head strides
        that keep rows on 16-byte boundaries.  Returns the rotated queries, bf16
        (q_out if given; it may be q itself)."""
        src = k.dtype
        if src is not _BF16 and src is not _F32:
            raise ValueError("k: expected bfloat16 or float32")
        kr = self._rows(k, "k", src, None, self.heads)
        n = k.shape[0]
        vr = self._rows(v, "v", src, n, self.heads)
        bt, _ = self._batch(lens, cu, n)
        hq, qr, given = 0, None, None
        if q is not None:
            qr, hq = self._rows(q, "q", src, n, None), q.shape[1]
            if q_out is not None:
                given = self._rows(q_out, "q_out", _BF16, n, hq)
        src = 1 if src is _F32 else 0  # MK_SRC_F32, MK_SRC_BF16
        if stream is None and _device() == self._index:
            return self._append(_raw_stream(self._index), bt, n, hq, qr, kr, vr, src, q_out, given,
                                theta)
        return self._on(stream, (q, k, v, lens, cu, q_out, self.k, self.v, self.table),
                        self._append, bt, n, hq, qr, kr, vr, src, q_out, given, theta)

    def _append(self, raw, bt, n, hq, qr, kr, vr, src, out, rows, theta):
        if qr is None:
            out = None
        elif rows is None:
            out, rows = self._dense(n, hq)
        status = (_entry.get("mk_kv_append") or _call("mk_kv_append"))(
            self._view, bt, hq, qr, kr, vr, src, rows, theta, raw)
        if status:
            raise L.MkError(status, "mk_kv_append")
        return out

    def _attend(self, decode, q, lens, cu, scale, out, return_lse, stream):
        qr = self._rows(q, "q", _BF16, None, None)
        n, hq, _ = q.shape
        bt, batch = self._batch(lens, cu, n)
        given = None if out is None else self._rows(out, "out", _BF16, n, hq)
        key = (self._index, decode, n, batch, hq, self.heads, self.dim)
        need = _scratch.get(key)
        if need is None:
            with torch.cuda.device(self.device):
                need = L.mk_attn_workspace_bytes(*key[1:])
            if len(_scratch) >= 1024:
                _scratch.clear()
            _scratch[key] = need
        name = "mk_attn_decode" if decode else "mk_attn_prefill"
        if scale is None:
            scale = self.dim ** -0.5
        if stream is None and _device() == self._index:
            return self._launch(_raw_stream(self._index), name, bt, n, hq, qr, scale, out, given,
                                return_lse, need)
        return self._on(stream, (q, lens, cu, out, self.k, self.v, self.table), self._launch,
                        name, bt, n, hq, qr, scale, out, given, return_lse, need)

    def _launch(self, raw, name, bt, n, hq, qr, scale, out, rows, return_lse, need):
        if rows is None:
            out, rows = self._dense(n, hq)
        ws = _empty(need, dtype=torch.uint8, device=self.device) if need else None
        lse = _empty((n, hq), dtype=_F32, device=self.device) if return_lse else None
        status = (_entry.get(name) or _call(name))(
            self._view, bt, hq, qr, scale, rows, lse.data_ptr() if return_lse else None,
            ws.data_ptr() if need else None, need, raw)
        if status:
            raise L.MkError(status, name)
        return (out, lse) if return_lse else out

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
        this device, of whichever cache, thread or stream, has run into a time limit
        (MK_ERR_TIMEOUT) or found bad contents (MK_ERR_INVALID_ARG) since the last
        check.  One check answers for all of them: a program with several users of a
        device checks in one place."""
        def call(raw):
            status = L.mk_kv_status(raw)
            if status != L.MK_OK:
                raise L.MkError(status, "KVCache")
        self._on(stream, (), call)
