"""What Decoder.cache hands out, on the CPU: the handle is a stand-in, and nothing is
launched."""
import types
import weakref

import pytest
import torch

from decode_megakernel_sm_gb300 import decoder
from decode_megakernel_sm_gb300.decoder import Decoder


class View:
    """Stands for KVCache, which wants CUDA tensors."""

    def __init__(self, k, v, table=None):
        self.k, self.v, self.table, self.why = k, v, table, None

    def _read_as(self, table, shape, why=None):
        assert shape == self.k.shape
        self.table, self.why = table, why


@pytest.fixture
def make(monkeypatch):
    monkeypatch.setattr(decoder, "KVCache", View)
    monkeypatch.setattr(decoder.L, "mk_set_kv_pages", lambda *a: None)
    monkeypatch.setattr(decoder, "_ptr", lambda t, dtype=None: 0)

    def make(shape):
        d = Decoder.__new__(Decoder)
        d.desc = types.SimpleNamespace(max_batch=2, max_seq=64, n_kv_heads=4, head_dim=64)
        d.kcache, d.vcache = ([torch.zeros(shape, dtype=torch.bfloat16)] * 2 for _ in range(2))
        d.h, d._kv_block, d._kv_table, d._views = None, 0, None, weakref.WeakSet()
        return d
    return make


TABLE = torch.zeros(2, 4, dtype=torch.int32)


def test_pools_are_no_contiguous_cache(make):
    dec = make((9, 4, 16, 64))
    with pytest.raises(ValueError, match="set_kv_pages first"):
        dec.cache(0)
    dec.set_kv_pages(16, TABLE)
    assert dec.cache(1).table is TABLE


@pytest.mark.parametrize("shape", [(1, 4, 64, 64), (2, 4, 63, 64), (2, 2, 64, 64), (2, 4, 64, 128),
                                   (2, 4, 4096)], ids=str)
def test_other_shapes_are_refused(make, shape):
    with pytest.raises(ValueError):
        make(shape).cache(0)


def test_contiguous(make):
    assert make((2, 4, 64, 64)).cache(0).table is None
    assert make((3, 4, 64, 64)).cache(1).table is None


def test_blocks_of_another_size_than_the_tensors(make):
    dec = make((9, 4, 16, 64))
    dec.set_kv_pages(32, TABLE)
    with pytest.raises(ValueError, match="32"):
        dec.cache(0)


def test_views_follow_the_handle(make):
    dec = make((9, 4, 64, 64))
    view = dec.cache(0)
    dec.set_kv_pages(64, TABLE)
    assert view.table is TABLE and view.why is None
    other = TABLE.clone()
    dec.set_kv_pages(64, other)
    assert view.table is other and view.why is None
    dec.set_kv_pages(0, None)
    assert view.table is None and view.why is None
    dec.set_kv_pages(16, TABLE)
    assert "[16]" in view.why
    del view
    assert not len(dec._views)
