"""Copies of a KVCache: a shallow one reads the same tensors, a deep or unpickled one its own."""
import copy
import pickle

import pytest
import torch

from decode_megakernel_sm_gb300 import Rotary
from tests.test_gpu_kv_append_ex import Fill
from tests.test_gpu_kv_int8 import Case8
from tests.test_gpu_kv_ops import Case

pytestmark = pytest.mark.gpu


def tensors(cache):
    return [t for t in (cache.k, cache.v, cache.table) + (cache.scales or ()) if t is not None]


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("block", [0, 16])
@pytest.mark.parametrize("again", [copy.copy, copy.deepcopy, lambda c: pickle.loads(pickle.dumps(c))],
                         ids=["copy", "deepcopy", "pickle"])
def test_copies(bits, block, again):
    c = (Case8 if bits == 8 else Case)((8, 2, 64), [300, 70], [1, 1], block=block, seed=40)
    want = c.cache.decode(c.q, c.lens)
    other = again(c.cache)
    mine = [x.data_ptr() == y.data_ptr() for x, y in zip(tensors(other), tensors(c.cache))]
    assert len(mine) == 2 + bool(block) + 2 * (bits == 8) and all(m == (again is copy.copy) for m in mine)
    assert torch.equal(other.decode(c.q, c.lens), want)
    # what becomes of the original's rows
    for t in (c.cache.k, c.cache.v):
        t.zero_()
    zeros = torch.zeros_like(want)
    assert torch.equal(other.decode(c.q, c.lens), zeros if again is copy.copy else want)
    assert torch.equal(c.cache.decode(c.q, c.lens), zeros)
    c.cache.check()


@pytest.mark.parametrize("bits", [16, 8])
def test_a_deep_copy_is_written_alone(bits):
    c = Fill((4, 2, 64), [50, 20], [20, 20], bits, seed=41)
    q, k, v = c.sources(torch.bfloat16)
    was = [t.clone() for t in tensors(c.cache)]
    other = copy.deepcopy(c.cache)
    got = other.append(q, k, v, c.lens, c.cu, rotary=copy.deepcopy(Rotary(64, 1e4)))
    assert all(torch.equal(x, y) for x, y in zip(tensors(c.cache), was))
    assert torch.equal(c.append(q, k, v, rotary=Rotary(64, 1e4)), got)
    assert all(torch.equal(x, y) for x, y in zip(tensors(c.cache), tensors(other)))
    c.cache.check()


def test_a_view_that_cannot_be_read_stays_so():
    c = Case((8, 2, 64), [300, 70], [1, 1], block=16, seed=42)
    c.cache._read_as(None, c.cache.k.shape, "why not")
    for again in (copy.copy, copy.deepcopy):
        with pytest.raises(ValueError, match="why not"):
            again(c.cache).decode(c.q, c.lens)
