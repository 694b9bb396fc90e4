"""Copies of a Rotary stand on their own: what a call reads of them is theirs."""
import copy
import ctypes as C
import pickle

import pytest

from decode_megakernel_sm_gb300 import Rotary
from decode_megakernel_sm_gb300 import _lib as L

FORMS = [Rotary(64, 1e4), Rotary(128, 5e5, dims=64, interleaved=True, factor=8, trained=8192, magnitude=1.25),
         Rotary(64, frequencies=[0.5 - 0.01 * t for t in range(8)], dims=16), Rotary(64, 1e4, dims=0)]


@pytest.mark.parametrize("again", [copy.copy, copy.deepcopy, lambda r: pickle.loads(pickle.dumps(r))],
                         ids=["copy", "deepcopy", "pickle"])
@pytest.mark.parametrize("form", range(len(FORMS)))
def test_copies(form, again):
    r = FORMS[form]
    other = again(r)
    for name in ("head_dim", "dims", "interleaved", "magnitude", "frequencies"):
        assert getattr(other, name) == getattr(r, name)
    a, b = (L.mk_rotary.from_buffer_copy(x._packed) for x in (r, other))
    assert (b.dims, b.interleaved, b.magnitude) == (a.dims, a.interleaved, a.magnitude)
    # the frequencies that the call reads are those that the copy keeps alive
    assert b.freq == (C.addressof(other._held) if r.dims else None)
    assert list(other._held) == list(r.frequencies)
