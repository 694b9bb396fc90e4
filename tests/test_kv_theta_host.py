"""The rotation that an append makes of a theta, on the CPU: by its value at the call, whatever
kind of number it is."""
import numpy as np
import pytest
import torch

from decode_megakernel_sm_gb300 import KVCache, Rotary


@pytest.fixture
def cache():
    c = KVCache.__new__(KVCache)  # (its tensors would have to be CUDA ones)
    c.dim, c._index = 64, 0
    return c


def rotary(cache, theta):
    return cache._ex(theta, None, None, None, 1e-5)[0]


@pytest.mark.parametrize("held", [torch.tensor(1e4, dtype=torch.float64), np.array(1e4)], ids=["tensor", "array"])
def test_a_theta_that_changes(cache, held):
    assert rotary(cache, held).frequencies == Rotary(64, 1e4).frequencies
    held.fill_(5e5) if isinstance(held, torch.Tensor) else held.fill(5e5)
    assert rotary(cache, held).frequencies == Rotary(64, 5e5).frequencies


def test_equal_thetas_share_their_numbers(cache):
    assert rotary(cache, 10000) is rotary(cache, 1e4) and rotary(cache, np.float32(1e4)) is rotary(cache, 1e4)
    assert rotary(cache, 0) is None and rotary(cache, 0.0) is None
    for bad in (0.5, -1.0, float("nan"), 1e31):
        with pytest.raises(ValueError):
            rotary(cache, bad)


def test_frequencies_are_numbers():
    r = Rotary(64, torch.tensor(1e4, dtype=torch.float64), magnitude=np.float32(1.25))
    assert r.frequencies == Rotary(64, 1e4).frequencies and all(type(f) is float for f in r.frequencies)
    assert type(r.magnitude) is float
