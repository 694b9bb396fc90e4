"""A Rotary is what it was made of: its calls read numbers packed then, so it refuses others."""
import pytest

from decode_megakernel_sm_gb300 import Rotary


@pytest.mark.parametrize("name,value", [("head_dim", 128), ("dims", 32), ("interleaved", True), ("magnitude", 2.0),
                                        ("frequencies", (0.1,) * 32), ("theta", 5e5)])
def test_assignments_are_refused(name, value):
    r = Rotary(64, 1e4)
    with pytest.raises(AttributeError):
        setattr(r, name, value)
    if name != "theta":
        with pytest.raises(AttributeError):
            delattr(r, name)
    assert (r.head_dim, r.dims, r.interleaved, r.magnitude) == (64, 64, False, 1.0)
    assert r.frequencies == Rotary(64, 1e4).frequencies
