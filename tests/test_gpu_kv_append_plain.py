"""The general append beside the plain one, on a bf16 cache without norms.

Both turn in fp32 and are off by at most e = 2^-20 of the pair's norm (test_gpu_kv_ops), then round
once, by at most 2^-8 of what they round: with x the 64-bit result they are within
2 (e + 2^-8 (|x| + e)) of one another, for which 2^-7 |x| and 2^-18 of the norm are allowed.
Values do not turn: equal."""
import pytest
import torch

from decode_megakernel_sm_gb300 import Rotary
from tests.test_gpu_kv_append_ex import Fill, made
from tests.test_gpu_kv_ops import BF

pytestmark = pytest.mark.gpu


def norms(x):
    """Of each element's pair, halves."""
    a, b = x.double().chunk(2, -1)
    return torch.hypot(a, b).repeat(1, 1, 2)


@pytest.mark.parametrize("src", [BF, torch.float32])
@pytest.mark.parametrize("heads,lens,new", [((8, 2, 64), [500, 70], [300, 70]), ((16, 4, 128), [900, 64, 1], [640, 33, 1]),
                                            ((6, 3, 128), [40_000], [100])], ids=str)
def test_the_general_append_gives_what_the_plain_one_does(heads, lens, new, src):
    c = Fill(heads, lens, new, seed=5)
    q, k, v = c.sources(src)
    plain = c.append(q, k, v, theta=5e5)
    was = c.k.clone(), c.v.clone()
    c.k.fill_(0.5), c.v.fill_(0.5)
    rotary = Rotary(c.d, 5e5)
    general = c.append(q, k, v, rotary=rotary)
    tok, blk, row = c.places()
    assert torch.equal(c.v[blk, :, row], was[1][blk, :, row])
    for a, b, x in ((general, plain, q), (c.k[blk, :, row], was[0][blk, :, row], k[tok])):
        want = made(x, c.positions() if x is q else c.positions()[tok], rotary, None, 0)[0]
        off = (a.double() - b.double()).abs()
        assert (off <= 2.0 ** -7 * want.abs() + 2.0 ** -18 * norms(x)).all()
    c.cache.check()
