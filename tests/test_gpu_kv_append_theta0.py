"""An append without a rotation leaves every number as it is: an infinity or a NaN of a head
reaches no other dim, in the plain append as in the general one."""
import math

import pytest
import torch

from decode_megakernel_sm_gb300 import Rotary
from tests.test_gpu_kv_append_ex import Fill
from tests.test_gpu_kv_ops import BF

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("src", [BF, torch.float32])
@pytest.mark.parametrize("how", [dict(theta=0), dict(rotary=Rotary(64, 1e4, dims=0))], ids=["theta", "rotary"])
@pytest.mark.parametrize("lens,new", [([100, 7], [100, 7]), ([900, 700], [900, 700])], ids=str)
def test_nothing_turns(src, how, lens, new):
    c = Fill((4, 2, 64), lens, new, seed=43)
    q, k, v = c.sources(src)
    for x in (q, k, v):
        x[3, 1, 40], x[4, 0, 0], x[5, 1, 63], x[6, 0, 7] = math.inf, -math.inf, math.nan, 3e38
    got = c.append(q, k, v, **how)
    tok, blk, row = c.places()
    for a, b in ((got, q), (c.k[blk, :, row], k[tok]), (c.v[blk, :, row], v[tok])):
        b = b.to(BF)
        assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(), b.nan_to_num())
    c.cache.check()
