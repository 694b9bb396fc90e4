"""Offsets that fall or leave the rows are reported by every cache operator, also where
no token belongs to the sequence that has them."""
import pytest
import torch

from decode_megakernel_sm_gb300 import MK_ERR_INVALID_ARG, MkError
from tests.test_gpu_kv_ops import BF, Case

pytestmark = pytest.mark.gpu


def offsets(n, batch):
    """Bad offsets of `batch` sequences over n rows: name -> cu."""
    rise = [n * i // batch for i in range(batch + 1)]
    return {
        "first falls": [n // 2, 0] + rise[2:],
        "first is negative, and empty": [-4, 0] + rise[2:],
        "first is beyond the rows": [n + 4, 0] + rise[2:],
        "ends beyond the rows": rise[:-1] + [n + 1],
        "ends negative": rise[:-1] + [-1],
        "falls in the middle, behind it all are full": rise[:batch // 2] + [n, n - 1] + [n] * (batch - batch // 2 - 1),
    }


@pytest.mark.parametrize("kind", ["append", "prefill"])
@pytest.mark.parametrize("batch", [3, 40])
@pytest.mark.parametrize("name", offsets(8, 3))
def test_bad_offsets_are_reported(kind, batch, name):
    c = Case((4, 2, 64), [40] * batch, [4] * batch, block=16, seed=80)
    cu = torch.tensor(offsets(c.n, batch)[name], dtype=torch.int32, device="cuda")
    assert cu.shape == c.cu.shape
    kv = torch.randn(c.n, 2, 64, generator=c.g, device="cuda").to(BF)

    def run(cu):
        if kind == "append":
            c.cache.append(c.q, kv, kv, c.lens, cu, theta=1e4)
        else:
            c.cache.prefill(c.q, c.lens, cu)
    c.cache.check()
    run(cu)
    with pytest.raises(MkError) as e:
        c.cache.check()
    assert e.value.status == MK_ERR_INVALID_ARG
    for good in (c.cu, torch.zeros_like(c.cu), torch.full_like(c.cu, c.n)):
        run(good)
        c.cache.check()
