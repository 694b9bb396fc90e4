"""Prefill over widened rows of an 8-bit cache whose waits run out: the calls end, say so, and
leave nothing behind for the next.  Rows are widened where the new tokens, padding among them,
are many for the sequences; the limit is shorter than the way from one sequence with tokens
to the next, over those between that have none."""
import pytest
import torch

from decode_megakernel_sm_gb300 import (MK_ERR_TIMEOUT, KVCache, MkError, mk_attn_int8_workspace_bytes,
                                        mk_attn_workspace_bytes, mk_kv_set_wait_timeout)
from tests.test_gpu_kv_int8 import quantised
from tests.test_gpu_kv_timeout import many

pytestmark = pytest.mark.gpu


def widened(n, batch, heads):
    """Whether a prefill of these sizes widens its rows first."""
    return mk_attn_int8_workspace_bytes(False, n, batch, *heads) > mk_attn_workspace_bytes(False, n, batch, *heads)


@pytest.mark.parametrize("heads", [(128, 1, 64), (128, 1, 128)])
@pytest.mark.parametrize("new", [[500, 400], [1500, 1, 700]], ids=str)
def test_waits_that_run_out(heads, new):
    gap = 8000 // (len(new) - 1)
    cache, q, lens, cu, dense, (few_lens, few_cu) = many(heads, new, max(new), gap)
    (k, ks), (v, vs) = quantised(cache.k), quantised(cache.v)
    cache, dense = (KVCache(k, v, c.table, scales=(ks, vs)) for c in (cache, dense))
    n, rows = len(q), 34 * lens.shape[0]
    assert widened(rows, lens.shape[0], heads) and widened(n, len(new), heads)
    padded = torch.empty(rows, *q.shape[1:], dtype=q.dtype, device="cuda")
    padded[:n] = q
    want = dense.prefill(q, few_lens, few_cu)
    dense.check()
    for _ in range(3):
        try:
            mk_kv_set_wait_timeout(1)
            cache.prefill(padded, lens, cu)
        finally:
            mk_kv_set_wait_timeout(0)
        with pytest.raises(MkError) as e:
            cache.check()
        assert e.value.status == MK_ERR_TIMEOUT
        # the next call finds shared and tensor memory as it needs them
        assert torch.equal(dense.prefill(q, few_lens, few_cu), want)
        cache.check()
    # sequences without new tokens have no work: the same work is cut in the same places
    assert torch.equal(cache.prefill(padded, lens, cu)[:n], want)
    cache.check()
