"""Prefill calls whose waits run out: they end, say so, and leave nothing behind for the
next call.  The limit is set so short that a block's own look-ups take longer: a batch
of very many sequences, most of them without a new token."""
import pytest
import torch

from decode_megakernel_sm_gb300 import (MK_ERR_INVALID_ARG, MK_ERR_TIMEOUT, KVCache, MkError,
                                        mk_kv_set_wait_timeout)

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def many(heads, new, n, gap):
    """A cache of sequences with `new` tokens each, n rows, and `gap` without any between them."""
    hq, hkv, d = heads
    g = torch.Generator(device="cuda")
    g.manual_seed(sum(new) + gap)
    batch = 1 + (len(new) - 1) * (gap + 1)
    at = range(0, batch, gap + 1)
    block = 64
    pages = -(-n // block)
    k, v = (torch.randn(len(new) * pages, hkv, block, d, generator=g, device="cuda").to(BF) for _ in range(2))
    table = torch.full((batch, pages), -1, dtype=torch.int32)
    lens, count = torch.zeros(batch, dtype=torch.int32), torch.zeros(batch, dtype=torch.int64)
    for i, b in enumerate(at):
        table[b] = torch.arange(i * pages, (i + 1) * pages)
        lens[b], count[b] = n, new[i]
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), count.cumsum(0)]).to(torch.int32)
    q = torch.randn(sum(new), hq, d, generator=g, device="cuda").to(BF)
    own = [b for b in at]
    dense = KVCache(k, v, table[own].cuda())
    few = torch.full((len(new),), n, dtype=torch.int32, device="cuda"), cu[[0] + [b + 1 for b in own]].cuda()
    return KVCache(k, v, table.cuda()), q, lens.cuda(), cu.cuda(), dense, few


@pytest.mark.parametrize("heads", [(8, 2, 64), (8, 2, 128)])
@pytest.mark.parametrize("new,gap", [([500, 400], 200_000), ([3000, 1, 700], 100_000)], ids=str)
def test_waits_that_run_out(heads, new, gap):
    cache, q, lens, cu, dense, (few_lens, few_cu) = many(heads, new, max(new), gap)
    want = dense.prefill(q, few_lens, few_cu)
    dense.check()
    for _ in range(3):
        try:
            mk_kv_set_wait_timeout(1)
            cache.prefill(q, lens, cu)
        finally:
            mk_kv_set_wait_timeout(0)
        with pytest.raises(MkError) as e:
            cache.check()
        assert e.value.status == MK_ERR_TIMEOUT
        # the next call finds shared and tensor memory as it needs them
        assert torch.equal(dense.prefill(q, few_lens, few_cu), want)
        cache.check()
    # sequences without new tokens have no work: the same work is cut in the same places
    assert torch.equal(cache.prefill(q, lens, cu), want)
    cache.check()


def test_a_time_out_hides_no_bad_contents_and_none_hide_it():
    cache, q, lens, cu, dense, (few_lens, few_cu) = many((8, 2, 64), [500, 400], 500, 200_000)
    for timeout_first in (True, False):
        bad = few_lens.clone()
        bad[0] = -1
        order = [lambda: dense.prefill(q, bad, few_cu), lambda: cache.prefill(q, lens, cu)]
        try:
            mk_kv_set_wait_timeout(1)
            for call in order[::-1] if timeout_first else order:
                call()
        finally:
            mk_kv_set_wait_timeout(0)
        with pytest.raises(MkError) as e:
            cache.check()
        assert e.value.status == MK_ERR_TIMEOUT
        cache.check()
    dense.prefill(q, bad, few_cu)
    with pytest.raises(MkError) as e:
        cache.check()
    assert e.value.status == MK_ERR_INVALID_ARG
