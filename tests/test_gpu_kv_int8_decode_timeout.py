"""Decode over an 8-bit cache whose waits run out: the calls end, say so, and leave nothing
behind for the next.  The limit is 1 ns.  A warp's copies are mostly there a step before it waits
for them, so the caches are larger than L2, which makes nearly every call have a warp that waits
(of 60 calls 36 to 60 gave up), and a test calls until it has seen three give up."""
import pytest
import torch

from decode_megakernel_sm_gb300 import MK_ERR_INVALID_ARG, MK_ERR_TIMEOUT, MkError, mk_kv_set_wait_timeout
from tests.test_gpu_kv_int8 import Case8

pytestmark = pytest.mark.gpu

CALLS = 200
EVEN, UNEVEN = [20_001] * 16, [30_001, 3, 0] * 6


def short(call):
    try:
        mk_kv_set_wait_timeout(1)
        return call()
    finally:
        mk_kv_set_wait_timeout(0)


def status(cache):
    try:
        cache.check()
    except MkError as e:
        return e.status
    return 0


# pages of one and of two halves of a unit, whole units and not, and caches in one piece whose
# group bytes begin anywhere; one head block to a kv head and two
@pytest.mark.parametrize("heads,block,lens", [
    ((32, 8, 64), 0, EVEN), ((32, 8, 64), 16, UNEVEN), ((32, 8, 64), 64, UNEVEN), ((32, 8, 64), 256, EVEN),
    ((16, 4, 128), 0, UNEVEN), ((16, 4, 128), 16, UNEVEN), ((16, 4, 128), 64, EVEN), ((16, 4, 128), 256, UNEVEN),
    ((64, 4, 64), 0, EVEN), ((64, 4, 64), 64, EVEN), ((64, 4, 128), 0, UNEVEN), ((64, 4, 128), 64, UNEVEN)], ids=str)
def test_waits_that_run_out(heads, block, lens):
    c = Case8(heads, lens, block=block, seed=30)
    want, want_lse = c.cache.decode(c.q, c.lens, return_lse=True)
    c.cache.check()
    seen = 0
    for _ in range(CALLS):
        got = short(lambda: c.cache.decode(c.q, c.lens))
        found = status(c.cache)
        if found == 0:  # nobody had to wait
            assert torch.equal(got, want)
            continue
        assert found == MK_ERR_TIMEOUT
        # the next call finds shared memory as it needs it
        out, lse = c.cache.decode(c.q, c.lens, return_lse=True)
        assert torch.equal(out, want) and torch.equal(lse, want_lse)
        c.cache.check()
        seen += 1
        if seen == 3:
            return
    assert False, f"{seen} of {CALLS} calls gave up"


def test_a_limit_that_is_long_enough_changes_nothing():
    c = Case8((32, 8, 64), EVEN, block=64, seed=31)
    want = c.cache.decode(c.q, c.lens)
    for ns in (1_000_000, 100_000_000, 1 << 62):
        try:
            mk_kv_set_wait_timeout(ns)
            assert torch.equal(c.cache.decode(c.q, c.lens), want)
        finally:
            mk_kv_set_wait_timeout(0)
        c.cache.check()


def test_a_captured_call_keeps_its_limit():
    c = Case8((32, 8, 64), EVEN, block=64, seed=32)
    want = c.cache.decode(c.q, c.lens)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        short(lambda: c.cache.decode(c.q, c.lens))
    for _ in range(CALLS):
        graph.replay()
        found = status(c.cache)
        assert found in (0, MK_ERR_TIMEOUT)
        if found:
            break
    assert found == MK_ERR_TIMEOUT
    assert torch.equal(c.cache.decode(c.q, c.lens), want)
    c.cache.check()


def test_a_time_out_hides_bad_contents_of_its_call_alone():
    c = Case8((32, 8, 64), EVEN, block=64, seed=33)
    bad = c.lens.clone()
    bad[1] = -1
    for _ in range(CALLS):
        short(lambda: c.cache.decode(c.q, bad))
        found = status(c.cache)
        assert found in (MK_ERR_INVALID_ARG, MK_ERR_TIMEOUT)
        if found == MK_ERR_TIMEOUT:
            break
    assert found == MK_ERR_TIMEOUT
    assert status(c.cache) == 0
    c.cache.decode(c.q, bad)
    assert status(c.cache) == MK_ERR_INVALID_ARG
