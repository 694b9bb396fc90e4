"""The limit of a prefill's waits is about its own progress: a kernel that widens rows before
it may take longer.  Here that kernel's last blocks are busy long after the others are done, so
that most SMs have a block of the prefill long before the rows are there: of every run of
tokens as long as all its warps, the last 32 alone have rows to widen (a token of 64 heads
takes a warp some 4 us, one without a position 1)."""
import pytest
import torch

from decode_megakernel_sm_gb300 import KVCache, mk_kv_set_wait_timeout
from tests.test_gpu_kv_int8 import quantised
from tests.test_gpu_kv_int8_widened_timeout import widened

pytestmark = pytest.mark.gpu


def test_the_time_of_the_widening_does_not_count():
    batch, heads, dim, rows = 200, 64, 64, 32
    run = 32 * torch.cuda.get_device_properties("cuda").multi_processor_count  # warps of the widening
    n = batch * run
    assert widened(n, batch, (heads, heads, dim))
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    k, v = (torch.randn(batch, heads, rows, dim, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    (k, ks), (v, vs) = quantised(k), quantised(v)
    cache = KVCache(k, v, None, scales=(ks, vs))
    lens = torch.full((batch,), rows, dtype=torch.int32, device="cuda")
    cu = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * run
    q = torch.zeros(n, heads, dim, dtype=torch.bfloat16, device="cuda")  # (8 GB)
    seen = q.view(batch, run, heads, dim)[:, -rows:]
    seen.copy_(torch.randn(seen.shape, generator=g, device="cuda"))
    out = torch.empty_like(q)

    def run_once():
        out.fill_(1.0)
        cache.prefill(q, lens, cu, out=out)
        cache.check()
        tokens = out.view(batch, run, heads, dim)
        assert not tokens[:, :-rows].any()  # nothing to attend to
        return tokens[:, -rows:].clone()

    want = run_once()
    for _ in range(3):
        try:
            mk_kv_set_wait_timeout(1)
            got = run_once()
        finally:
            mk_kv_set_wait_timeout(0)
        assert torch.equal(got, want)
