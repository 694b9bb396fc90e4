"""The cache views that a Decoder hands out read what the handle reads."""
import pytest
import torch

import synth
from decode_megakernel_sm_gb300 import Decoder, KVCache

pytestmark = pytest.mark.gpu


def test_views_follow_set_kv_pages():
    cfg = synth.with_cache(synth.custom(n_layers=2, prefill=(0, 0), steps=100))
    W = synth.make_weights(cfg, 5, "cuda")
    ks, vs = synth.make_kv(cfg, [0], 5, "cuda")
    pk, pv, table = synth.paged_pools(ks, vs, 16, 5)
    for pool in pk + pv:
        pool.copy_(torch.randn(pool.shape, device="cuda"))
    dec = Decoder(cfg, W, pk, pv, max_batch=1, max_seq=cfg["max_seq"])
    try:
        with pytest.raises(ValueError, match="set_kv_pages"):
            dec.cache(1)
        dec.set_kv_pages(16, table)
        view = dec.cache(1)
        q = torch.randn(1, cfg["n_q_heads"], cfg["head_dim"], device="cuda").bfloat16()
        lens = torch.tensor([77], dtype=torch.int32, device="cuda")
        first = view.decode(q, lens)
        assert torch.equal(first, KVCache(pk[1], pv[1], table).decode(q, lens))
        other = table.flip(1).contiguous()
        dec.set_kv_pages(16, other)
        second = view.decode(q, lens)
        assert torch.equal(second, KVCache(pk[1], pv[1], other).decode(q, lens))
        assert not torch.equal(first, second)
        dec.set_kv_pages(0, None)
        with pytest.raises(ValueError, match="set_kv_pages"):
            view.decode(q, lens)
        view.check()
    finally:
        dec.close()
