"""The cache operators together, as they are used: prompts are filled in with
append and prefill layer by layer (plain torch products around them), further
tokens go through append and decode, and the decode step continues from that
cache.  Everything is checked against the CPU oracle, which takes the same
tokens one at a time.

Tolerance: the oracle rounds nothing but the cache rows.  Here a layer's
attention has three more roundings to bf16 (queries, weights, output), each off
by at most 2^-8 of its norm; the linear maps around them keep relative norms.
So a cache row of layer l is off by at most (3 l + 1) 2^-8 of its norm, the
logits after L layers by (3 L + 1) 2^-8 of theirs."""
import numpy as np
import pytest
import torch

import oracle
import synth
from decode_megakernel_sm_gb300 import Decoder

pytestmark = pytest.mark.gpu

CASES = {
    "tiny": dict(cfg=dict(n_layers=3, steps=80), lens=[37], paged=None),
    "tiny_paged": dict(cfg=dict(n_layers=3, steps=150), lens=[133], paged=16),
    "batch": dict(cfg=dict(n_layers=2, hidden=2048, n_q_heads=8, n_kv_heads=2, ffn=1024, vocab=2000,
                           batch=3, steps=80, rope_theta=5e5), lens=[37, 1, 64], paged=32),
    "d128": dict(cfg=dict(n_layers=2, hidden=2048, n_q_heads=8, n_kv_heads=2, head_dim=128, ffn=512,
                          vocab=2000, steps=60, rope_theta=5e5), lens=[41], paged=None),
}


def norm(x, gain, eps):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * gain.float()


def forward(cfg, W, dec, tokens, lens, cu):
    """Logits of every row of `tokens`, through the cache operators; cu None: one
    token per sequence."""
    d = cfg["head_dim"]
    x = W["embed"][tokens].float()
    for l, w in enumerate(W["layers"]):
        h = norm(x, w["attn_norm"], cfg["rms_eps"])
        q, k, v = ((h @ w[n].float().T).unflatten(1, (-1, d)) for n in ("wq", "wk", "wv"))
        cache = dec.cache(l)
        q = cache.append(q, k, v, lens, cu, theta=cfg["rope_theta"])
        o = cache.decode(q, lens) if cu is None else cache.prefill(q, lens, cu)
        x = x + o.flatten(1).float() @ w["wo"].float().T
        h = norm(x, w["mlp_norm"], cfg["rms_eps"])
        x = x + (torch.nn.functional.silu(h @ w["w_gate"].float().T) *
                 (h @ w["w_up"].float().T)) @ w["w_down"].float().T
    cache.check()
    return norm(x, W["final_norm"], cfg["rms_eps"]) @ W["embed"].float().T


def off(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


@pytest.mark.parametrize("name", CASES)
def test_prompt_then_tokens_then_steps(name):
    case = CASES[name]
    cfg = synth.with_cache(synth.custom(prefill=(0, 0), **case["cfg"]))
    B, L, seed = cfg["batch"], cfg["n_layers"], 71
    W = synth.make_weights(cfg, seed, "cuda")
    ks, vs = synth.make_kv(cfg, [0] * B, seed, "cuda")
    ko, vo = ([oracle._bits(t.cpu()).copy() for t in ts] for ts in (ks, vs))
    om = oracle.OracleModel(cfg, W)
    if case["paged"]:
        pk, pv, table = synth.paged_pools(ks, vs, case["paged"], seed)
        dec = Decoder(cfg, W, pk, pv, max_batch=B, max_seq=cfg["max_seq"])
        dec.set_kv_pages(case["paged"], table)
    else:
        dec = Decoder(cfg, W, ks, vs)
    dec.build_schedule(B, cfg["max_seq"])

    def rows(l, kind, b, n):  # the first n cache rows, [n][Hkv][d]
        if not case["paged"]:
            return (ks, vs)[kind][l][b, :, :n].transpose(0, 1).float().cpu().numpy()
        pool, p = (pk, pv)[kind][l], torch.arange(n, device="cuda")
        return pool[table[b, p // case["paged"]].long(), :, p % case["paged"]].float().cpu().numpy()

    def oracle_row(l, kind, b, n):
        o = ((ko, vo)[kind][l][b, :, :n].astype(np.uint32) << 16).view(np.float32)
        return o.transpose(1, 0, 2)

    def oracle_step(toks, pos):  # one token of every sequence
        out = []
        for b in range(B):
            lg, _, _, _ = om.step([a[b:b + 1] for a in ko], [a[b:b + 1] for a in vo], [toks[b]],
                                  [pos[b]])
            out.append(lg[0])
        return np.stack(out)

    tol = (3 * L + 1) * 2.0 ** -8
    try:
        # prompts, all at once
        lens_l = case["lens"]
        g = torch.Generator().manual_seed(seed)
        prompt = [torch.randint(0, cfg["vocab"], (n,), generator=g).tolist() for n in lens_l]
        cu = torch.tensor([0] + list(np.cumsum(lens_l)), dtype=torch.int32, device="cuda")
        lens = torch.tensor(lens_l, dtype=torch.int32, device="cuda")
        logits = forward(cfg, W, dec, torch.tensor(sum(prompt, []), device="cuda"), lens, cu)
        for b in range(B):
            for i, t in enumerate(prompt[b]):
                lo, _, _, _ = om.step([a[b:b + 1] for a in ko], [a[b:b + 1] for a in vo], [t], [i])
                assert off(logits[cu[b] + i].double().cpu().numpy(), lo[0]) <= tol
        for l in range(L):
            for kind in (0, 1):
                for b, n in enumerate(lens_l):
                    assert off(rows(l, kind, b, n), oracle_row(l, kind, b, n)) <= (3 * l + 1) * 2.0 ** -8

        # three tokens through append + decode, three through the decode step
        pos = list(lens_l)
        for i in range(6):
            toks = torch.randint(0, cfg["vocab"], (B,), generator=g)
            if i < 3:
                lens.add_(1)
                got = forward(cfg, W, dec, toks.cuda(), lens, None)
            else:
                got = torch.empty((B, cfg["vocab"]), dtype=torch.float32, device="cuda")
                am = torch.empty(B, dtype=torch.int32, device="cuda")
                dec.step(toks.to("cuda", torch.int32),
                         torch.tensor(pos, dtype=torch.int32, device="cuda"), got, am)
                assert dec.sync_status() == 0
            want = oracle_step(toks.tolist(), pos)
            for b in range(B):
                assert off(got[b].double().cpu().numpy(), want[b]) <= tol
            pos = [p + 1 for p in pos]
    finally:
        dec.close()
