"""Cases of the KV-cache operators: the rotating append (``kv_append``), the
attention of one new token per sequence (``attn_decode``) and the attention of
a chunk of new tokens per sequence (``attn_prefill``) over a cache in pages or
in one piece.

``own`` false: ``run`` computes the operators in plain torch arithmetic in 32
bits (angles in 64); true: it calls the package.

A case: ``op``; query heads ``hq``, kv heads ``hkv``, head size ``d``; page
rows ``block`` (0: a contiguous cache); ``batch`` sequences whose cache lengths
after the append lie in [``lo``, ``hi``]; and for append and prefill the new
tokens per sequence, in [``new_lo``, ``new_hi``] (0: all of the sequence's
rows, a fresh prompt).  Lengths follow from the case alone.
"""
import math
import random

import torch

own = False

THETA = 5e5

# The head shapes of this repository's configurations and tests, and generic
# ones: one kv head for all query heads, and a kv head for each.
HEADS = [(32, 8, 64), (16, 4, 128), (4, 2, 64), (6, 3, 64), (8, 2, 128), (8, 1, 64), (12, 12, 64),
         (10, 2, 128), (16, 1, 128)]
BLOCKS = [0, 16, 32, 64, 256, 4096]


def listed():
    def c(name, op, heads, block, batch, lo, hi, new_lo=1, new_hi=1, src="bf16"):
        return dict(name=name, op=op, hq=heads[0], hkv=heads[1], d=heads[2], block=block,
                    batch=batch, lo=lo, hi=hi, new_lo=new_lo, new_hi=new_hi, src=src)

    return [
        # one sequence's decode step: latency only
        c("append_one", "append", (32, 8, 64), 16, 1, 1024, 1024),
        # a serving batch's decode step, rows straight from fp32 projections
        c("append_batch32", "append", (32, 8, 64), 64, 32, 512, 2048, src="f32"),
        # eight prompts of different lengths filled at once
        c("append_prompts", "append", (32, 8, 64), 64, 8, 512, 2048, 0, 0),
        # long prompts of a 128-dim model, the largest append
        c("append_long", "append", (16, 4, 128), 256, 4, 8192, 8192, 0, 0, "f32"),
        # one sequence at 1K context: latency, and the split over the length
        c("decode_one_1k", "decode", (32, 8, 64), 16, 1, 1024, 1024),
        # the ordinary small batch at mixed lengths
        c("decode_batch8", "decode", (32, 8, 64), 64, 8, 512, 2048),
        # a few odd sequences of a 128-dim model (an empty slot to thousands), contiguous
        c("decode_odd_d128", "decode", (16, 4, 128), 0, 5, 0, 5001),
        # a full batch at 32K context: the cache's bytes at the card's rate
        c("decode_batch32_32k", "decode", (32, 8, 64), 256, 32, 16384, 32768),
        # one fresh prompt of 1K tokens
        c("prefill_one_1k", "prefill", (32, 8, 64), 64, 1, 1024, 1024, 0, 0),
        # eight fresh prompts of mixed lengths
        c("prefill_prompts", "prefill", (32, 8, 64), 64, 8, 512, 2048, 0, 0),
        # few new tokens over long caches (drafts to verify, short turns)
        c("prefill_short_chunks", "prefill", (32, 8, 64), 16, 4, 8000, 20000, 5, 16),
        # an 8K prompt of a 128-dim model: the largest, matrix products
        c("prefill_long_d128", "prefill", (16, 4, 128), 256, 1, 8192, 8192, 0, 0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill"])
    hq, hkv, d = rng.choice(HEADS)
    block = rng.choice(BLOCKS)
    src = rng.choice(["bf16", "f32"]) if op == "append" else "bf16"
    batch = _log(rng, 1, 32)
    if op == "decode":
        hi = _log(rng, 1, 32768 if hkv * d <= 512 else 8192)
        lo = rng.choice([hi, hi // 4, 0])
        new = (1, 1)
    else:
        # the rows of one sequence, within the largest listed case's work
        most = 32768 // batch if op == "append" else int(8192 / math.sqrt(batch * hq * d / 2048))
        hi = _log(rng, 1, max(1, min(8192, most)))
        lo = max(1, rng.choice([hi, hi // 2, hi // 8]))
        kind = rng.choice(["fresh", "chunk", "few"])
        new = {"fresh": (0, 0), "chunk": (max(1, lo // 3), max(1, lo // 2)),
               "few": (1, min(lo, 7))}[kind]
    return dict(op=op, hq=hq, hkv=hkv, d=d, block=block, batch=batch, lo=lo, hi=hi, new_lo=new[0],
                new_hi=new[1], src=src)


def _batch(case):
    """(cache lengths after the append, new tokens) of every sequence."""
    r = random.Random("%(op)s %(hq)d %(d)d %(batch)d %(lo)d %(hi)d %(new_lo)d %(new_hi)d" % case)
    lens = [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    if case["batch"] > 1:
        lens[0], lens[-1] = case["hi"], case["lo"]
    if case["op"] == "decode":
        return lens, [1] * case["batch"]
    if case["new_hi"] == 0:
        return lens, list(lens)
    return lens, [min(n, r.randint(case["new_lo"], case["new_hi"])) for n in lens]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device="cuda", dtype=dtype)

    lens, new = _batch(case)
    hq, hkv, d, batch, block = (case[k] for k in ("hq", "hkv", "d", "batch", "block"))
    n, longest = sum(new), max(lens + [1])
    cu = [0]
    for m in new:
        cu.append(cu[-1] + m)
    s = dict(op=case["op"], n=n, batch=batch, hq=hq, hkv=hkv, d=d, longest=longest,
             most_new=max(new), scale=1.0 / math.sqrt(d), block=block)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["one_each"] = all(m == 1 for m in new)  # a decode step: the program knows it makes one
    if block:
        pages = -(-longest // block)
        blocks = batch * pages + 3
        order = torch.randperm(blocks, generator=torch.Generator().manual_seed(seed + 5))
        s["table"] = order[:batch * pages].reshape(batch, pages).to(torch.int32).cuda()
        s["k"], s["v"] = normal(blocks, hkv, block, d), normal(blocks, hkv, block, d)
    else:
        rows = longest + 5
        s["table"] = None
        s["k"], s["v"] = normal(batch, hkv, rows, d), normal(batch, hkv, rows, d)
    if case["op"] == "append":
        # the queries' projection, and a fused one with keys and values side by side
        src = torch.float32 if case["src"] == "f32" else torch.bfloat16
        s["q_new"] = normal(n, hq, d, dtype=src)
        kv = normal(n, 2 * hkv * d, dtype=src)
        s["k_new"] = kv[:, :hkv * d].unflatten(1, (hkv, d))
        s["v_new"] = kv[:, hkv * d:].unflatten(1, (hkv, d))
    else:
        # queries as the append leaves them; wide enough that the softmax has peaks
        s["q"] = (normal(n, hq, d, dtype=torch.float32) * 1.5).to(torch.bfloat16)
    return s


def run(s):
    if own:
        from decode_megakernel_sm_gb300 import KVCache

        cache = KVCache(s["k"], s["v"], s["table"])
        if s["op"] == "append":
            q = cache.append(s["q_new"], s["k_new"], s["v_new"], s["lens"],
                             None if s["one_each"] else s["cu"], theta=THETA)
            return q, s["k"], s["v"]
        if s["op"] == "decode":
            return cache.decode(s["q"], s["lens"], scale=s["scale"], return_lse=True)
        return cache.prefill(s["q"], s["lens"], s["cu"], scale=s["scale"], return_lse=True)
    return _plain_append(s) if s["op"] == "append" else _plain_attention(s)


def _places(s):
    """(sequence, position in it) of every new token."""
    t = torch.arange(s["n"], device="cuda")
    seq = (t[:, None] >= s["cu"][None, 1:]).sum(1)
    return seq, s["lens"][seq] - s["cu"][seq + 1] + t


def _plain_append(s):
    seq, pos = _places(s)
    half = s["d"] // 2
    freq = THETA ** (torch.arange(half, device="cuda", dtype=torch.float64) * (-2.0 / s["d"]))
    angle = pos.double()[:, None] * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def rotated(x):
        a, b = x[..., :half].float(), x[..., half:].float()
        return torch.cat((a * cos - b * sin, b * cos + a * sin), -1).to(torch.bfloat16)

    if s["table"] is None:
        block, row = seq, pos
    else:
        block, row = s["table"][seq, pos // s["block"]].long(), pos % s["block"]
    s["k"][block, :, row] = rotated(s["k_new"])
    s["v"][block, :, row] = s["v_new"].to(torch.bfloat16)
    return rotated(s["q_new"]), s["k"], s["v"]


def _plain_attention(s):
    batch, hkv, d, longest, most = s["batch"], s["hkv"], s["d"], s["longest"], s["most_new"]

    def rows(pool):  # [batch][hkv][longest][d]
        if s["table"] is not None:
            pool = pool[s["table"].long()].transpose(1, 2).flatten(2, 3)
        return pool[:, :, :longest].float()

    seq, pos = _places(s)
    at = seq * most + torch.arange(s["n"], device="cuda") - s["cu"][seq]
    q = torch.zeros(batch * most, s["hq"], d, device="cuda")
    q[at] = s["q"].float()
    last = torch.full((batch * most,), -1, dtype=torch.int64, device="cuda")
    last[at] = pos
    # [batch][hkv][group * most][d]
    q = q.reshape(batch, most, hkv, -1, d).permute(0, 2, 3, 1, 4)
    group = q.shape[2]
    x = q.reshape(batch, hkv, group * most, d) @ rows(s["k"]).transpose(2, 3) * s["scale"]
    seen = torch.arange(longest, device="cuda") <= last.reshape(batch, 1, most, 1)
    x = x.reshape(batch, hkv, group, most, longest).masked_fill_(~seen[:, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = x.sub_(top.clamp(min=-1e30)).exp_()
    total = x.sum(-1, keepdim=True)
    o = x.reshape(batch, hkv, group * most, longest) @ rows(s["v"])
    o = o.reshape(batch, hkv, group, most, d) / total.clamp(min=1e-30)
    lse = (top + total.log())[..., 0]

    def back(y):  # [batch][hkv][group][most]... -> [token][query head]...
        return y.movedim(3, 1).flatten(0, 1).flatten(1, 2)[at]

    return back(o).to(torch.bfloat16), back(lse)


def work(case):
    lens, new = _batch(case)
    hq, hkv, d, n = case["hq"], case["hkv"], case["d"], sum(new)
    if case["op"] == "append":
        src = 4 if case["src"] == "f32" else 2
        return {"bytes": n * (hq + 2 * hkv) * d * (src + 2) + 8 * case["batch"],
                "flops": 3 * n * (hq + hkv) * d}
    pairs = sum(m * (2 * length - m + 1) // 2 for length, m in zip(lens, new))
    return {"bytes": 4 * hkv * d * sum(lens) + n * hq * (4 * d + 4) + 8 * case["batch"],
            "flops": 4 * hq * d * pairs}


def exact(case, seed):
    s = prepare(case, seed)
    lens, new = _batch(case)
    hq, hkv, d, block = case["hq"], case["hkv"], case["d"], case["block"]
    dev = s["k"].device

    def addresses(b, first, last):  # pool block and row of positions [first, last) of sequence b
        p = torch.arange(first, last, device=dev)
        if not block:
            return torch.full_like(p, b), p
        return s["table"][b].to(torch.int64)[torch.div(p, block, rounding_mode="floor")], p % block

    if case["op"] == "append":
        k, v, q = s["k"].double(), s["v"].double(), s["q_new"].double()
        at = 0
        for b, (length, m) in enumerate(zip(lens, new)):
            p = torch.arange(length - m, length, device=dev, dtype=torch.float64)
            turn = torch.outer(p, torch.exp(torch.arange(d // 2, device=dev, dtype=torch.float64)
                                            * (-2 * math.log(THETA) / d)))
            turn = torch.polar(torch.ones_like(turn), turn)[:, None]

            def spin(x):  # the pair (t, t + d / 2) as a complex number times e^(i angle)
                z = torch.complex(x[..., :d // 2].contiguous(), x[..., d // 2:].contiguous()) * turn
                return torch.cat((z.real, z.imag), -1)

            at_block, at_row = addresses(b, length - m, length)
            k[at_block, :, at_row] = spin(s["k_new"][at:at + m].double())
            v[at_block, :, at_row] = s["v_new"][at:at + m].double()
            q[at:at + m] = spin(s["q_new"][at:at + m].double())
            at += m
        return q, k, v

    out = torch.zeros(s["n"], hq, d, dtype=torch.float64, device=dev)
    lse = torch.full((s["n"], hq), -math.inf, dtype=torch.float64, device=dev)
    at = 0
    for b, (length, m) in enumerate(zip(lens, new)):
        at_block, at_row = addresses(b, 0, length)
        keys, values = s["k"][at_block, :, at_row].double(), s["v"][at_block, :, at_row].double()
        for first in range(0, m, 2048):
            size = min(2048, m - first)
            hidden = torch.arange(length, device=dev)[None] > \
                torch.arange(length - m + first, length - m + first + size, device=dev)[:, None]
            for h in range(hq):
                token = slice(at + first, at + first + size)
                kv = h * hkv // hq
                logit = torch.einsum("td,jd->tj", s["q"][token, h].double(), keys[:, kv])
                logit = logit.div_(math.sqrt(d)).masked_fill_(hidden, -math.inf)
                lse[token, h] = torch.logsumexp(logit, 1)
                out[token, h] = torch.softmax(logit, 1) @ values[:, kv]
        at += m
    return out, lse
