"""KV-cache operators against plain 64-bit implementations of their formulas.

Tolerances, per element, derived before the first run (a bf16 rounding is off
by at most 2^-8 of the value):
  append: the pair's rotation in fp32 (angle, sincos, two products, one sum: a
    few units of 2^-24 of the pair's norm, 2^-20 allowed), then one rounding.
  attention: with A = sum p |v| / sum p, the output is rounded once (2^-8 |o|),
    and each weight is off by at most r: the score's error twice (numerator and
    sum), where a score is a dot product of D exact products summed in fp32 in
    any order, with truncation (D 2^-23 scale sum |q k|, bounded by |q||k|), the
    exponential (2^-14 allowed: exp2 of an fp32 argument up to 2^6 has an
    argument off by 2^-18), plus the rounding of the weights before the second
    product where the kernel makes one: WEIGHT below.
  lse: the score's error, plus 2^-20 (1 + |lse|) for exp, sum and log."""
import math
import pathlib
import subprocess
import sys

import pytest
import torch

from decode_megakernel_sm_gb300 import KVCache, MK_ERR_INVALID_ARG, MkError

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
# rounding of the weights: decode carries them in two bf16 parts, prefill in one
WEIGHT = {"decode": 2.0 ** -15, "prefill": 2.0 ** -8}


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


class Case:
    """A cache with random rows, NaN in every row that no sequence has, block ids
    that nothing should read set to -1."""

    def __init__(self, heads, lens, new=None, block=16, seed=0, stored=None, spare=3, fill=math.nan):
        self.hq, self.hkv, self.d = heads
        self.lens_l, self.new_l, self.block = list(lens), list(new or [1] * len(lens)), block
        g = self.g = gen(seed)
        B, longest = len(lens), max(list(lens) + [1])
        stored = lens if stored is None else stored  # rows that hold data already
        if block:
            pages = -(-longest // block) + 1
            n_blocks = B * pages + spare
            table = torch.randperm(n_blocks, generator=torch.Generator().manual_seed(seed))
            table = table[:B * pages].reshape(B, pages).to(torch.int32)
            for b, n in enumerate(lens):
                table[b, -(-n // block):] = -1
            self.table = table.cuda()
            shape = (n_blocks, self.hkv, block, self.d)
        else:
            self.table = None
            shape = (B, self.hkv, longest + 3, self.d)
        self.k, self.v = (torch.full(shape, fill, dtype=BF, device="cuda") for _ in range(2))
        for b, n in enumerate(stored):
            blk, row = self.at(b, 0, n)
            for pool in (self.k, self.v):
                pool[blk, :, row] = torch.randn(n, self.hkv, self.d, generator=g, device="cuda").to(BF)
        self.cache = KVCache(self.k, self.v, self.table)
        self.lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        cu = [0]
        for m in self.new_l:
            cu.append(cu[-1] + m)
        self.cu_l, self.n = cu, cu[-1]
        self.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        self.q = (torch.randn(self.n, self.hq, self.d, generator=g, device="cuda") * 1.5).to(BF)

    def at(self, b, first, last):
        p = torch.arange(first, last, device="cuda")
        if not self.block:
            return torch.full_like(p, b), p
        return self.table[b].long()[p // self.block], p % self.block

    def rows(self, b):
        blk, row = self.at(b, 0, self.lens_l[b])
        return self.k[blk, :, row].double(), self.v[blk, :, row].double()  # [rows][hkv][d]

    def reference(self, scale=None):
        """(out, lse, A, score error) in 64 bits."""
        scale = 1 / math.sqrt(self.d) if scale is None else scale
        G = self.hq // self.hkv
        out = torch.zeros(self.n, self.hq, self.d, dtype=torch.float64, device="cuda")
        A, lse = torch.zeros_like(out), torch.full((self.n, self.hq), -math.inf,
                                                   dtype=torch.float64, device="cuda")
        err = torch.zeros_like(lse)
        for b, (n, m) in enumerate(zip(self.lens_l, self.new_l)):
            K, V = self.rows(b)
            for i in range(m):
                seen, t = n - m + i + 1, self.cu_l[b] + i
                if seen <= 0:
                    continue
                q = self.q[t].double().reshape(self.hkv, G, self.d)
                s = torch.einsum("hgd,jhd->hgj", q, K[:seen]) * scale
                top = s.amax(-1, keepdim=True)
                p = (s - top).exp()
                total = p.sum(-1, keepdim=True)
                w = p / total
                out[t] = torch.einsum("hgj,jhd->hgd", w, V[:seen]).reshape(self.hq, self.d)
                A[t] = torch.einsum("hgj,jhd->hgd", w, V[:seen].abs()).reshape(self.hq, self.d)
                lse[t] = (top + total.log()).reshape(self.hq)
                norm = q.norm(dim=-1) * K[:seen].norm(dim=-1).amax(0)[:, None]
                err[t] = (norm * abs(scale) * self.d * 2.0 ** -23).reshape(self.hq)
        return out, lse, A, err

    def run(self, kind, **kw):
        if kind == "decode":
            return self.cache.decode(self.q, self.lens, return_lse=True, **kw)
        return self.cache.prefill(self.q, self.lens, self.cu, return_lse=True, **kw)

    def check(self, kind, got, scale=None):
        out, lse = got
        ro, rl, A, err = self.reference(scale)
        tol = 2.0 ** -8 * ro.abs() + (2 * err + 2.0 ** -14 + WEIGHT[kind])[..., None] * A
        bad = ~((out.double() - ro).abs() <= tol)
        assert not bad.any(), f"out: {int(bad.sum())} of {bad.numel()}, first {bad.nonzero()[0]}, " \
            f"worst {((out.double() - ro).abs() - tol).max()}"
        empty = torch.isinf(rl)
        assert torch.equal(torch.isinf(lse), empty) and (lse[empty] < 0).all()
        off = (lse.double() - rl).abs()[~empty]
        allowed = (err + 2.0 ** -20 * (1 + rl.abs()))[~empty]
        assert (off <= allowed).all(), f"lse off by {(off - allowed).max()}"
        self.cache.check()


HEADS = [(4, 2, 64), (6, 3, 64), (32, 8, 64), (16, 4, 128), (8, 1, 64), (3, 3, 128), (12, 1, 128),
         (40, 2, 64), (33, 1, 64)]
LENS = [[1], [0], [15, 16, 17], [0, 1, 2, 0, 33], [63, 64, 65, 127, 128, 129], [300, 1, 1000, 513],
        [4099]]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("lens", LENS, ids=str)
def test_decode(heads, lens):
    c = Case(heads, lens, block=16, seed=1)
    c.check("decode", c.run("decode"))


@pytest.mark.parametrize("block", [0, 16, 64, 256, 4096])
@pytest.mark.parametrize("heads", [(8, 2, 64), (8, 2, 128)])
def test_decode_blocks(heads, block):
    c = Case(heads, [700, 3, 0, 5000, 256, 257], block=block, seed=2)
    c.check("decode", c.run("decode"))


def test_decode_many_sequences():
    # more sequences than threads of a block, most of them short or empty
    lens = [(7 * b * b) % 61 if b % 3 else 0 for b in range(700)]
    lens[411] = 3001
    c = Case((4, 2, 64), lens, block=16, seed=3)
    c.check("decode", c.run("decode"))


def test_decode_long():
    c = Case((8, 2, 64), [100_003, 17, 65_536], block=256, seed=4)
    c.check("decode", c.run("decode"))


CHUNKS = [([1], [1]), ([1, 0, 2], [1, 0, 2]), ([17, 16, 15], [17, 3, 1]),
          ([130, 128, 127, 129], [130, 128, 127, 129]), ([300, 5, 900], [1, 5, 77]),
          ([257, 1000], [256, 31]), ([3, 4], [5, 4])]  # the last: positions below zero


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("lens,new", CHUNKS, ids=str)
def test_prefill(heads, lens, new):
    c = Case(heads, lens, new, block=16, seed=5)
    c.check("prefill", c.run("prefill"))


@pytest.mark.parametrize("block", [0, 16, 32, 64, 256, 4096])
@pytest.mark.parametrize("heads", [(8, 2, 64), (8, 2, 128), (5, 1, 64)])
def test_prefill_blocks(heads, block):
    c = Case(heads, [700, 3, 1500, 0, 256, 257], [129, 3, 64, 0, 256, 1], block=block, seed=6)
    c.check("prefill", c.run("prefill"))


def test_prefill_many_sequences():
    lens = [(5 * b * b) % 97 for b in range(600)]
    new = [n if b % 2 else n // 2 for b, n in enumerate(lens)]
    c = Case((4, 2, 64), lens, new, block=16, seed=7)
    c.check("prefill", c.run("prefill"))


def test_prefill_few_tokens_over_long_caches():
    c = Case((8, 2, 64), [20_011, 9000, 12_345], [3, 1, 16], block=64, seed=8)
    c.check("prefill", c.run("prefill"))


def test_prefill_equals_decode_of_the_same_tokens():
    c = Case((8, 2, 128), [500, 77, 1, 1300], [1, 1, 1, 1], block=32, seed=9)
    c.check("decode", c.run("decode"))
    c.check("prefill", c.run("prefill"))


@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("scale", [0.0, 1.0, -0.3, 40.0])
def test_scales(kind, scale):
    c = Case((8, 2, 64), [500, 200], [1, 1], block=16, seed=10)
    c.check(kind, c.run(kind, scale=scale), scale)


@pytest.mark.parametrize("kind", ["decode", "prefill"])
@pytest.mark.parametrize("peak", ["first", "last", "rising", "equal"])
def test_score_shapes(kind, peak):
    # one key far above the rest, running maxima that rise all the way, no peak
    c = Case((4, 2, 64), [900, 431], [1, 1], block=16, seed=11)
    for b, n in enumerate(c.lens_l):
        blk, row = c.at(b, 0, n)
        w = {"first": torch.zeros(n), "last": torch.zeros(n), "rising": torch.linspace(-8, 8, n),
             "equal": torch.zeros(n)}[peak].cuda()
        if peak == "first":
            w[0] = 20
        if peak == "last":
            w[-1] = 20
        c.k[blk, :, row] = (w[:, None, None] * torch.ones(n, c.hkv, c.d, device="cuda")).to(BF)
    c.q.fill_(1.0)
    c.check(kind, c.run(kind))


def test_causal_rows_do_not_see_later_ones():
    # NaN and infinities in the later tokens' own values and keys: the earlier
    # tokens of the same chunk stay as they were, bit for bit
    for heads, n, poison in (((8, 2, 64), 200, 150), ((4, 4, 128), 300, 1), ((8, 1, 64), 40, 39)):
        c = Case(heads, [n, 64], [n, 64], block=32, seed=12)
        clean, clean_lse = c.run("prefill")
        blk, row = c.at(0, poison, n)
        c.v[blk[0], :, row[0]] = math.nan
        c.v[blk[-1], 0, row[-1]] = math.inf
        c.k[blk[0], :, row[0], 0] = math.inf
        out, lse = c.run("prefill")
        keep = torch.ones(c.n, dtype=torch.bool, device="cuda")
        keep[poison:n] = False
        assert torch.isfinite(clean).all()
        ro, rl, A, err = Case.reference(c)
        tol = 2.0 ** -8 * ro.abs() + (2 * err + 2.0 ** -14 + WEIGHT["prefill"])[..., None] * A
        assert ((out.double() - ro).abs() <= tol)[keep].all()
        assert torch.equal(lse[keep], clean_lse[keep])
        assert torch.isnan(out[poison:n]).any(-1).all()


def test_infinite_scores():
    # a key whose score is -inf has no weight; +inf and NaN make the row NaN
    c = Case((2, 1, 64), [300], [1], block=16, seed=13)
    c.q.fill_(1.0)
    blk, row = c.at(0, 0, 300)
    for kind in ("decode", "prefill"):
        c.k[blk[40], :, row[40]] = -math.inf
        out, lse = c.run(kind)
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
        c.k[blk[40], :, row[40]] = math.inf
        assert torch.isnan(c.run(kind)[0]).all()
        c.k[blk[40], :, row[40]] = 0.0


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_strides_and_given_outputs(kind):
    c = Case((6, 3, 64), [200, 90, 33], [1, 1, 1], block=16, seed=14)
    plain, plain_lse = c.run(kind)
    wide = torch.randn(c.n, 8, 3, 64, device="cuda").to(BF)
    wide[:, 1:7, 1] = c.q
    q = wide[:, 1:7, 1]  # token stride 8 * 3 * 64, head stride 3 * 64
    room = torch.full((c.hq, c.n + 2, 64), 7.0, dtype=BF, device="cuda")
    out = room.transpose(0, 1)[1:1 + c.n]  # heads first in memory
    c.q, q_was = q, c.q
    got, lse = c.run(kind, out=out)
    c.q = q_was
    assert got is out and torch.equal(out, plain) and torch.equal(lse, plain_lse)
    assert (room[:, 0] == 7).all() and (room[:, -1] == 7).all()


@pytest.mark.parametrize("kind", ["append", "prefill"])
def test_padding_rows_stay(kind):
    # tokens behind the last sequence's, as in a batch padded to a fixed size
    c = Case((4, 2, 64), [40, 21], [7, 5], block=16, seed=15)
    pad = 9
    q = torch.cat([c.q, torch.full((pad, 4, 64), math.nan, dtype=BF, device="cuda")])
    out = torch.full((c.n + pad, 4, 64), 3.0, dtype=BF, device="cuda")
    if kind == "prefill":
        want, _ = c.run("prefill")
        got, lse = c.cache.prefill(q, c.lens, c.cu, out=out, return_lse=True)
        assert torch.equal(got[:c.n], want)
    else:
        kv = torch.randn(c.n + pad, 2, 64, device="cuda").to(BF)
        before = c.k.clone(), c.v.clone()
        c.cache.append(q, kv, kv, c.lens, c.cu, theta=1e4, q_out=out)
        for pool, was in zip((c.k, c.v), before):
            same = (pool.view(torch.int16) == was.view(torch.int16)).all(-1).all(1)  # [block][row]
            assert int((~same).sum()) == c.n
    assert (out[c.n:] == 3).all()
    c.cache.check()


def rotated(x, pos, theta):
    if theta == 0:
        return x.double()
    half = x.shape[-1] // 2
    a = pos.double()[:, None, None] * theta ** (-torch.arange(half, device="cuda",
                                                              dtype=torch.float64) / half)
    lo, hi = x[..., :half].double(), x[..., half:].double()
    return torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1)


def close_rotated(got, x, pos, theta):
    want = rotated(x, pos, theta)
    half = x.shape[-1] // 2
    norm = x.double().unflatten(-1, (2, half)).norm(dim=-2).repeat(1, 1, 2)
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -20 * norm
    assert ((got.double() - want).abs() <= tol).all(), (got.double() - want).abs().max()


@pytest.mark.parametrize("src", [BF, torch.float32])
@pytest.mark.parametrize("heads", [(4, 2, 64), (16, 4, 128), (7, 7, 64)])
@pytest.mark.parametrize("block", [0, 16, 256])
@pytest.mark.parametrize("lens,new", [([1], [1]), ([300, 17, 0, 1, 64], [5, 17, 0, 1, 33]),
                                      ([1000, 900], [1, 1]), ([3, 40], [5, 40])])
def test_append(src, heads, block, lens, new):
    stored = [max(0, n - m) for n, m in zip(lens, new)]
    c = Case(heads, lens, new, block=block, seed=16, stored=stored, fill=0.5)
    q, k, v = (torch.randn(c.n, h, c.d, generator=c.g, device="cuda").to(src)
               for h in (c.hq, c.hkv, c.hkv))
    before = c.k.clone(), c.v.clone()
    theta = 5e5
    got = c.cache.append(q, k, v, c.lens, None if all(m == 1 for m in new) else c.cu, theta=theta)
    assert got.dtype == BF and got.shape == q.shape
    expect_v, touched = before[1].clone(), torch.zeros(c.k.shape[0], c.k.shape[2], dtype=torch.bool,
                                                       device="cuda")
    for b, (n, m) in enumerate(zip(lens, new)):
        skip = max(0, m - n)  # tokens below position zero
        t = slice(c.cu_l[b] + skip, c.cu_l[b + 1])
        pos = torch.arange(n - m + skip, n, device="cuda")
        close_rotated(got[t], q[t], pos, theta)
        blk, row = c.at(b, n - m + skip, n)
        close_rotated(c.k[blk, :, row], k[t], pos, theta)
        expect_v[blk, :, row] = v[t].to(BF)
        touched[blk, row] = True
    assert torch.equal(c.v, expect_v)
    assert torch.equal(c.k.transpose(1, 2)[~touched], before[0].transpose(1, 2)[~touched])
    c.cache.check()


@pytest.mark.parametrize("theta", [0.0, 1.0, 1e4, 5e5, 1e8])
def test_append_far_positions(theta):
    # one token at a position where an angle in 32 bits would be off by radians;
    # nothing but the table says how long the cache is
    n, block = 16_000_000, 4096
    pages = -(-n // block)
    k = torch.zeros(2, 2, block, 64, dtype=BF, device="cuda")
    v = torch.zeros_like(k)
    table = torch.full((1, pages), -1, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    x = torch.randn(1, 2, 64, generator=gen(17), device="cuda")
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    cache = KVCache(k, v, table)
    q = cache.append(x, x, x, lens, theta=theta)
    close_rotated(q, x, lens - 1, theta)
    assert torch.equal(k[1, :, (n - 1) % block], q[0])
    cache.check()


def test_append_without_queries_and_in_place():
    c = Case((4, 2, 64), [20, 9], [6, 9], block=16, seed=18, fill=0.0)
    fused = torch.randn(c.n, 8 * 64, generator=c.g, device="cuda").to(BF)
    q, k, v = (fused[:, i:j].unflatten(1, (-1, 64)) for i, j in ((0, 256), (256, 384), (384, 512)))
    want_q, was = c.cache.append(q, k, v, c.lens, c.cu, theta=1e4), (c.k.clone(), c.v.clone())
    c.k.zero_()
    c.v.zero_()
    assert c.cache.append(None, k, v, c.lens, c.cu, theta=1e4) is None
    # (rows that were there before are gone; the new ones are the same)
    for b in range(2):
        blk, row = c.at(b, c.lens_l[b] - c.new_l[b], c.lens_l[b])
        assert torch.equal(c.k[blk, :, row], was[0][blk, :, row])
        assert torch.equal(c.v[blk, :, row], was[1][blk, :, row])
    got = c.cache.append(q, k, v, c.lens, c.cu, theta=1e4, q_out=q)
    assert got is q and torch.equal(q, want_q)


def test_offsets_beyond_32_bits():
    # pools of 2^31 + elements each; the sequences use the first and last blocks
    heads, block = (8, 8, 64), 4096
    n_blocks = (1 << 31) // (8 * block * 64) + 3
    c = Case(heads, [5000, 4097, 700], [5000, 1, 300], block=block, seed=19, stored=[0, 0, 0])
    k = torch.empty(n_blocks, 8, block, 64, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    table = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    table[0, 0], table[0, 1], table[1, 0], table[1, 1], table[2, 0] = \
        n_blocks - 1, 0, 1, n_blocks - 2, n_blocks - 3
    c.k, c.v, c.table, c.cache = k, v, table, KVCache(k, v, table)
    for b, n in enumerate(c.lens_l):
        x = torch.randn(n, 8, 64, generator=c.g, device="cuda")
        y = torch.randn(n, 8, 64, generator=c.g, device="cuda")
        one = torch.tensor([n], dtype=torch.int32, device="cuda")
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        KVCache(k, v, table[b:b + 1]).append(None, x, y, one, cu, theta=1e4)
        K, V = c.rows(b)
        assert torch.equal(V, y.to(BF).double())
        close_rotated(K, x, torch.arange(n, device="cuda"), 1e4)
    c.check("prefill", c.run("prefill"))
    c.q = c.q[:3].contiguous()
    c.new_l, c.cu_l, c.n = [1, 1, 1], [0, 1, 2, 3], 3
    c.check("decode", c.run("decode"))


def test_bad_contents_are_reported():
    def broken(change):
        c = Case((4, 2, 64), [100, 60], [1, 1], block=16, seed=20)
        change(c)
        return c

    def page(c):
        c.table[0, 2] = c.k.shape[0]

    def negative_page(c):
        c.table[1, 3] = -5

    def too_long(c):
        c.lens[0] = c.table.shape[1] * 16 + 1

    def negative(c):
        c.lens[1] = -3

    for change in (page, negative_page, too_long, negative):
        for kind in ("decode", "prefill"):
            c = broken(change)
            c.cache.check()
            c.run(kind)
            with pytest.raises(MkError) as e:
                c.cache.check()
            assert e.value.status == MK_ERR_INVALID_ARG
            c.cache.check()  # reported once
    # an append checks the rows it writes
    for change in (lambda c: c.table.__setitem__((0, 99 // 16), -1), too_long, negative):
        c = broken(change)
        kv = torch.zeros(2, 2, 64, dtype=BF, device="cuda")
        c.cache.append(c.q, kv, kv, c.lens, theta=1e4)
        with pytest.raises(MkError):
            c.cache.check()


def test_refusals():
    c = Case((4, 2, 64), [40, 20], [1, 1], block=16, seed=21)
    kv = torch.zeros(2, 2, 64, dtype=BF, device="cuda")
    f32 = c.q.float()
    with pytest.raises(ValueError, match="q:"):
        c.cache.decode(f32, c.lens)
    with pytest.raises(ValueError, match="q:"):
        c.cache.decode(c.q[..., :32], c.lens)
    with pytest.raises(ValueError, match="q:"):
        c.cache.decode(c.q.cpu(), c.lens)
    with pytest.raises(ValueError, match="lens"):
        c.cache.decode(c.q, c.lens.long())
    with pytest.raises(ValueError, match="cu"):
        c.cache.decode(c.q[:1], c.lens)
    with pytest.raises(ValueError, match="cu"):
        c.cache.prefill(c.q, c.lens, None)
    with pytest.raises(ValueError, match="cu"):
        c.cache.prefill(c.q, c.lens, c.cu[:2])
    with pytest.raises(ValueError, match="cache of 2"):
        c.cache.decode(c.q, torch.ones(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="out:"):
        c.cache.decode(c.q, c.lens, out=f32)
    with pytest.raises(ValueError, match="v:"):
        c.cache.append(c.q, kv, kv.float(), c.lens, theta=1e4)
    with pytest.raises(ValueError, match="q:"):
        c.cache.append(f32, kv, kv, c.lens, theta=1e4)
    with pytest.raises(ValueError, match="backward"):
        c.cache.decode(c.q.clone().requires_grad_(), c.lens)
    with pytest.raises(ValueError):
        KVCache(c.k, c.v[:, :1], c.table)
    with pytest.raises(ValueError):
        KVCache(c.k.transpose(1, 2), c.v.transpose(1, 2), c.table)
    with pytest.raises(ValueError):
        KVCache(c.k, c.v, c.table.long())
    with pytest.raises(MkError):  # heads that do not divide
        c.cache.decode(torch.zeros(2, 3, 64, dtype=BF, device="cuda"), c.lens)
    with pytest.raises(MkError):  # rows off the 16-byte boundaries
        odd = torch.zeros(2 * 260, dtype=BF, device="cuda")[4:4 + 516].as_strided((2, 4, 64), (260, 64, 1))
        c.cache.decode(odd, c.lens)
    with pytest.raises(MkError):
        c.cache.append(c.q, kv, kv, c.lens, theta=-1.0)


def test_empty_calls():
    c = Case((4, 2, 64), [40, 20], [1, 1], block=16, seed=22)
    none, cu = c.q[:0], torch.zeros(3, dtype=torch.int32, device="cuda")
    out, lse = c.cache.prefill(none, c.lens, cu, return_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    kv = torch.zeros(0, 2, 64, dtype=BF, device="cuda")
    assert c.cache.append(none, kv, kv, c.lens, cu, theta=1e4).shape == (0, 4, 64)
    assert c.cache.decode(none, c.lens[:0]).shape == (0, 4, 64)


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_other_stream(kind):
    c = Case((32, 8, 64), [3000, 2000], [1, 1], block=16, seed=23)
    want = c.run(kind)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        got = c.run(kind, stream=side)
        again = c.run(kind)  # on the current stream at the same time
        side.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(again[0], want[0])


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_repeats_are_bit_equal(kind):
    c = Case((32, 8, 64), [3000, 1, 0, 777, 2111], [1, 1, 1, 1, 1], block=64, seed=24)
    want = c.run(kind)
    for _ in range(10):
        got = c.run(kind)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_graph_of_a_decode_step_follows_lens():
    # append + decode captured once, replayed while the sequences grow; a second
    # graph of the same calls replays at the same time on another stream
    c = Case((8, 2, 64), [40, 0, 129], [1, 1, 1], block=16, seed=25, stored=[40, 0, 129])
    pages = torch.arange(c.k.shape[0], device="cuda", dtype=torch.int32)
    c.k.nan_to_num_(0.0)
    c.v.nan_to_num_(0.0)
    table = pages[:(c.k.shape[0] // 3) * 3].reshape(3, -1).contiguous()
    c.table, c.cache = table, KVCache(c.k, c.v, table)
    lens = torch.tensor([40, 0, 129], dtype=torch.int32, device="cuda")
    q, k, v = (torch.zeros(3, h, 64, dtype=BF, device="cuda") for h in (8, 2, 2))

    def step():
        lens.add_(1)
        qr = c.cache.append(q, k, v, lens, theta=1e4)
        return qr, c.cache.decode(qr, lens, return_lse=True)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qr, got = step()
    lens.copy_(torch.tensor([40, 0, 129]))
    other = Case((32, 8, 64), [5000], [1], block=16, seed=26)
    want = other.run("decode")
    graph2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph2):
        got2 = other.run("decode")
    for i in range(6):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=c.g, device="cuda"))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph2.replay()
        graph.replay()
        torch.cuda.synchronize()
        c.lens_l = lens.tolist()
        assert c.lens_l == [41 + i, 1 + i, 130 + i]
        c.q = qr
        c.check("decode", got)
        assert torch.equal(got2[0], want[0])


def test_shared_prefix_blocks():
    # two sequences whose first blocks are the same ones
    c = Case((8, 2, 64), [100, 100], [1, 1], block=16, seed=27)
    c.table[1, :4] = c.table[0, :4]
    c.check("decode", c.run("decode"))
    c.check("prefill", c.run("prefill"))


@pytest.mark.parametrize("kind", ["decode", "prefill"])
def test_query_orders(kind):
    # queries with heads first in memory, and one row shared by all heads
    c = Case((6, 3, 64), [200, 90, 33], [1, 1, 1], block=16, seed=28)
    plain, plain_lse = c.run(kind)
    c.q = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    got, lse = c.run(kind)
    assert torch.equal(got, plain) and torch.equal(lse, plain_lse)
    c.q = c.q[:, :1].expand(-1, 6, -1)
    assert c.q.stride(1) == 0
    c.check(kind, c.run(kind))
    c = Case((1, 1, 128), [40], [1], block=0, seed=29)  # a single row
    c.check(kind, c.run(kind))


def test_attention_workspace_is_checked():
    from decode_megakernel_sm_gb300 import _lib as L
    c = Case((4, 2, 64), [40, 20], [1, 1], block=16, seed=30)
    view = L.mk_kv_view(c.k.data_ptr(), c.v.data_ptr(), *c.k.shape, c.table.data_ptr(),
                        c.table.shape[1])
    rows = L.mk_rows(c.q.data_ptr(), 256, 64)
    out = torch.empty_like(c.q)
    to = L.mk_rows(out.data_ptr(), 256, 64)
    for decode, f, cu in ((True, L.mk_attn_decode, None), (False, L.mk_attn_prefill, c.cu.data_ptr())):
        need = L.mk_attn_workspace_bytes(decode, 2, 2, 4, 2, 64)
        assert need > 0
        ws = torch.empty(need + 256, dtype=torch.uint8, device="cuda")
        bt = L.mk_kv_batch(2, 2, c.lens.data_ptr(), cu)
        for p, n in ((None, need), (ws.data_ptr(), need - 1), (ws.data_ptr() + 16, need)):
            with pytest.raises(MkError) as e:
                f(view, bt, 4, rows, 0.125, to, None, p, n)
            assert e.value.status == MK_ERR_INVALID_ARG
        f(view, bt, 4, rows, 0.125, to, None, ws.data_ptr(), need)
        ref, _, A, err = c.reference(0.125)
        assert ((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -7 * A).all()


@pytest.mark.parametrize("heads", [(2, 2, 64), (9, 3, 128), (64, 1, 64), (128, 1, 128), (30, 2, 64)])
def test_prefill_head_groups(heads):
    # group sizes that fill a tile of 128 rows exactly, nearly, and with one token
    c = Case(heads, [190, 5, 400], [190, 5, 33], block=32, seed=31)
    c.check("prefill", c.run("prefill"))


def test_prefill_refuses_wide_groups():
    c = Case((129, 1, 64), [5], [5], block=16, seed=32)
    with pytest.raises(MkError):
        c.run("prefill")


@pytest.mark.parametrize("lens,new", [
    ([5000] * 3, [5000, 1, 77]),           # jobs cut into many parts
    ([1300] * 40, [40] * 40),              # many short chunks over long caches
    ([20000, 3, 3, 3], [9, 3, 2, 1]),      # one sequence holds all the work
    ([129] * 64, [129] * 64),              # more jobs than SMs, each two units
])
@pytest.mark.parametrize("heads", [(8, 2, 64), (4, 2, 128)])
def test_prefill_cuts(heads, lens, new):
    c = Case(heads, lens, new, block=64, seed=33)
    c.check("prefill", c.run("prefill"))


@pytest.mark.parametrize("heads", [(8, 2, 64), (4, 2, 128)])
def test_prefill_runs_of_jobs_without_rows(heads):
    """Most sequences of a padded batch hold no rows at all: a block's piece of the
    work then has runs of jobs with nothing to multiply between the others."""
    lens = [(40 + 7 * b if b % 10 == 3 else 0) for b in range(600)]
    c = Case(heads, lens, [33] * 600, block=16, seed=51)
    c.check("prefill", c.run("prefill"))


@pytest.mark.parametrize("kind", ["append", "prefill"])
@pytest.mark.parametrize("cu", [[0, 9, 4, 12], [0, 4, 9, 13], [0, 4, 2 ** 31 - 1, 12], [0, -2 ** 31, 7, 12],
                                [-3, 4, 9, 12]], ids=str)
def test_offsets_that_fall_or_leave_the_rows(kind, cu):
    """Bad offsets touch nothing outside the sequences' rows, and are reported."""
    c = Case((4, 2, 64), [40, 21, 33], [4, 5, 3], block=16, seed=52)
    bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
    before = c.k.clone()
    if kind == "append":
        kv = torch.randn(c.n, 2, 64, device="cuda").to(BF)
        c.cache.append(c.q, kv, kv, c.lens, bad, theta=1e4)
        own = torch.zeros(c.k.shape[0], c.k.shape[2], dtype=torch.bool, device="cuda")
        for b, n in enumerate(c.lens_l):
            own[c.at(b, 0, n)] = True
        same = (c.k.view(torch.int16) == before.view(torch.int16)).all(-1).all(1)
        assert same[~own].all()
    else:
        c.cache.prefill(c.q, c.lens, bad)
    with pytest.raises(MkError) as e:
        c.cache.check()
    assert e.value.status == MK_ERR_INVALID_ARG


def test_rows_before_the_first_sequence_are_padding():
    c = Case((4, 2, 64), [40, 21], [7, 5], block=16, seed=53)
    want = c.run("prefill")[0]
    q = torch.cat([torch.full_like(c.q[:3], math.nan), c.q])
    cu = c.cu + 3
    out = torch.full((c.n + 3, 4, 64), 3.0, dtype=BF, device="cuda")
    c.cache.prefill(q, c.lens, cu, out=out)
    assert torch.equal(out[3:], want) and (out[:3] == 3).all()
    kv = torch.randn(c.n + 3, 2, 64, device="cuda").to(BF)
    other = Case((4, 2, 64), [40, 21], [7, 5], block=16, seed=53)
    out.fill_(3.0)
    got = c.cache.append(q, kv, kv, c.lens, cu, theta=1e4, q_out=out)
    ref = other.cache.append(c.q, kv[3:], kv[3:], other.lens, other.cu, theta=1e4)
    assert torch.equal(got[3:], ref) and (got[:3] == 3).all()
    for a, b in ((c.k, other.k), (c.v, other.v)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    c.cache.check()


def test_first_calls_may_be_captured():
    """A process whose first use of the operators is inside a capture."""
    code = """
import torch
from decode_megakernel_sm_gb300 import KVCache
def case(d):
    torch.manual_seed(d)
    k = torch.zeros(2, 2, 300, d, dtype=torch.bfloat16, device="cuda")
    new = [torch.randn(200, h, d, device="cuda").bfloat16() for h in (8, 2, 2)]
    one = torch.randn(2, 8, d, device="cuda").bfloat16()
    lens = torch.tensor([120, 80], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 120, 200], dtype=torch.int32, device="cuda")
    cache = KVCache(k, k.clone())
    def run():
        q = cache.append(*new, lens, cu, theta=1e4)
        return cache.prefill(q, lens, cu), cache.decode(one, lens)
    return cache, run
cases = [case(64), case(128)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = [run() for _, run in cases]
graph.replay()
torch.cuda.synchronize()
for (cache, run), g in zip(cases, got):
    for a, b in zip(run(), g):
        assert a.abs().sum() > 0 and torch.equal(a, b)
    cache.check()
"""
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300,
                   cwd=pathlib.Path(__file__).resolve().parents[1])


def test_calls_at_once_on_two_streams():
    cases = [Case((16, 4, 128), [900, 3000], [900, 200], block=64, seed=54),
             Case((32, 8, 64), [2500, 400], [300, 400], block=16, seed=55)]
    want = [c.run("prefill") for c in cases]
    steps = [(c, torch.randn(2, c.hq, c.d, generator=c.g, device="cuda").to(BF)) for c in cases]
    want_step = [c.cache.decode(q, c.lens) for c, q in steps]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for (c, q), w, ws, s in zip(steps, want, want_step, streams):
            got.append((w, c.run("prefill", stream=s)))
            got.append(((ws,), (c.cache.decode(q, c.lens, stream=s),)))
    torch.cuda.synchronize()
    for w, g in got:
        assert all(torch.equal(a, b) for a, b in zip(w, g))
    cases[0].cache.check()


def test_prefill_redoes_rows_of_a_long_cache():
    # a NaN among the last token's own values: all other rows of its tile are redone
    c = Case((8, 2, 64), [100_000], [32], block=64, seed=56)
    blk, row = c.at(0, 99_999, 100_000)
    ro, rl, A, err = c.reference()
    c.v[blk, 0, row, 5] = math.nan
    out, _ = c.run("prefill")
    tol = 2.0 ** -8 * ro.abs() + (2 * err + 2.0 ** -14 + WEIGHT["prefill"])[..., None] * A
    ok = (out.double() - ro).abs() <= tol
    assert ok[:31].all() and ok[31, 4:].all() and torch.isnan(out[31, :4, 5]).all()
    assert ok[31, :4].sum() == 4 * 63
    c.cache.check()


def test_outputs_that_overlap_or_name_the_queries_are_refused():
    c = Case((4, 2, 64), [40, 20], [1, 1], block=16, seed=57)
    with pytest.raises(MkError):
        c.cache.decode(c.q, c.lens, out=c.q)
    with pytest.raises(MkError):
        c.cache.decode(c.q, c.lens, out=torch.empty(1, 4, 64, dtype=BF, device="cuda").expand(2, 4, 64))
    with pytest.raises(MkError):
        c.cache.decode(c.q, c.lens, scale=math.nan)
    with pytest.raises(ValueError, match="backward"):
        KVCache(c.k.clone().requires_grad_(), c.v, c.table)
    # queries may be spread out from fewer rows
    one = c.q[:1].expand(2, 4, 64)
    assert torch.equal(c.cache.decode(one, c.lens), c.cache.decode(one.contiguous(), c.lens))
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    assert torch.equal(c.cache.prefill(one, c.lens, cu), c.cache.prefill(one.contiguous(), c.lens, cu))


def widened(c, rows=1 << 20):
    """The same cache through a table that could name far longer sequences, as a
    server's does: the choice of a kernel looks at what the table can hold."""
    pages = max(c.table.shape[1], rows // c.block)
    table = torch.full((c.table.shape[0], pages), -1, dtype=torch.int32, device="cuda")
    table[:, :c.table.shape[1]] = c.table
    return KVCache(c.k, c.v, table)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("lens", LENS + [[2040, 3, 700], [130] * 40], ids=str)
def test_decode_of_wide_tables(heads, lens):
    c = Case(heads, lens, block=16, seed=58)
    c.check("decode", c.run("decode"))
    c.cache = widened(c)
    c.check("decode", c.run("decode"))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("heads", [(8, 2, 64), (32, 2, 128), (12, 1, 128), (33, 1, 64)])
def test_decode_keeps_infinite_and_nan_values_to_their_dims(heads, wide):
    c = Case(heads, [700, 65, 1], block=16, seed=59)
    if wide:
        c.cache = widened(c)
    want, want_lse = c.run("decode")
    ro, rl, A, err = c.reference()
    for b, at, dim, value in ((0, 3, 7, math.inf), (0, 400, 9, math.nan), (1, 64, 0, -math.inf)):
        blk, row = c.at(b, at, at + 1)
        c.v[blk[0], 0, row[0], dim] = value
    out, lse = c.run("decode")
    assert torch.equal(lse[2], want_lse[2]) and torch.equal(out[2], want[2])
    assert ((lse - want_lse).abs() <= 2.0 ** -18 * (1 + want_lse.abs()) + 2 * err).all()
    g = c.hq // c.hkv
    tol = 2.0 ** -8 * ro.abs() + (2 * err + 2.0 ** -14 + WEIGHT["decode"])[..., None] * A
    ok = (out.double() - ro).abs() <= tol
    spoilt = torch.zeros_like(ok)
    spoilt[0, :g, 7] = spoilt[0, :g, 9] = spoilt[1, :g, 0] = True
    assert ok[~spoilt].all()
    assert (out[0, :g, 7] == math.inf).all() and torch.isnan(out[0, :g, 9]).all()
    assert (out[1, :g, 0] == -math.inf).all()
    c.cache.check()


def test_batches_of_padding_alone():
    # no sequence has a new token: nothing is written
    c = Case((4, 2, 64), [40, 0], [3, 4], block=16, seed=60)
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = torch.full((7, 4, 64), 3.0, dtype=BF, device="cuda")
    c.cache.prefill(c.q, c.lens, cu, out=out)
    before = c.k.clone(), c.v.clone()
    kv = torch.randn(7, 2, 64, device="cuda").to(BF)
    c.cache.append(c.q, kv, kv, c.lens, cu, theta=1e4, q_out=out)
    assert (out == 3).all()
    for pool, was in zip((c.k, c.v), before):
        assert torch.equal(pool.view(torch.int16), was.view(torch.int16))
    c.cache.check()
