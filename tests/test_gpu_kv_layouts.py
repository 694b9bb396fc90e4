"""KV-cache operators on rows in other orders than [token][head][dim], with many new
tokens per sequence, and appends on a stream of their own.

Results are compared bit by bit with the same call on dense rows where the
arithmetic is the same, and with the 64-bit reference (tolerances: test_gpu_kv_ops)."""
import pytest
import torch

from tests.test_gpu_kv_ops import BF, Case, close_rotated

pytestmark = pytest.mark.gpu

HEADS = [(6, 3, 64), (8, 2, 128), (32, 8, 64), (5, 1, 64)]
CHUNKS = [([200, 90, 33], [200, 41, 1]), ([1500], [1500]), ([3000, 0, 700], [9, 0, 300])]


def orders(x):
    """x, [tokens][heads][dim], in layouts that a caller may have: name -> equal rows."""
    n, h, d = x.shape
    fused = torch.full((n, h + 5, d), 9.0, dtype=x.dtype, device="cuda")
    fused[:, 2:2 + h] = x
    apart = torch.full((n, h, 3, d), 9.0, dtype=x.dtype, device="cuda")
    apart[:, :, 1] = x
    heads_first = torch.full((h, n + 3, d), 9.0, dtype=x.dtype, device="cuda")
    heads_first[:, 1:1 + n] = x.transpose(0, 1)
    return {"fused": fused[:, 2:2 + h], "apart": apart[:, :, 1],
            "heads first": heads_first.transpose(0, 1)[1:1 + n]}


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("lens,new", CHUNKS, ids=str)
def test_prefill_of_strided_rows(heads, lens, new):
    c = Case(heads, lens, new, block=16, seed=70)
    dense = c.run("prefill")
    c.check("prefill", dense)
    for name, q in orders(c.q).items():
        assert torch.equal(q, c.q)
        got = c.cache.prefill(q, c.lens, c.cu, return_lse=True)
        assert torch.equal(got[0], dense[0]) and torch.equal(got[1], dense[1]), name
    for name, out in orders(torch.zeros_like(c.q)).items():
        whole = out._base.clone()
        got, lse = c.run("prefill", out=out)
        assert got is out and torch.equal(out, dense[0]) and torch.equal(lse, dense[1]), name
        out.zero_()
        assert torch.equal(out._base, whole), name  # nothing beside the rows
    c.cache.check()


@pytest.mark.parametrize("heads", [(6, 3, 64), (8, 2, 128)])
def test_prefill_of_rows_shared_by_heads_or_tokens(heads):
    c = Case(heads, [200, 90], [150, 41], block=32, seed=71)
    for q in (c.q[:, :1].expand(-1, heads[0], -1), c.q[:1].expand(c.n, -1, -1)):
        c.q = q
        c.check("prefill", c.run("prefill"))


@pytest.mark.parametrize("src", [BF, torch.float32])
@pytest.mark.parametrize("heads", HEADS)
def test_append_of_strided_rows(src, heads):
    lens, new = [300, 17, 0, 64], [250, 17, 0, 33]
    stored = [n - m for n, m in zip(lens, new)]
    c = Case(heads, lens, new, block=16, seed=72, stored=stored, fill=0.5)
    before = c.k.clone(), c.v.clone()
    q, k, v = (torch.randn(c.n, h, c.d, generator=c.g, device="cuda").to(src)
               for h in (c.hq, c.hkv, c.hkv))
    want = c.cache.append(q, k, v, c.lens, c.cu, theta=1e4)
    cached = c.k.clone(), c.v.clone()
    pos = torch.cat([torch.arange(n - m, n, device="cuda") for n, m in zip(lens, new)])
    close_rotated(want, q, pos, 1e4)
    for name in orders(q):
        c.k.copy_(before[0])
        c.v.copy_(before[1])
        out = orders(torch.zeros(c.n, c.hq, c.d, dtype=BF, device="cuda"))[name]
        whole = out._base.clone()
        got = c.cache.append(orders(q)[name], orders(k)[name], orders(v)[name], c.lens, c.cu,
                             theta=1e4, q_out=out)
        assert got is out and torch.equal(out, want), name
        assert torch.equal(c.k, cached[0]) and torch.equal(c.v, cached[1]), name
        out.zero_()
        assert torch.equal(out._base, whole), name
    if src is BF:
        for name, x in orders(q).items():  # in place
            whole = x._base.clone()
            assert c.cache.append(x, k, v, c.lens, c.cu, theta=1e4, q_out=x) is x
            assert torch.equal(x, want), name
            x.copy_(q)
            assert torch.equal(x._base, whole), name
    c.cache.check()


def test_append_on_a_stream_of_its_own():
    c = Case((32, 8, 64), [2000, 900], [1500, 900], block=16, seed=73, stored=[500, 0], fill=0.5)
    before = c.k.clone(), c.v.clone()
    q, k, v = (torch.randn(c.n, h, c.d, generator=c.g, device="cuda").to(BF) for h in (32, 8, 8))
    want = c.cache.append(q, k, v, c.lens, c.cu, theta=1e4)
    cached = c.k.clone(), c.v.clone()
    other = Case((16, 4, 128), [3000], [3000], block=64, seed=74)
    want_other = other.run("prefill")
    side = torch.cuda.Stream()
    for _ in range(5):
        c.k.copy_(before[0])
        c.v.copy_(before[1])
        torch.cuda.synchronize()
        got = c.cache.append(q, k, v, c.lens, c.cu, theta=1e4, stream=side)
        again = other.run("prefill")  # on the current stream at the same time
        side.synchronize()
        assert torch.equal(got, want) and torch.equal(c.k, cached[0]) and torch.equal(c.v, cached[1])
        assert torch.equal(again[0], want_other[0]) and torch.equal(again[1], want_other[1])
    c.cache.check()


@pytest.mark.parametrize("heads,tokens", [((32, 8, 64), n) for n in (950, 1090, 1150, 1200)] +
                         [((16, 4, 128), n) for n in (1090, 2000, 2300)])
def test_prefill_of_about_as_many_jobs_as_blocks(heads, tokens):
    c = Case(heads, [tokens], [tokens], block=64, seed=75)
    c.check("prefill", c.run("prefill"))
