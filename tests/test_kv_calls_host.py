"""The cache operators' host code over a stand-in for the CUDA runtime: which calls are
launched, which are refused, and what becomes of the runtime's errors."""
import shutil

import pytest

from decode_megakernel_sm_gb300 import _lib as L
from tests.kv_fake import Fake

pytestmark = pytest.mark.skipif(not (shutil.which("nvcc") and shutil.which("g++")),
                                reason="builds the host code")

G = 1 << 30
K, V, TABLE, LENS, CU, WS, FREE = (G * i for i in range(1, 8))  # addresses far apart


@pytest.fixture(scope="module")
def built():
    return Fake()


@pytest.fixture
def fake(built):
    built.lib.fake_reset()
    return built


def view(**kw):
    a = dict(k=K, v=V, n_blocks=8, n_kv_heads=2, block=16, head_dim=64, d_table=TABLE, table_stride=4)
    a.update(kw)
    return L.mk_kv_view(*[a[n] for n, _ in L.mk_kv_view._fields_])


POOL = 8 * 2 * 16 * 64 * 2  # bytes of the view's pools


def batch(n=7, batch=2, cu=CU):
    return L.mk_kv_batch(batch, n, LENS, cu)


def rows(p=FREE, ts=256, hs=64):
    return L.mk_rows(p, ts, hs)


def append(fake, q=None, k=None, v=None, qo=None, src=L.MK_SRC_BF16, kv=None, hq=4, n=7, theta=1e4):
    return fake.lib.mk_kv_append(kv or view(), batch(n), hq, q or rows(), k or rows(FREE + 4 * G),
                                 v or rows(FREE + 5 * G), src, qo or rows(FREE + G), theta, None)


def attn(fake, kind, q=None, out=None, lse=None, ws=WS, n=7, hq=4, scale=0.125, kv=None):
    decode = kind == "decode"
    bt = batch(2 if decode else n, cu=None if decode else CU)
    return getattr(fake.lib, f"mk_attn_{kind}")(kv or view(), bt, hq, q or rows(), scale,
                                                out or rows(FREE + G), lse, ws, 1 << 28, None)


KINDS = ["decode", "prefill"]
# q and out as [n][4][64] bf16 in one buffer, out at a distance: rows that share memory
SHARING = {
    "shifted by a token": (rows(), rows(FREE + 512)),
    "shifted by half a token": (rows(), rows(FREE + 256)),
    "before it": (rows(FREE + 512), rows(FREE)),
    "slices that meet": (rows(ts=512), rows(FREE + 3 * 128, ts=512)),
    "interleaved heads that meet": (rows(ts=512, hs=128), rows(FREE + 128 + 64, ts=512, hs=128)),
    "other strides": (rows(), rows(FREE, ts=512, hs=64)),
    "heads first": (rows(ts=64, hs=448), rows(FREE + 128, ts=64, hs=448)),
    "one row for all": (rows(FREE + 512, ts=0), rows(FREE)),
}
APART = {
    "far apart": (rows(), rows(FREE + G)),
    "end to end": (rows(), rows(FREE + 7 * 512)),
    "slices of one row": (rows(ts=512), rows(FREE + 512, ts=512)),
    "slices the other way": (rows(FREE + 512, ts=512), rows(ts=512)),
    "heads in turn": (rows(ts=512, hs=128), rows(FREE + 128, ts=512, hs=128)),
    "heads first in turn": (rows(ts=64, hs=1024), rows(FREE + 1024, ts=64, hs=1024)),
    "heads in turn, one in four": (rows(ts=1024, hs=128), rows(FREE + 128, ts=1024, hs=256)),
    "one row for all": (rows(FREE + 8192, ts=0), rows(FREE)),
}


@pytest.mark.parametrize("name", SHARING)
def test_outputs_that_share_memory_with_the_queries_are_refused(fake, name):
    q, out = SHARING[name]
    for kind in KINDS:
        assert attn(fake, kind, q=q, out=out) == L.MK_ERR_INVALID_ARG
    if name != "one row for all":
        assert append(fake, q=q, qo=out) == L.MK_ERR_INVALID_ARG
    assert fake.launches() == []


@pytest.mark.parametrize("name", APART)
def test_outputs_beside_the_queries_are_taken(fake, name):
    q, out = APART[name]
    for kind in KINDS:
        assert attn(fake, kind, q=q, out=out) == L.MK_OK
    assert append(fake, q=q, qo=out) == L.MK_OK
    assert len(fake.launches()) >= 4


def test_queries_turn_in_place(fake):
    for r in (rows(), rows(ts=512), rows(ts=64, hs=1024)):
        assert append(fake, q=r, qo=r) == L.MK_OK
    # the same rows, read as fp32 or in another order
    assert append(fake, q=rows(), qo=rows(), src=L.MK_SRC_F32) == L.MK_ERR_INVALID_ARG
    assert append(fake, q=rows(ts=256, hs=64), qo=rows(ts=64, hs=448)) == L.MK_ERR_INVALID_ARG


def test_append_in_a_fused_projection(fake):
    # [n][4 + 2 + 2][64]: queries in place, keys and values beside them
    def part(i):
        return rows(FREE + 128 * i, ts=512)
    assert append(fake, q=part(0), qo=part(0), k=part(4), v=part(6)) == L.MK_OK
    assert append(fake, q=part(0), qo=part(2), k=part(4), v=part(6)) == L.MK_ERR_INVALID_ARG
    assert append(fake, q=rows(FREE + 2 * G), qo=part(4), k=part(4), v=part(6)) == L.MK_ERR_INVALID_ARG
    assert append(fake, q=rows(FREE + 2 * G), qo=part(2), k=part(4), v=part(6)) == L.MK_ERR_INVALID_ARG
    assert append(fake, n=1, q=part(0), qo=part(0), k=part(4), v=part(6)) == L.MK_OK


@pytest.mark.parametrize("at", [K, V, K + POOL - 256, V - 512])
def test_outputs_in_the_cache_are_refused(fake, at):
    for kind in KINDS:
        assert attn(fake, kind, out=rows(at)) == L.MK_ERR_INVALID_ARG
        assert attn(fake, kind, lse=at) == (L.MK_ERR_INVALID_ARG if at != V - 512 else L.MK_OK)
    assert append(fake, qo=rows(at)) == L.MK_ERR_INVALID_ARG


def test_outputs_at_the_cache_are_taken(fake):
    assert attn(fake, "prefill", out=rows(K + POOL)) == L.MK_OK
    assert attn(fake, "prefill", out=rows(K - 7 * 512)) == L.MK_OK
    assert attn(fake, "decode", lse=K + POOL) == L.MK_OK
    # keys that are their own values are read, not written
    assert attn(fake, "decode", kv=view(v=K)) == L.MK_OK
    assert append(fake, kv=view(v=K)) == L.MK_ERR_INVALID_ARG
    assert append(fake, kv=view(v=K + POOL - 256)) == L.MK_ERR_INVALID_ARG
    assert append(fake, kv=view(v=K + POOL)) == L.MK_OK


@pytest.mark.parametrize("kind", KINDS)
def test_scratch_and_lse_share_nothing(fake, kind):
    for ws in (FREE, FREE + G, K, V - 256, FREE + 2 * G):
        assert attn(fake, kind, ws=ws, lse=FREE + 2 * G) == L.MK_ERR_INVALID_ARG
    for lse in (FREE, FREE + G):
        assert attn(fake, kind, lse=lse) == L.MK_ERR_INVALID_ARG
    assert fake.launches() == []
    assert attn(fake, kind, lse=FREE + 2 * G) == L.MK_OK


def test_strides_of_any_size(fake):
    assert attn(fake, "decode", q=rows(FREE + G, ts=1 << 62), out=rows()) == L.MK_OK
    assert attn(fake, "decode", q=rows(ts=-256)) == L.MK_OK
    assert attn(fake, "decode", q=rows(FREE + 512, ts=-256), out=rows(FREE)) == L.MK_ERR_INVALID_ARG


@pytest.mark.parametrize("by", [1, 2, 3])
def test_vectors_off_their_alignment_are_refused(fake, by):
    """A kernel that loads an int off its 4-byte boundary faults."""
    for bt in (L.mk_kv_batch(2, 7, LENS + by, CU), L.mk_kv_batch(2, 7, LENS, CU + by)):
        assert fake.lib.mk_kv_append(view(), bt, 4, rows(), rows(FREE + 4 * G), rows(FREE + 5 * G), 0,
                                     rows(FREE + G), 1e4, None) == L.MK_ERR_INVALID_ARG
        assert fake.lib.mk_attn_prefill(view(), bt, 4, rows(), 0.125, rows(FREE + G), None, WS, 1 << 28,
                                        None) == L.MK_ERR_INVALID_ARG
    assert fake.lib.mk_attn_decode(view(), L.mk_kv_batch(2, 2, LENS + by, None), 4, rows(), 0.125,
                                   rows(FREE + G), None, WS, 1 << 28, None) == L.MK_ERR_INVALID_ARG
    odd = view(d_table=TABLE + by)
    assert append(fake, kv=odd) == L.MK_ERR_INVALID_ARG
    for kind in KINDS:
        assert attn(fake, kind, kv=odd) == L.MK_ERR_INVALID_ARG
        assert attn(fake, kind, lse=FREE + 2 * G + by) == L.MK_ERR_INVALID_ARG
    assert fake.launches() == []


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("scale", [2.5e38, -2.5e38, 3.4e38])
def test_scales_that_overflow_in_powers_of_two_are_refused(fake, kind, scale):
    # the kernels work with scale * log2 e: infinite, it makes a score of 0 NaN
    assert attn(fake, kind, scale=scale) == L.MK_ERR_INVALID_ARG
    assert fake.launches() == []
    assert attn(fake, kind, scale=2.3e38 if scale > 0 else -2.3e38) == L.MK_OK


# ---- the runtime's errors ----
WIDE = dict(table_stride=1 << 16)  # decode takes two launches for tables like this
CALLS = {
    "append": (append, 1, {}),
    "decode by clusters": (attn, 1, dict(kind="decode")),
    "decode by the line": (attn, 2, dict(kind="decode", kv=view(**WIDE))),
    "prefill": (attn, 2, dict(kind="prefill")),
    "prefill of 128 dims": (attn, 2, dict(kind="prefill", kv=view(head_dim=128), q=rows(ts=512, hs=128),
                                          out=rows(FREE + G, ts=512, hs=128))),
}
INVALID_VALUE, OUT_OF_MEMORY = 1, 2


@pytest.mark.parametrize("name", CALLS)
def test_a_failed_launch_is_its_own_calls_error(fake, name):
    call, launches, kw = CALLS[name]
    for i in range(launches):
        fake.lib.fake_reset()
        fake.fail("launch", after=i)
        assert call(fake, **kw) == L.MK_ERR_CUDA
        assert fake.lib.fake_peek() == 0  # nothing left for the next call to find
        assert len(fake.launches()) == i
        assert call(fake, **kw) == L.MK_OK
        assert len(fake.launches()) == i + launches


@pytest.mark.parametrize("name", CALLS)
def test_an_error_of_another_call_is_not_reported(fake, name):
    call, launches, kw = CALLS[name]
    fake.lib.fake_pending(OUT_OF_MEMORY)
    assert call(fake, **kw) == L.MK_OK
    assert len(fake.launches()) == launches


@pytest.mark.parametrize("failing", ["device", "attribute"])
@pytest.mark.parametrize("name", CALLS)
def test_failed_queries_launch_nothing_and_leave_nothing(fake, name, failing):
    call, launches, kw = CALLS[name]
    fake.fail(failing, error=INVALID_VALUE)
    assert call(fake, **kw) == L.MK_ERR_CUDA
    assert fake.launches() == [] and fake.lib.fake_peek() == 0
    assert call(fake, **kw) == L.MK_OK


@pytest.mark.parametrize("failing", ["copy", "sync", "launch"])
def test_a_failed_status_leaves_nothing(fake, failing):
    fake.fail(failing)
    assert fake.lib.mk_kv_status(None) == L.MK_ERR_CUDA
    assert fake.lib.fake_peek() == 0
    assert fake.lib.mk_kv_status(None) == L.MK_OK


# ---- findings ----
CONTENTS, TIMEOUT = 1, 2  # the word's bits


@pytest.mark.parametrize("bits,status", [(0, L.MK_OK), (CONTENTS, L.MK_ERR_INVALID_ARG),
                                         (TIMEOUT, L.MK_ERR_TIMEOUT), (3, L.MK_ERR_TIMEOUT)])
def test_findings_are_reported_once(fake, bits, status):
    fake.lib.fake_set(b"kv_status_word", bits)
    assert fake.lib.mk_kv_status(None) == status
    assert fake.lib.mk_kv_status(None) == L.MK_OK


@pytest.mark.parametrize("found", [0, CONTENTS])
@pytest.mark.parametrize("meanwhile", [CONTENTS, TIMEOUT])
def test_what_another_stream_finds_meanwhile_is_kept(fake, found, meanwhile):
    fake.lib.fake_set(b"kv_status_word", found)
    fake.lib.fake_poke_at_sync(b"kv_status_word", meanwhile, 1)  # behind the taking
    assert fake.lib.mk_kv_status(None) == (L.MK_ERR_INVALID_ARG if found else L.MK_OK)
    assert fake.lib.mk_kv_status(None) == (L.MK_ERR_TIMEOUT if meanwhile == TIMEOUT else L.MK_ERR_INVALID_ARG)


def test_wait_timeouts(fake):
    f = fake.lib.mk_kv_set_wait_timeout
    assert f(2 ** 62 + 1) == L.MK_ERR_INVALID_ARG
    for ns in (2 ** 62, 1, 0):
        assert f(ns) == L.MK_OK


def test_prefill_is_compiled_to_the_registers_that_it_deals_out():
    """The kernel would wait for registers that its launch does not hold, so a call
    refuses to run with any other number; the compiler's log says it beforehand."""
    import os
    import re

    from decode_megakernel_sm_gb300 import build as B
    L.lib()
    log = os.path.join(B.BUILD, "kv_ops.cu.o.log")
    if not os.path.exists(log):
        pytest.skip("the library was not built here")
    source = open(os.path.join(B.CSRC, "kv_prefill.cuh")).read()
    regs, threads = (int(re.search(rf"constexpr int {n} = (\d+);", source)[1]) for n in ("PF_REGS", "PF_THREADS"))
    dealt = [int(n) for n in re.findall(r"setmaxnreg\.(?:dec|inc)\.sync\.aligned\.u32 (\d+);", source)]
    assert 128 * dealt[0] + (threads - 128) * dealt[1] <= regs * threads
    used = re.findall(r"Compiling entry function '\w*kv_prefill_kernel\w*'.*?Used (\d+) registers",
                      open(log).read(), re.S)
    assert len(used) == 2 and all(int(n) == regs for n in used)
