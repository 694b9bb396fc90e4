"""Refusals of the KV-cache operators, on the CPU: every bad argument comes back
as a status before anything is launched."""
import ctypes as C

import pytest
import torch

from decode_megakernel_sm_gb300 import KVCache
from decode_megakernel_sm_gb300 import _lib as L

P = 1 << 20  # a pointer that nothing reads: these calls are refused first


def view(**kw):
    a = dict(k=P, v=P, n_blocks=8, n_kv_heads=2, block=16, head_dim=64, d_table=P, table_stride=4)
    a.update(kw)
    return L.mk_kv_view(*[a[n] for n, _ in L.mk_kv_view._fields_])


def batch(**kw):
    a = dict(batch=2, n_tokens=2, d_lens=P, d_cu=None)
    a.update(kw)
    return L.mk_kv_batch(*[a[n] for n, _ in L.mk_kv_batch._fields_])


def rows(p=P, ts=256, hs=64):
    return L.mk_rows(p, ts, hs)


def append(kv=None, bt=None, hq=4, q=None, k=None, v=None, src=L.MK_SRC_BF16, qo=None, theta=1e4):
    return L.lib().mk_kv_append(kv or view(), bt or batch(), hq, q or rows(), k or rows(),
                                v or rows(), src, qo or rows(), theta, None)


def attn(kind, kv=None, bt=None, hq=4, q=None, out=None, lse=None, ws=P, ws_bytes=1 << 40):
    f = getattr(L.lib(), f"mk_attn_{kind}")
    if bt is None:
        bt = batch() if kind == "decode" else batch(n_tokens=7, d_cu=P)
    return f(kv or view(), bt, hq, q or rows(), 0.125, out or rows(), lse, ws, ws_bytes, None)


BAD_VIEWS = [dict(k=None), dict(v=None), dict(k=P + 8), dict(v=P + 2), dict(n_blocks=0),
             dict(n_kv_heads=0), dict(block=0), dict(block=8), dict(block=24), dict(block=8192),
             dict(table_stride=0), dict(d_table=None, n_blocks=1)]
BAD_BATCHES = [dict(batch=-1), dict(n_tokens=-1), dict(d_lens=None), dict(n_tokens=3)]


@pytest.mark.parametrize("bad", BAD_VIEWS)
def test_bad_views(bad):
    assert append(kv=view(**bad)) == L.MK_ERR_INVALID_ARG
    for kind in ("decode", "prefill"):
        assert attn(kind, kv=view(**bad)) == L.MK_ERR_INVALID_ARG


@pytest.mark.parametrize("bad", BAD_BATCHES)
def test_bad_batches(bad):
    assert append(bt=batch(**bad)) == L.MK_ERR_INVALID_ARG
    assert attn("decode", bt=batch(**bad)) == L.MK_ERR_INVALID_ARG


def test_batch_kind():
    # decode takes one token per sequence, prefill takes offsets
    assert attn("decode", bt=batch(d_cu=P)) == L.MK_ERR_INVALID_ARG
    assert attn("prefill", bt=batch()) == L.MK_ERR_INVALID_ARG
    assert attn("prefill", bt=batch(batch=-1, d_cu=P)) == L.MK_ERR_INVALID_ARG
    assert attn("prefill", bt=batch(d_lens=None, d_cu=P)) == L.MK_ERR_INVALID_ARG


@pytest.mark.parametrize("dim", [0, 32, 96, 256])
def test_head_sizes(dim):
    assert append(kv=view(head_dim=dim)) == L.MK_ERR_UNSUPPORTED
    for kind in ("decode", "prefill"):
        assert attn(kind, kv=view(head_dim=dim)) == L.MK_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", [rows(None), rows(P + 8), rows(P, 257), rows(P, 256, 60)])
def test_bad_rows(bad):
    for name in ("q", "k", "v", "qo"):
        assert append(**{name: bad}) == L.MK_ERR_INVALID_ARG, name
    for kind in ("decode", "prefill"):
        assert attn(kind, q=bad) == L.MK_ERR_INVALID_ARG
        assert attn(kind, out=bad) == L.MK_ERR_INVALID_ARG


def test_fp32_rows_may_be_closer():
    # 4 elements of 4 bytes are a 16-byte step, 2 are not
    assert append(k=rows(P, 258), src=L.MK_SRC_F32) == L.MK_ERR_INVALID_ARG
    assert append(src=7) == L.MK_ERR_INVALID_ARG


@pytest.mark.parametrize("theta", [-1.0, 0.5, float("nan"), float("inf")])
def test_bad_theta(theta):
    assert append(theta=theta) == L.MK_ERR_INVALID_ARG


def test_heads():
    assert append(hq=-1) == L.MK_ERR_INVALID_ARG
    for kind in ("decode", "prefill"):
        for hq in (0, -2, 3):
            assert attn(kind, hq=hq) == L.MK_ERR_INVALID_ARG


def test_null_structs():
    L_ = L.lib()
    assert L_.mk_kv_append(None, batch(), 4, rows(), rows(), rows(), 0, rows(), 1e4,
                           None) == L.MK_ERR_INVALID_ARG
    assert L_.mk_attn_decode(view(), None, 4, rows(), 1.0, rows(), None, P, 1 << 40,
                             None) == L.MK_ERR_INVALID_ARG
    assert L_.mk_kv_append(view(), batch(), 4, None, rows(), rows(), 0, rows(), 1e4,
                           None) == L.MK_ERR_INVALID_ARG


def test_workspace_arguments():
    f, n = L.lib().mk_attn_workspace_bytes, C.c_size_t()
    for bad in [(2, 1, 1, 4, 2, 64), (0, -1, 1, 4, 2, 64), (0, 1, -1, 4, 2, 64),
                (0, 1, 1, 0, 2, 64), (0, 1, 1, 3, 2, 64), (0, 1, 1, 4, 0, 64)]:
        assert f(*bad, C.byref(n)) == L.MK_ERR_INVALID_ARG
    assert f(0, 1, 1, 4, 2, 64, None) == L.MK_ERR_INVALID_ARG
    assert f(0, 1, 1, 4, 2, 80, C.byref(n)) == L.MK_ERR_UNSUPPORTED


def test_nothing_to_do_is_fine():
    assert append(bt=batch(batch=0, n_tokens=0, d_lens=None)) == L.MK_OK
    assert append(bt=batch(n_tokens=0, d_cu=P)) == L.MK_OK


def test_cache_wants_cuda_tensors():
    t = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        KVCache(t, t)


@pytest.mark.parametrize("ts,hs", [(0, 64), (256, 0), (192, 64), (64, 64), (64, 320), (256, 32)])
def test_outputs_must_not_overlap(ts, hs):
    # [7][4][64]: rows that share elements, at strides that inputs may have
    bt = batch(n_tokens=7, d_cu=P)
    assert append(bt=bt, qo=rows(ts=ts, hs=hs)) == L.MK_ERR_INVALID_ARG
    assert attn("prefill", bt=bt, out=rows(2 * P, ts, hs)) == L.MK_ERR_INVALID_ARG


def test_output_is_not_the_queries():
    for kind in ("decode", "prefill"):
        assert attn(kind, q=rows(P), out=rows(P)) == L.MK_ERR_INVALID_ARG


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf")])
def test_scales_are_finite(scale):
    for kind, bt in (("decode", batch()), ("prefill", batch(n_tokens=7, d_cu=P))):
        f = getattr(L.lib(), f"mk_attn_{kind}")
        assert f(view(), bt, 4, rows(), scale, rows(2 * P), None, P, 1 << 40, None) == L.MK_ERR_INVALID_ARG
