"""Refusals of the paged cache's C ABI that need no GPU: nothing is enqueued for any of these."""
import ctypes

import pytest

from shared_prefix_decode_xattention_b200 import build, xgr

D = 1 << 20        # a pointer that is never followed: every call below is refused before a launch


@pytest.fixture(scope="module")
def L():
    build.build()
    return xgr.lib()


def cache(**kw):
    base = dict(d_k=D, d_v=D, d_k_scale=D, d_v_scale=D, n_pages=100, page_size=64, n_kv_heads=4, head_dim=128,
                format=xgr.XGR_CACHE_E4M3)
    base.update(kw)
    return xgr.xgr_cache(**base)


def rows(**kw):
    base = dict(n_rows=3, max_pages=10, d_table=D, d_len=D)
    base.update(kw)
    return xgr.xgr_cache_rows(**base)


def attend(c=None, r=None, o=None, **kw):
    a = dict(cu=D, n_tokens=3, max_q=1, hq=16, q=D, stride=16 * 128, out=2 * D, lse=D, ws=D, ws_bytes=1 << 40, status=D)
    a.update(kw)
    opts = xgr.xgr_attn_opts(**{**dict(scale=0, softcap=0, mask=1, window=0), **(o or {})})
    return xgr.lib().xgr_cache_attend(ctypes.byref(c or cache()), ctypes.byref(r or rows()), a["cu"], a["n_tokens"],
                                      a["max_q"], a["hq"], a["q"], a["stride"], ctypes.byref(opts), a["out"], a["lse"],
                                      a["ws"], a["ws_bytes"], a["status"], None)


def store(c=None, r=None, **kw):
    a = dict(cu=D, n_tokens=3, max_n=1, k=D, v=D, stride=512, status=D)
    a.update(kw)
    return xgr.lib().xgr_cache_store(ctypes.byref(c or cache()), ctypes.byref(r or rows()), a["cu"], a["n_tokens"],
                                     a["max_n"], a["k"], a["v"], a["stride"], a["status"], None)


def fork(c=None, r=None, **kw):
    a = dict(n_out=3, parent=D, n_new=None, table=2 * D, length=3 * D, ws=D, ws_bytes=1 << 40, status=D)
    a.update(kw)
    return xgr.lib().xgr_cache_fork(ctypes.byref(c or cache()), ctypes.byref(r or rows()), a["n_out"], a["parent"],
                                    a["n_new"], a["table"], a["length"], a["ws"], a["ws_bytes"], a["status"], None)


def compact(c=None, r=None, **kw):
    a = dict(table=2 * D, used=D, ws=D, ws_bytes=1 << 40, status=D)
    a.update(kw)
    return xgr.lib().xgr_cache_compact(ctypes.byref(c or cache()), ctypes.byref(r or rows()), a["table"], a["used"],
                                       a["ws"], a["ws_bytes"], a["status"], None)


def test_struct_sizes(L):
    assert ctypes.sizeof(xgr.xgr_cache) == 56
    assert ctypes.sizeof(xgr.xgr_cache_rows) == 24
    assert ctypes.sizeof(xgr.xgr_attn_opts) == 40


@pytest.mark.parametrize("call", [attend, store, fork, compact])
@pytest.mark.parametrize("bad,st", [
    (dict(page_size=48), xgr.XGR_ERR_UNIMPLEMENTED), (dict(page_size=256), xgr.XGR_ERR_UNIMPLEMENTED),
    (dict(head_dim=96), xgr.XGR_ERR_UNIMPLEMENTED), (dict(format=2), xgr.XGR_ERR_ARG),
    (dict(n_pages=0), xgr.XGR_ERR_SHAPE), (dict(n_pages=(1 << 30) + 1), xgr.XGR_ERR_SHAPE),
    (dict(n_kv_heads=0), xgr.XGR_ERR_SHAPE), (dict(n_pages=1 << 30, page_size=128), xgr.XGR_ERR_SHAPE), (dict(d_k=None), xgr.XGR_ERR_ARG), (dict(d_v=D + 8), xgr.XGR_ERR_ARG),
    (dict(d_v_scale=D + 2), xgr.XGR_ERR_ARG)])
def test_bad_caches(L, call, bad, st):
    assert call(c=cache(**bad)) == st


@pytest.mark.parametrize("call", [attend, store, fork, compact])
@pytest.mark.parametrize("bad,st", [
    (dict(n_rows=-1), xgr.XGR_ERR_SHAPE), (dict(n_rows=(1 << 22) + 1), xgr.XGR_ERR_SHAPE),
    (dict(max_pages=0), xgr.XGR_ERR_SHAPE),
    (dict(max_pages=1 << 25), xgr.XGR_ERR_SHAPE), (dict(d_table=None), xgr.XGR_ERR_ARG),
    (dict(d_len=D + 1), xgr.XGR_ERR_ARG)])
def test_bad_rows(L, call, bad, st):
    assert call(r=rows(**bad)) == st


@pytest.mark.parametrize("call", [attend, store, fork, compact])
def test_status_word_is_needed(L, call):
    assert call(status=None) == xgr.XGR_ERR_ARG


@pytest.mark.parametrize("kw,o,st", [
    (dict(hq=18), {}, xgr.XGR_ERR_SHAPE), (dict(hq=0), {}, xgr.XGR_ERR_SHAPE), (dict(stride=2040), {}, xgr.XGR_ERR_SHAPE),
    (dict(stride=2052), {}, xgr.XGR_ERR_SHAPE), (dict(n_tokens=-1), {}, xgr.XGR_ERR_SHAPE), (dict(max_q=-1), {}, xgr.XGR_ERR_SHAPE),
    (dict(q=D + 8), {}, xgr.XGR_ERR_ARG), (dict(out=D + 4096), {}, xgr.XGR_ERR_ARG), (dict(out=None), {}, xgr.XGR_ERR_ARG), (dict(lse=D + 2), {}, xgr.XGR_ERR_ARG),
    (dict(cu=None), {}, xgr.XGR_ERR_ARG), (dict(ws=D + 16), {}, xgr.XGR_ERR_ARG), (dict(ws_bytes=1000), {}, xgr.XGR_ERR_CAPACITY),
    ({}, dict(mask=2), xgr.XGR_ERR_ARG), ({}, dict(mask=0, d_prefix=D), xgr.XGR_ERR_ARG), ({}, dict(window=-1), xgr.XGR_ERR_SHAPE),
    ({}, dict(softcap=-1.0), xgr.XGR_ERR_ARG), ({}, dict(softcap=float("nan")), xgr.XGR_ERR_ARG),
    ({}, dict(scale=float("inf")), xgr.XGR_ERR_ARG), ({}, dict(scale=-1.0), xgr.XGR_ERR_ARG), ({}, dict(d_slopes=D + 1), xgr.XGR_ERR_ARG),
    (dict(n_tokens=1 << 30, hq=16), {}, xgr.XGR_ERR_SHAPE)])
def test_attend_refusals(L, kw, o, st):
    assert attend(o=o, **kw) == st


@pytest.mark.parametrize("kw,st", [
    (dict(stride=504), xgr.XGR_ERR_SHAPE), (dict(stride=516), xgr.XGR_ERR_SHAPE), (dict(k=None), xgr.XGR_ERR_ARG),
    (dict(v=D + 2), xgr.XGR_ERR_ARG), (dict(cu=None), xgr.XGR_ERR_ARG), (dict(n_tokens=-3), xgr.XGR_ERR_SHAPE),
    (dict(max_n=-1), xgr.XGR_ERR_SHAPE)])
def test_store_refusals(L, kw, st):
    assert store(**kw) == st


@pytest.mark.parametrize("kw,st", [
    (dict(n_out=-1), xgr.XGR_ERR_SHAPE), (dict(n_out=1 << 29), xgr.XGR_ERR_SHAPE), (dict(parent=None), xgr.XGR_ERR_ARG),
    (dict(table=D + 40), xgr.XGR_ERR_ARG), (dict(length=D), xgr.XGR_ERR_ARG), (dict(length=2 * D + 2), xgr.XGR_ERR_ARG),
    (dict(ws=None), xgr.XGR_ERR_ARG), (dict(ws_bytes=100), xgr.XGR_ERR_CAPACITY), (dict(n_new=D + 2), xgr.XGR_ERR_ARG)])
def test_fork_refusals(L, kw, st):
    assert fork(**kw) == st


@pytest.mark.parametrize("kw,st", [
    (dict(table=D + 40), xgr.XGR_ERR_ARG), (dict(used=None), xgr.XGR_ERR_ARG), (dict(ws=D + 8), xgr.XGR_ERR_ARG),
    (dict(ws_bytes=100), xgr.XGR_ERR_CAPACITY)])
def test_compact_refusals(L, kw, st):
    assert compact(**kw) == st


def test_nothing_to_do_is_ok(L):
    assert attend(n_tokens=0) == 0 and attend(r=rows(n_rows=0, d_table=None, d_len=None)) == 0
    assert store(n_tokens=0) == 0 and fork(n_out=0) == 0


def test_workspace_sizes(L):
    c = cache()
    assert xgr.xgr_cache_attend_bytes(c, 16, 100, 100) % 256 == 0
    assert xgr.xgr_cache_fork_bytes(c, 1000, 1000) > 2 * 4 * 100 and xgr.xgr_cache_compact_bytes(c) % 256 == 0
    with pytest.raises(xgr.XgrError):
        xgr.xgr_cache_attend_bytes(c, 15, 100, 100)
    with pytest.raises(xgr.XgrError):
        xgr.xgr_cache_fork_bytes(c, 10, -1)
    assert L.xgr_cache_compact_bytes(ctypes.byref(c), None) == xgr.XGR_ERR_ARG
    assert L.xgr_cache_compact_bytes(None, None) == xgr.XGR_ERR_ARG
