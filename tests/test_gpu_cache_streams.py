"""The paged 8-bit cache's calls on a stream that is not torch's current one."""
import numpy as np
import pytest
import torch

import oracle.cache as oc
from shared_prefix_decode_xattention_b200 import xgr
from shared_prefix_decode_xattention_b200.cache import PagedCache
from tests.cache_harness import bf16, close, i32, random_cache, random_table, same_cache, to_device, to_host

pytestmark = pytest.mark.gpu


def small(seed=0):
    rng = np.random.default_rng(seed)
    cache = random_cache(rng, 40, 2, 16, 64, "int8")
    for s in ("ks", "vs"):
        cache[s] = (2.0 ** np.round(np.log2(cache[s]))).astype(np.float32)
    lens = np.array([40, 33, 64])
    return rng, cache, lens, random_table(rng, lens, 16, 40)


@pytest.mark.parametrize("as_handle", [False, True])
def test_every_call_on_a_stream_of_the_callers(as_handle):
    rng, cache, lens, table = small()
    pc = to_device(cache)
    rows, width = table.shape
    side = torch.cuda.Stream()
    st = side.cuda_stream if as_handle else side
    t, ln, ones, cu = i32(table), i32(lens), i32(np.ones(rows)), i32(np.arange(rows + 1))
    parent = np.array([1, 1, 2], np.int32)
    t2, l2, t3, used, par = i32(np.zeros((rows, width))), i32(np.zeros(rows)), i32(np.zeros((rows, width))), i32([0]), i32(parent)
    k, k64 = bf16(rng.standard_normal((rows, 2, 64)))
    q, q64 = bf16(rng.standard_normal((rows, 4, 64)))
    out, lse = torch.empty_like(q), torch.empty((rows, 4), device="cuda")
    torch.cuda.synchronize()
    pc.fork(t, ln, par, ones, t2, l2, stream=st)
    pc.store(t2, l2, cu, k, k, max_n=1, stream=st)
    pc.attend(t2, l2, cu, q, out, lse, max_q=1, stream=st)
    pc.compact(t2, l2, t3, used, stream=st)
    assert pc.device_status() == 0
    table, lens, _ = oc.fork(cache, table, lens, parent, np.ones(rows, np.int32))
    oc.store(cache, table, lens, np.arange(rows + 1), k64, k64)
    ref, ref_lse = oc.attend(cache, table, lens, np.arange(rows + 1), q64)
    close(out, lse, ref, ref_lse, np.full((rows, 4, 1), 127 * cache["vs"].max()), 64, 40.0)
    table, u = oc.compact(cache, table, lens)
    assert np.array_equal(t3.cpu().numpy(), table) and used.item() == u
    same_cache(to_host(pc), cache)


def test_a_workspace_is_memory_of_the_stream_that_uses_it():
    """A block that the current stream gave back, and may still be working on, is not taken for another stream's call."""
    rng, cache, lens, table = small()
    pc = to_device(cache)
    q, _ = bf16(rng.standard_normal((3, 4, 64)))
    out, lse = torch.empty_like(q), torch.empty((3, 4), device="cuda")
    t, ln, cu, side = i32(table), i32(lens), i32(np.arange(4)), torch.cuda.Stream()
    size = pc.attend_bytes(4, 3, 3)
    x = torch.empty(size, dtype=torch.uint8, device="cuda")
    at = x.data_ptr()
    torch.cuda.synchronize()
    del x
    pc.attend(t, ln, cu, q, out, lse, max_q=1, stream=side)
    y = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert y.data_ptr() == at
    assert pc.device_status() == 0


def test_a_capture_on_another_stream_than_the_current_one_is_seen():
    rng, cache, lens, table = small()
    pc, fresh = to_device(cache), to_device(cache)
    q, _ = bf16(rng.standard_normal((3, 4, 64)))
    out, lse = torch.empty_like(q), torch.empty((3, 4), device="cuda")
    t, ln, cu, side, other = i32(table), i32(lens), i32(np.arange(4)), torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    pc.attend(t, ln, cu, q, out, lse, max_q=1, stream=side)
    torch.cuda.synchronize()
    want = out.clone()
    g, seen = torch.cuda.CUDAGraph(), None
    with torch.cuda.stream(side):
        g.capture_begin(capture_error_mode="relaxed")
        with torch.cuda.stream(other):
            try:
                fresh.attend(t, ln, cu, q, out, lse, max_q=1, stream=side)
            except xgr.XgrError as e:
                seen = e.status
            pc.attend(t, ln, cu, q, out, lse, max_q=1, stream=side)      # has a workspace there
        g.capture_end()
    assert seen == xgr.XGR_ERR_STATE
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and pc.device_status() == 0


def test_faults_of_other_streams_are_not_lost():
    """A cache made while its stream is busy, a fault met on another stream at once."""
    rng, cache, lens, table = small()
    c = to_device(cache)
    q, _ = bf16(rng.standard_normal((3, 4, 64)))
    out, lse = torch.empty_like(q), torch.empty((3, 4), device="cuda")
    ws = torch.empty(c.attend_bytes(4, 3, 3), dtype=torch.uint8, device="cuda")
    bad = table.copy()
    bad[1, 1] = 1000
    t, ln, cu, side = i32(bad), i32(lens), i32(np.arange(4)), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)                                        # some 30 ms of the current stream
    pc = PagedCache(c.k, c.v, c.k_scale, c.v_scale)
    pc.attend(t, ln, cu, q, out, lse, max_q=1, stream=side, workspace=ws)
    assert pc.device_status() == xgr.XGR_DEV_INDEX
    assert pc.device_status() == 0


def test_a_cache_is_not_made_under_a_capture():
    _, cache, _, _ = small()
    c = to_device(cache)
    g, seen = torch.cuda.CUDAGraph(), None
    x = torch.zeros(4, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        x.add_(1)
        try:
            PagedCache(c.k, c.v, c.k_scale, c.v_scale)
        except xgr.XgrError as e:
            seen = e.status
    assert seen == xgr.XGR_ERR_STATE
