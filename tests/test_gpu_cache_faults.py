"""The paged 8-bit cache's calls on token ranges that do not fit together."""
import numpy as np
import pytest
import torch

import oracle.cache as oc
from shared_prefix_decode_xattention_b200 import xgr
from tests.cache_harness import bf16, close, i32, random_cache, random_table, same_cache, to_device, to_host

pytestmark = pytest.mark.gpu

ROWS = 9


def spoiled(cu):
    """d_cu with one bad entry, where a search over it begins, ends and between."""
    for at, value in ((2, cu[-1] + 1), (2, cu[6]), (4, cu[7]), (4, cu[3] - 1), (5, -3), (0, cu[2]), (1, 1 << 30), (ROWS, cu[-1] + 1),
                      (ROWS, cu[4])):
        bad = cu.copy()
        bad[at] = value
        yield bad


@pytest.mark.parametrize("n,G", [(2, 4), (8, 3), (16, 5)])         # 16-, 32- and 256-row tiles
@pytest.mark.parametrize("L", [90, 3000])
def test_attend_of_a_bad_order_does_nothing(n, G, L):
    """Rows short and long enough to be cut among blocks; the workspace holds large numbers from before."""
    rng = np.random.default_rng(n)
    lens = rng.integers(L // 2, L, ROWS)
    pages = int(sum(-(-int(x) // 64) for x in lens)) + 2
    cache = random_cache(rng, pages, 2, 64, 64, "int8")
    table = random_table(rng, lens, 64, pages)
    cu = np.arange(ROWS + 1) * n
    q, q64 = bf16(rng.standard_normal((ROWS * n, 2 * G, 64)))
    pc = to_device(cache)
    t, ln = i32(table), i32(lens)
    ws = torch.full((pc.attend_bytes(2 * G, ROWS, ROWS * n),), 0x7d, dtype=torch.uint8, device="cuda")
    out, lse = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda"), torch.full(q.shape[:2], 7.0, device="cuda")
    for bad in spoiled(cu):
        for first in (None, i32(np.zeros(ROWS * n))):
            pc.attend(t, ln, i32(bad), q, out, lse, max_q=1 << 20, workspace=ws, first=first)
            assert pc.device_status() == xgr.XGR_DEV_INDEX, bad
            assert (out == 7).all() and (lse == 7).all(), bad
    pc.attend(t, ln, i32(cu), q, out, lse, max_q=n, workspace=ws)
    ref, ref_lse = oc.attend(cache, table, lens, cu, q64)
    close(out, lse, ref, ref_lse, np.full((ROWS * n, 2 * G, 1), 127 * cache["vs"].max()), 64, 40.0)
    assert pc.device_status() == 0


@pytest.mark.parametrize("page,d", [(16, 64), (64, 128)])
def test_store_of_a_bad_order_leaves_whole_rows_out(page, d):
    """Each row's pages are either those of the call or those from before, and the fault is reported."""
    rng = np.random.default_rng(page)
    lens, n = rng.integers(60, 200, ROWS), 40
    pages = int(sum(-(-int(x) // page) for x in lens)) + 2
    cache = random_cache(rng, pages, 2, page, d, "e4m3")
    for s in ("ks", "vs"):
        cache[s] = (2.0 ** np.round(np.log2(cache[s]))).astype(np.float32)
    table = random_table(rng, lens, page, pages)
    cu = np.arange(ROWS + 1) * n
    k, k64 = bf16(rng.standard_normal((ROWS * n, 2, d)))
    v, v64 = bf16(rng.standard_normal((ROWS * n, 2, d)))

    def copy_of(c):
        return {x: (y.copy() if isinstance(y, np.ndarray) else y) for x, y in c.items()}
    for bad in spoiled(cu):
        pc = to_device(cache)
        pc.store(i32(table), i32(lens), i32(bad), k, v, max_n=1 << 20)
        assert pc.device_status() == xgr.XGR_DEV_INDEX, bad
        got = to_host(pc)
        for r in range(ROWS):
            held = table[r, : -(-int(lens[r]) // page)]
            whole = copy_of(cache)
            lo, hi = int(bad[r]), int(bad[r + 1])
            if 0 <= lo <= hi <= cu[-1] and hi - lo <= lens[r]:
                oc.store(whole, table[r: r + 1], lens[r: r + 1], np.array([0, hi - lo]), k64[lo:hi], v64[lo:hi])
            same = [all(np.array_equal(got[x][held].view(np.uint8), c[x][held].view(np.uint8)) for x in ("k", "v", "ks", "vs"))
                    for c in (cache, whole)]
            assert any(same), (bad, r)
    pc = to_device(cache)
    pc.store(i32(table), i32(lens), i32(cu), k, v, max_n=n)
    assert pc.device_status() == 0
    oc.store(cache, table, lens, cu, k64, v64)
    same_cache(to_host(pc), cache)


def test_store_of_single_tokens_leaves_out_the_rows_at_fault():
    rng = np.random.default_rng(0)
    lens = rng.integers(20, 60, ROWS)
    cache = random_cache(rng, 40, 2, 16, 64, "int8")
    for s in ("ks", "vs"):
        cache[s] = (2.0 ** np.round(np.log2(cache[s]))).astype(np.float32)
    table = random_table(rng, lens, 16, 40)
    k, k64 = bf16(rng.standard_normal((ROWS, 2, 64)))
    pc = to_device(cache)
    bad = np.arange(ROWS + 1)
    bad[4] = 100                                    # rows 3 (4 tokens too many) and 4 (from nowhere)
    pc.store(i32(table), i32(lens), i32(bad), k, k, max_n=1)
    assert pc.device_status() & xgr.XGR_DEV_INDEX
    keep = [r for r in range(ROWS) if r not in (3, 4)]
    oc.store(cache, table[keep], lens[keep], np.arange(len(keep) + 1), k64[keep], k64[keep])
    same_cache(to_host(pc), cache)


def test_calls_on_no_rows_and_no_tokens():
    rng = np.random.default_rng(0)
    cache = random_cache(rng, 12, 2, 16, 64, "int8")
    pc = to_device(cache)
    none, zero = torch.empty((0, 3), dtype=torch.int32, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda")
    used = i32([7])
    pc.compact(none, zero, torch.empty_like(none), used)
    assert used.item() == 0
    t2, l2 = i32(np.zeros((2, 3))), i32([5, 5])
    pc.fork(none, zero, i32([-1, -1]), i32([4, 4]), t2, l2)            # rows without parents are empty, whatever they want
    assert (t2 == -1).all() and l2.tolist() == [0, 0]
    pc.fork(t2, l2, i32([0, 1]), i32([17, 0]), t3 := torch.empty_like(t2), l3 := torch.empty_like(l2))
    assert t3.tolist() == [[0, 1, -1], [-1, -1, -1]] and l3.tolist() == [17, 0]
    q = torch.ones((3, 4, 64), dtype=torch.bfloat16, device="cuda")
    for mask, n in (("full", 1), ("causal", 1), ("full", 70)):
        out, lse = torch.full_like(q, 7.0), torch.full((3, 4), 7.0, device="cuda")
        pc.attend(t3, l3, i32([0, 0, 0]), q, out, lse, max_q=n, mask=mask)             # tokens of no row
        assert (out == 7).all() and (lse == 7).all()
        pc.attend(none, zero, i32([0]), q, out, lse, max_q=n, mask=mask)
        assert (out == 7).all() and (lse == 7).all()
        if mask == "full":                                                             # a row of no keys
            pc.attend(t3, l3, i32([0, 0, 3]), q, out, lse, max_q=max(n, 3), mask=mask)
            assert not out.any() and torch.isneginf(lse).all()
    pc.store(t3, l3, i32([0, 0, 0]), q[:, :2], q[:, :2], max_n=3)
    assert pc.device_status() == 0
    same_cache(to_host(pc), cache)
