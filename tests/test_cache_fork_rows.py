"""What a fork of the paged cache leaves of the rows it starts from: pages of rows without children are free in the same
call, a row that is its own parent stays as it is.  By the oracle on the CPU, and the same calls on the GPU."""
import os

import numpy as np
import pytest

import oracle.cache as oc
from tests.cache_harness import random_cache, random_table


def copy_of(c):
    return {x: (y.copy() if isinstance(y, np.ndarray) else y) for x, y in c.items()}


def start():
    rng = np.random.default_rng(3)
    cache = random_cache(rng, 40, 2, 16, 64, "e4m3")
    for s in ("ks", "vs"):
        cache[s] = (2.0 ** np.round(np.log2(cache[s]))).astype(np.float32)
    lens = np.array([10, 26, 40, 16], np.int32)
    return rng, cache, random_table(rng, lens, 16, 40, extra=3), lens


def test_a_page_of_a_row_without_children_is_given_away():
    _, cache, _, _ = start()
    table, lens = np.array([[0, -1], [1, -1]], np.int32), np.array([10, 10], np.int32)
    was = copy_of(cache)
    out, length, status = oc.fork(cache, table, lens, np.array([1, 1]))
    assert out.tolist() == [[1, -1], [0, -1]] and length.tolist() == [10, 10] and status == 0
    assert np.array_equal(cache["k"][0], was["k"][1]) and not np.array_equal(cache["k"][0], was["k"][0])


def test_the_header_says_so():
    path = os.path.join(os.path.dirname(__file__), "..", "include", "xgr_cache.h")
    with open(path) as f:
        text = " ".join(f.read().replace("\n *", " ").split())
    assert "Pages of rows without children are free in this very call" in text
    assert "can be taken back" not in text and "are not changed" not in text


def kept_rows(rng, table, lens):
    """Parents: every row its own, then children of rows 2, 0, 2, 1."""
    n = len(lens)
    parent = np.r_[np.arange(n), [2, 0, 2, 1]].astype(np.int32)
    grow = np.r_[np.zeros(n), [1, 3, 20, 5]].astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(grow)])
    x = rng.standard_normal((2, cu[-1], 2, 64)) * 50         # (large: their pages' scales grow)
    return n, parent, grow, cu, x


def test_rows_that_are_their_own_parents_can_be_gone_back_to():
    rng, cache, table, lens = start()
    n, parent, grow, cu, x = kept_rows(rng, table, lens)
    before = [oc.row_kv(cache, table[r], int(lens[r]), g) for r in range(n) for g in range(2)]
    out, length, status = oc.fork(cache, table, lens, parent, grow)
    assert status == 0 and np.array_equal(out[:n], table) and np.array_equal(length[:n], lens)
    oc.store(cache, out, length, cu, x[0], x[1])
    after = [oc.row_kv(cache, out[r], int(lens[r]), g) for r in range(n) for g in range(2)]
    for a, b in zip(before, after):
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.gpu
def test_going_back_on_the_gpu():
    import torch
    from tests.cache_harness import bf16, i32, same_cache, to_device, to_host
    rng, cache, table, lens = start()
    n, parent, grow, cu, x = kept_rows(rng, table, lens)
    pc = to_device(cache)
    q, _ = bf16(rng.standard_normal((n, 4, 64)))

    def attend(t, ln):
        out, lse = torch.empty_like(q), torch.empty((n, 4), device="cuda")
        pc.attend(t, ln, i32(np.arange(n + 1)), q, out, lse, max_q=1)
        return out, lse
    want = attend(i32(table), i32(lens))
    t2, l2 = i32(np.zeros((len(parent), table.shape[1]))), i32(np.zeros(len(parent)))
    pc.fork(i32(table), i32(lens), i32(parent), i32(grow), t2, l2)
    k, k64 = bf16(x[0])
    v, v64 = bf16(x[1])
    pc.store(t2, l2, i32(cu), k, v, max_n=int(grow.max()))
    out, length, _ = oc.fork(cache, table, lens, parent, grow)
    oc.store(cache, out, length, cu, k64, v64)
    same_cache(to_host(pc), cache)
    got = attend(t2[:n].contiguous(), l2[:n].contiguous())
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    # the two rows on pages 0 and 1 of which one has both children
    small = {**copy_of(cache)}
    pc = to_device(small)
    t, ln, t2, l2 = i32([[0, -1], [1, -1]]), i32([10, 10]), i32(np.zeros((2, 2))), i32([0, 0])
    pc.fork(t, ln, i32([1, 1]), None, t2, l2)
    assert t2.tolist() == [[1, -1], [0, -1]]
    oc.fork(small, np.array([[0, -1], [1, -1]]), np.array([10, 10]), np.array([1, 1]))
    same_cache(to_host(pc), small)
    assert pc.device_status() == 0
