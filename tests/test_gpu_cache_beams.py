"""Beams over a prompt in the paged 8-bit cache: more of them than the prompt has tokens."""
import numpy as np
import pytest
import torch

import oracle.cache as oc
from shared_prefix_decode_xattention_b200 import xgr
from tests.cache_harness import bf16, close, i32, random_cache, random_table, to_device

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(), dict(window=9), dict(window=2 ** 31 - 1), dict(softcap=20.0, slopes=[0.1, 0.02, 0.3, 0.0, 0.2, 0.05]),
                                dict(first=True)])
@pytest.mark.parametrize("n,G,d,page", [(9, 1, 64, 16), (20, 1, 128, 32), (15, 3, 64, 64), (90, 3, 128, 16), (300, 2, 64, 128)])
def test_more_beams_than_keys(n, G, d, page, kw):
    """Prompts of none, one and some tokens, shorter and longer than the beams are many."""
    rng = np.random.default_rng(n)
    lens = np.array([0, 1, n - 1, 7, n, n + 5, 40])
    count = np.array([n, n, n, n, n, n, 0])
    cache = random_cache(rng, 120, 2, page, d, "int8")
    table = random_table(rng, lens, page, 120)
    cu = np.concatenate([[0], np.cumsum(count)])
    T = int(cu[-1])
    q, q64 = bf16(rng.standard_normal((T, 2 * G, d)))
    kw = dict(kw)
    if "slopes" in kw:
        kw["slopes"] = kw["slopes"][: 2 * G]
    if kw.get("first"):
        kw["first"] = rng.integers(-3, n, T).astype(np.int32)
    ref, ref_lse = oc.attend(cache, table, lens, cu, q64, mask="full", **kw)
    pc = to_device(cache)
    out, lse = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda"), torch.full(q.shape[:2], 7.0, device="cuda")
    if "slopes" in kw:
        kw["slopes"] = torch.tensor(kw["slopes"], dtype=torch.float32, device="cuda")
    if "first" in kw:
        kw["first"] = i32(kw["first"])
    pc.attend(i32(table), i32(lens), i32(cu), q, out, lse, max_q=n, mask="full", **kw)
    assert pc.device_status() == 0
    qk = 40.0 + (0.3 * n if "slopes" in kw else 0)
    close(out, lse, ref, ref_lse, np.full((T, 2 * G, 1), 127 * cache["vs"].max()), d, qk)


def test_more_tokens_than_keys_are_refused_where_they_are_the_rows_own():
    rng = np.random.default_rng(0)
    cache = random_cache(rng, 10, 1, 16, 64, "e4m3")
    pc = to_device(cache)
    t, ln, cu = i32([[0, 1, -1], [2, -1, -1]]), i32([20, 4]), i32([0, 3, 8])
    q, _ = bf16(rng.standard_normal((8, 1, 64)))
    out, lse = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((8, 1), 7.0, device="cuda")
    pc.attend(t, ln, cu, q, out, lse, max_q=5)
    assert pc.device_status() == xgr.XGR_DEV_INDEX and (out[3:] == 7).all() and (out[:3] != 7).any()
    before = pc.k.view(torch.uint8).clone()
    pc.store(t, ln, cu, q, q, max_n=5)
    assert pc.device_status() == xgr.XGR_DEV_INDEX and torch.equal(pc.k.view(torch.uint8)[2], before[2])
