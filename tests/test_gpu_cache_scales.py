"""The attention over the paged 8-bit cache with V scales far from one another and from 1: pages of zeros, pages that a
query does not see or gives next to no weight, tiny and huge ones.  Against the definition in 64 bits, the error
measured against the values that a query attends to (not against the largest of the row)."""
import numpy as np
import pytest
import torch

import oracle.cache as oc
from tests.cache_harness import bf16, i32, random_cache, random_table, to_device

pytestmark = pytest.mark.gpu

HKV = 2


def check(cache, table, lens, cu, q, q64, kw, extra_rows=()):
    """One call; every output within what its roundings allow.

    out: half a bf16 step, 2^-8 |o|; every weight w_j = p_j b_j rounded to fp16, 2^-11 relative where it is a normal
    number, so 2^-11 sum_j p_j |v_j|, half of that again for the exponentials and sums (the exponent's own rounding at a
    size of up to 256 is 2^-17, 2^-17 relative); a weight below fp16's normal numbers is off by 2^-25 of a scale at which
    the row's largest weight is 2^2 at least (14 of bias, 12 of reference), so 2^-27 of it, for each key.  2^-133: bf16's
    smallest number.
    lse: D + 8 roundings of a score, 32 of the sum, its largest terms bounded as in the other tests."""
    hq, d = q.shape[1], q.shape[2]
    G = hq // HKV
    ref, ref_lse = oc.attend(cache, table, lens, cu, q64, **kw)
    pc = to_device(cache)
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    dev = {x: (i32(y) if x == "first" else torch.tensor(y, dtype=torch.float32, device="cuda") if x == "slopes" else y)
           for x, y in kw.items()}
    pc.attend(i32(table), i32(lens), i32(cu), q, out, lse, max_q=int(np.diff(cu).max()), **dev)
    assert pc.device_status() == 0
    o, z = out.double().cpu().numpy(), lse.double().cpu().numpy()
    page = cache["k"].shape[2]
    for r in range(len(lens)):
        L, n = int(lens[r]), int(cu[r + 1] - cu[r])
        kv = [oc.row_kv(cache, table[r], L, g) for g in range(HKV)]
        b = [np.repeat(cache["vs"][table[r][: -(-L // page)], g].astype(np.float64), page)[:L] for g in range(HKV)]
        for i in range(n):
            t = int(cu[r]) + i
            lo, hi, pos = oc.visible(L, n, i, kw.get("mask", "causal"), kw.get("window", 0), None,
                                     None if "first" not in kw else int(kw["first"][t]))
            if lo >= hi:
                assert np.isneginf(z[t]).all() and not o[t].any()
                continue
            for h in range(hq):
                k, v = kv[h // G]
                s = k[lo:hi] @ q64[t, h] * d ** -0.5
                qk = np.abs(k[lo:hi]) @ np.abs(q64[t, h]) * d ** -0.5
                if "softcap" in kw:
                    s = kw["softcap"] * np.tanh(s / kw["softcap"])
                if "slopes" in kw:
                    s = s - kw["slopes"][h] * np.abs(pos - np.arange(lo, hi))
                p = np.exp(s - ref_lse[t, h])
                near = p @ np.abs(v[lo:hi])
                peak = (p * b[h // G][lo:hi]).max() * oc.QMAX[cache["fmt"]]
                tol = (2.0 ** -8 * np.abs(ref[t, h]) + 1.5 * 2.0 ** -11 * near + (hi - lo) * 2.0 ** -27 * peak + 2.0 ** -133)
                err = np.abs(o[t, h] - ref[t, h])
                assert (err <= tol).all(), (t, h, o[t, h][:4], ref[t, h][:4])
                tol = 2.0 ** -24 * ((d + 8) * qk.max() + 16 * np.abs(s).max() + 16 * abs(ref_lse[t, h]) + 32)
                assert abs(z[t, h] - ref_lse[t, h]) <= tol, (t, h, z[t, h], ref_lse[t, h])


def scales_of(kind, rng, shape, ids):
    """V scales [n_pages][Hkv]; ids: the row's pages in order."""
    s = (2.0 ** rng.uniform(-1, 1, shape) / 100).astype(np.float64)
    if kind == "outlier first":              # beside the rest of the row, where a mask or a bias hides it
        s[ids[:2]] *= 2.0 ** 60
    elif kind == "outlier last":
        s[ids[-1]] *= 2.0 ** 45
    elif kind == "tiny":
        s = 2.0 ** rng.integers(-126, -100, shape).astype(np.float64)
    elif kind == "huge":
        s = 2.0 ** rng.integers(95, 113, shape).astype(np.float64)
    elif kind == "zeros":
        s[:] = 0.0
    elif kind == "smallest":                 # as a store leaves pages of zeros
        s[:] = 2.0 ** -126
    elif kind == "some smallest":
        s[rng.random(shape) < 0.4] = 2.0 ** -126
        s[rng.random(shape) < 0.2] *= 2.0 ** 20
    elif kind == "wild":
        s = 2.0 ** rng.integers(-126, 100, shape).astype(np.float64)
    return s.astype(np.float32)


KINDS = ["outlier first", "outlier last", "tiny", "huge", "zeros", "smallest", "some smallest", "wild"]


def row_case(kind, n, G, d, fmt, L, extra, seed=0, page=16, **kw):
    rng = np.random.default_rng(seed)
    pages = -(-L // page) + 3
    cache = random_cache(rng, pages, HKV, page, d, fmt)
    table = random_table(rng, [L], page, pages, extra)
    cache["vs"] = scales_of(kind, rng, cache["vs"].shape, table[0, : -(-L // page)])
    q, q64 = bf16(rng.standard_normal((n, HKV * G, d)))
    check(cache, table, np.array([L]), np.array([0, n]), q, q64, kw)


FEW = [(1, 4, 128, "e4m3"), (1, 3, 64, "int8"), (9, 2, 128, "int8"), (7, 4, 64, "e4m3")]      # 16- and 32-row tiles


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,G,d,fmt", FEW)
def test_few_rows(kind, n, G, d, fmt):
    row_case(kind, n, G, d, fmt, 300, 2)                                  # a whole row
    row_case(kind, n, G, d, fmt, 2500, 2, seed=1, page=64)                # cut among blocks
    row_case(kind, n, G, d, fmt, 200, 2, seed=2, slopes=[0.3] * (HKV * G))


@pytest.mark.parametrize("window", [264, 268, 250, 40])
@pytest.mark.parametrize("n,G,d,fmt", FEW)
def test_few_rows_hidden_page(window, n, G, d, fmt):
    """The outlier's page lies in the tile at the window's edge, none or some of its keys seen."""
    row_case("outlier first", n, G, d, fmt, 300, 2, window=window)
    row_case("outlier first", n, G, d, fmt, 300, 200, window=window, softcap=20.0)


@pytest.mark.parametrize("n,G,d,fmt", FEW)
def test_few_rows_faint_page(n, G, d, fmt):
    """A bias leaves the outlier's page a weight that its scale makes up for, or next to none."""
    row_case("outlier first", n, G, d, fmt, 250, 2, slopes=[0.2, 0.25, 0.17, 1.0, 0.21, 0.15, 0.22, 0.3][: HKV * G])


MANY = [(100, 4, 128, "e4m3"), (100, 1, 64, "int8"), (40, 3, 128, "int8"), (300, 2, 64, "e4m3")]     # 256-row tiles


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,G,d,fmt", MANY)
def test_many_rows(kind, n, G, d, fmt):
    row_case(kind, n, G, d, fmt, 320, 2)
    row_case(kind, n, G, d, fmt, 320, 2, seed=1, mask="full", softcap=20.0)
    row_case(kind, n, G, d, fmt, 1500, 2, seed=2, page=64)                # cut among blocks
    row_case(kind, n, G, d, fmt, 310, 2, seed=3, slopes=[0.3, 0.1, 0.2, 0.25, 0.4, 0.15, 0.22, 0.35][: HKV * G])


@pytest.mark.parametrize("n,G,d,fmt", MANY)
def test_many_rows_hidden_page(n, G, d, fmt):
    first = (np.arange(n) * 7 % 80).astype(np.int32)            # of the outliers' 32 keys queries see all, some or none
    row_case("outlier first", n, G, d, fmt, 320, 2, first=first)
    row_case("outlier first", n, G, d, fmt, 1320, 2, first=first, mask="full")


@pytest.mark.parametrize("n", [1, 70])
def test_lse_of_long_heads_of_zeros(n):
    """V all zero, as a store leaves it, in 200 rows of the same 40000 keys whose first score lower than the rest: the
    sum stays finite, also where a block takes all keys of a row.  Every score is 64 ones times a code and a scale:
    exact but for the scale's three roundings, so the sum is known."""
    L, page, d, rows = 40000, 128, 64, 200
    cache = random_cache(np.random.default_rng(0), 320, HKV, page, d, "int8")
    cache["k"][:] = 64
    cache["v"][:] = 0
    cache["vs"][:] = 2.0 ** -126
    cache["ks"][:] = np.float32(4.7 / 512)
    cache["ks"][5] = 0.0
    ids = np.r_[5, np.delete(np.arange(320), 5)][None, : -(-L // page)]
    pc = to_device(cache)
    q = torch.ones((rows * n, HKV, d), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda"), torch.full(q.shape[:2], 7.0, device="cuda")
    pc.attend(i32(ids.repeat(rows, 0)), i32([L] * rows), i32(np.arange(rows + 1) * n), q, out, lse, max_q=n, mask="full")
    assert pc.device_status() == 0
    score = 512 * float(np.float32(4.7 / 512))
    want = score + np.log(L - page + page * np.exp(-score))
    # (the sum of at most 40000 terms of one sign, in any order: each addition 2^-24 of it; hundreds in a chain)
    assert (lse.double() - want).abs().max().item() <= 2.0 ** -24 * (16 * want + 16 * score + 1000)
    assert not out.any()


@pytest.mark.parametrize("n,G,L,extra", [(66, 5, 671, 20), (66, 1, 671, 20), (66, 1, 256, 1), (1, 4, 671, 20), (1, 4, 256, 1),
                                         (9, 2, 671, 20)])
def test_faint_pages_of_larger_scales(n, G, L, extra):
    """The last pages hold the smallest scales and nearly all weight; the ones before, whose weights a bias brings to
    2^-50 to 2^-90, have scales that make up for it.  In one block, and cut among blocks."""
    rng = np.random.default_rng(n + L)
    page, d = 128, 64
    pages = -(-L // page)
    cache = random_cache(rng, pages + 2, HKV, page, d, "int8")
    table = random_table(rng, [L], page, pages + 2, extra)
    last = 2 if L > 256 else 1
    cache["vs"][table[0, : pages - last]] = 2.0 ** -50
    cache["vs"][table[0, pages - last: pages]] = 2.0 ** -126
    q, q64 = bf16(rng.standard_normal((n, HKV * G, d)))
    check(cache, table, np.array([L]), np.array([0, n]), q, q64, dict(mask="full", slopes=[0.388] * (HKV * G)))
