"""The paged 8-bit cache on the GPU against its oracle in 64 bits: the attention
(types, head layouts, lengths, masks, scales, strides, streams, faults), the
store, fork and compact (bit for bit), and a beam decode of them together."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.cache as oc
from shared_prefix_decode_xattention_b200 import xgr
from tests.cache_harness import (DT, bf16, close, i32, random_cache, random_table, same_cache, to_device,
                                 to_host)

pytestmark = pytest.mark.gpu


def attend_case(seed, lens, n, hkv, G, page, d, fmt, spread=1.0, q_scale=1.0, cap=0.0, window=0, slopes=None,
                mask="causal", prefix=None, first=None, scale=0.0, edit=None, junk=-1, extra=2, max_q=None):
    """One call against the oracle; `edit(cache)` may spoil what must not be read."""
    rng = np.random.default_rng(seed)
    lens, n = np.asarray(lens), np.asarray(n)
    n_pages = int(sum(-(-int(x) // page) for x in lens)) + 4
    cache = random_cache(rng, n_pages, hkv, page, d, fmt, spread)
    table = random_table(rng, lens, page, n_pages, extra, junk)
    cu = np.concatenate([[0], np.cumsum(n)])
    T, hq = int(cu[-1]), hkv * G
    q, q64 = bf16(rng.standard_normal((T, hq, d)) * q_scale)
    ref, ref_lse = oc.attend(cache, table, lens, cu, q64, mask, scale, cap, window, slopes, prefix, first)
    if edit:
        edit(cache, table)
    pc = to_device(cache)
    out = torch.full((T, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T, hq), 7.0, device="cuda")
    pc.attend(i32(table), i32(lens), i32(cu), q, out, lse, max_q=int(n.max()) if max_q is None else max_q,
              scale=scale, softcap=cap, mask=mask, window=window,
              slopes=None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device="cuda"),
              prefix=None if prefix is None else i32(prefix), first=None if first is None else i32(first))
    assert pc.device_status() == 0
    vmax, qk = np.zeros((T, hq, 1)), 0.0
    for r in range(len(lens)):
        for g in range(hkv if n[r] else 0):
            k, v = oc.row_kv(cache if not edit else clean_copy(cache), table[r], int(lens[r]), g)
            h = slice(g * G, (g + 1) * G)
            vmax[cu[r]:cu[r + 1], h] = np.nanmax(np.abs(v), initial=0)
            x = np.einsum("thd,kd->thk", np.abs(q64[cu[r]:cu[r + 1], h]), np.abs(k))
            qk = max(qk, np.nanmax(x, initial=0) * (scale or d ** -0.5))
    if slopes is not None:
        qk += float(np.max(slopes)) * int(lens.max()) / 8
    close(out, lse, ref, ref_lse, vmax, d, qk)
    return out, lse


def clean_copy(cache):
    c = dict(cache)
    c["ks"], c["vs"] = np.nan_to_num(cache["ks"]), np.nan_to_num(cache["vs"])
    return c


LENS = [1, 15, 16, 17, 31, 33, 127, 128, 129, 255, 257, 700]


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_attend_single_tokens(page, d, fmt):
    attend_case(page + d, LENS, np.ones(len(LENS), int), 2, 4, page, d, fmt)


@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 16, 17, 32, 40])
def test_attend_head_layouts(G):
    attend_case(G, [1, 40, 300], [1, 1, 1], 1 + (G % 3), G, 32, 128 if G % 2 else 64, "e4m3" if G % 2 else "int8")


@pytest.mark.parametrize("mask", ["full", "causal", "prefix"])
@pytest.mark.parametrize("kw", [dict(), dict(window=1), dict(window=37), dict(cap=20.0), dict(slopes=[0.5, 0.25, 0.125, 1.0]),
                                dict(cap=5.0, window=50, slopes=[0.01, 0.3, 0.0, 0.07], first=True)])
def test_attend_masks_and_scores(mask, kw):
    lens, n = [0, 5, 33, 64, 200, 450], [0, 5, 1, 0, 21, 40]
    kw = dict(kw)
    T = sum(n)
    if kw.get("first"):
        # documents; some queries' first key lies behind the query itself: nothing is seen
        kw["first"] = np.random.default_rng(5).integers(0, 460, T).astype(np.int32)
    prefix = [3, 9, 12, 1, 190, 1000] if mask == "prefix" else None
    for d, fmt, page in ((64, "int8", 16), (128, "e4m3", 64)):
        attend_case(11, lens, n, 2, 2, page, d, fmt, mask=mask, prefix=prefix, **kw)


@pytest.mark.parametrize("n,G,d", [(128, 4, 128), (130, 4, 64), (33, 1, 128), (9, 4, 128), (300, 1, 64), (64, 2, 128)])
@pytest.mark.parametrize("mask", ["full", "causal"])
def test_attend_many_rows(n, G, d, mask):
    """Tiles of more query rows than a decode step's, whole and ragged ones."""
    attend_case(n + G, [max(n, 500), n, n + 1], [n, n, 1], 1, G, 64, d, "e4m3", mask=mask)


def test_attend_many_rows_masked():
    rng = np.random.default_rng(9)
    lens, n = [600, 260], [150, 200]
    first = rng.integers(0, 700, 350).astype(np.int32)
    for kw in (dict(cap=30.0, mask="prefix", prefix=[400, 100]), dict(window=90, slopes=[0.1, 0.02]),
               dict(first=first), dict(first=first, mask="full", window=64)):
        attend_case(3, lens, n, 1, 2, 32, 128, "int8", **kw)
        attend_case(3, lens, n, 1, 2, 16, 64, "e4m3", **kw)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_attend_long_rows_are_split(fmt):
    attend_case(4, [20011, 3, 9000], [1, 1, 1], 2, 4, 128, 128, fmt)
    attend_case(4, [20011, 3, 9000], [2, 1, 3], 1, 8, 64, 64, fmt, slopes=[0.001] * 8, cap=30.0)
    attend_case(5, [30000], [1], 1, 1, 16, 128, fmt, window=25000)


def test_attend_many_rows_long():
    attend_case(6, [9001, 40], [70, 40], 1, 4, 64, 128, "e4m3", mask="full")
    attend_case(6, [9001, 40], [70, 40], 1, 4, 64, 128, "int8", cap=50.0)


@pytest.mark.parametrize("n", [1, 100])
def test_attend_scales_of_any_size(n):
    """V scales up to 2^24 apart (K's stay near each other, or one key takes all)."""
    for d, fmt in ((64, "e4m3"), (128, "int8")):
        rng = np.random.default_rng(2)
        lens = np.array([300, 450])
        cache = random_cache(rng, 50, 2, 16, d, fmt, 1.0)
        cache["vs"] *= (2.0 ** rng.integers(-12, 13, cache["vs"].shape)).astype(np.float32)
        cache["vs"][rng.random(cache["vs"].shape) < 0.2] = 0.0       # pages of zeros
        cache["ks"][rng.random(cache["ks"].shape) < 0.1] = 0.0
        table = random_table(rng, lens, 16, 50)
        cu = np.array([0, n, n + 1])
        q, q64 = bf16(rng.standard_normal((n + 1, 4, d)))
        ref, ref_lse = oc.attend(cache, table, lens, cu, q64)
        pc = to_device(cache)
        out, lse = torch.empty_like(q), torch.empty((n + 1, 4), device="cuda")
        pc.attend(i32(table), i32(lens), i32(cu), q, out, lse, max_q=n)
        vmax = np.zeros((n + 1, 4, 1))
        for r in range(2):
            for g in range(2):
                vmax[cu[r]:cu[r + 1], 2 * g: 2 * g + 2] = np.abs(oc.row_kv(cache, table[r], lens[r], g)[1]).max()
        close(out, lse, ref, ref_lse, vmax, d, 40.0)


@pytest.mark.parametrize("q_scale", [2.0 ** -100, 2.0 ** 90, 1e-30])
def test_attend_queries_of_any_size(q_scale):
    """The scale takes the queries' size back, as a caller with unnormalised queries would."""
    attend_case(8, [100, 50], [1, 20], 2, 2, 32, 128, "int8", q_scale=q_scale, scale=float(0.09 / q_scale))


@pytest.mark.parametrize("n", [1, 90])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_attend_reads_nothing_behind_a_row(n, fmt):
    """NaN codes, NaN scales and page ids of nowhere behind the rows' ends."""
    lens = [max(n, 100), 161, 90]

    def spoil(cache, table):
        held = set()
        for r, L in enumerate(lens):
            for p in range(-(-L // 64)):
                pid = int(table[r, p])
                held.add(pid)
                end = min(64, L - 64 * p)
                cache["k"][pid, :, end:] = 0x7f
                cache["v"][pid, :, end:] = 0xff
        for pid in set(range(cache["k"].shape[0])) - held:
            cache["k"][pid] = cache["v"][pid] = 0x7f
            cache["ks"][pid] = cache["vs"][pid] = np.nan
    attend_case(12, lens, [n, 1, 1], 2, 2, 64, 128, fmt, edit=spoil, junk=1 << 29, extra=40)
    attend_case(12, lens, [n, 1, 1], 2, 2, 64, 64, fmt, edit=spoil, junk=-7, extra=1)


@pytest.mark.parametrize("n", [1, 80])
def test_attend_masked_nan_pages(n):
    """A page whose scales are NaN (a store met a NaN): queries that do not see it are exact, those that do are NaN."""
    rng = np.random.default_rng(3)
    L, page = 300, 64
    cache = random_cache(rng, 6, 1, page, 128, "e4m3")
    table = random_table(rng, [L], page, 6)
    cu = np.array([0, n])
    q, q64 = bf16(rng.standard_normal((n, 2, 128)))
    first = np.where(np.arange(n) % 2 == 0, 70, 10).astype(np.int32)      # page 0 (keys 0..63): hidden from even ones
    ref, ref_lse = oc.attend(cache, table, [L], cu, q64, first=first)
    for which in ("ks", "vs"):
        sick = {**cache, which: cache[which].copy()}
        sick[which][table[0, 0]] = np.nan
        pc = to_device(sick)
        out, lse = torch.empty_like(q), torch.empty((n, 2), device="cuda")
        pc.attend(i32(table), i32([L]), i32(cu), q, out, lse, max_q=n, first=i32(first))
        assert torch.isnan(out[1::2]).all() and (which == "vs" or torch.isnan(lse[1::2]).all())
        vmax = np.full((n, 2, 1), np.abs(oc.row_kv(cache, table[0], L, 0)[1]).max())
        close(out[::2], lse[::2], ref[::2], ref_lse[::2], vmax[::2], 128, 40.0)


@pytest.mark.parametrize("most,G", [(1, 4), (9, 3), (40, 2)])
def test_attend_many_ragged_rows(most, G):
    """More rows (and tiles) than the plan has threads, rows without tokens and without keys among them."""
    rng = np.random.default_rng(most)
    n_rows = 2100 if most == 1 else 800
    n = np.minimum(rng.integers(0, most + 1, n_rows), rng.integers(0, most + 1, n_rows))
    lens = np.maximum(n, rng.integers(0, 60, n_rows))
    lens[5], n[5] = 2500, most
    attend_case(most, lens, n, 2, G, 16, 64, "int8" if most == 9 else "e4m3", extra=1, window=0 if most == 1 else 50)


def test_attend_few_long_segments_of_many_rows():
    """Few 256-row segments over long keys (equal parts), beside one with many (a line of units)."""
    attend_case(1, [5000], [65], 1, 4, 128, 64, "int8", mask="full")                    # a whole tile and a narrow one
    attend_case(2, [3000, 2000], [64, 128], 2, 2, 64, 128, "e4m3", mask="full")         # narrow, whole
    attend_case(3, [400, 300, 260, 220, 1400], [260, 256, 200, 130, 300], 2, 2, 64, 64, "e4m3")


def test_attend_captured_graphs_on_two_streams():
    """Two graphs, captured on two streams of one cache, replayed at the same time."""
    rng = np.random.default_rng(4)
    cache = random_cache(rng, 300, 2, 32, 64, "e4m3")
    pc = to_device(cache)
    lens = np.array([4000, 3900])
    t, ln = i32(random_table(rng, lens, 32, 300)), i32(lens)
    runs = []
    for n in (1, 50):
        s, cu = torch.cuda.Stream(), i32([0, n, 2 * n])
        q, _ = bf16(rng.standard_normal((2 * n, 4, 64)))
        o, z = torch.empty_like(q), torch.empty((2 * n, 4), device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            pc.attend(t, ln, cu, q, o, z, max_q=n)
        torch.cuda.synchronize()
        want = o.clone(), z.clone()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            for _ in range(20):
                pc.attend(t, ln, cu, q, o, z, max_q=n)
        runs.append((s, g, o, z, want, cu, q))
    for _ in range(5):
        for s, g, o, z, *_ in runs:
            with torch.cuda.stream(s):
                o.zero_()
                g.replay()
        torch.cuda.synchronize()
        for s, g, o, z, want, *_ in runs:
            assert torch.equal(o, want[0]) and torch.equal(z, want[1])
    assert pc.device_status() == 0


def test_whole_step_in_one_graph():
    """Fork, store, attend and compact captured on torch's own capture stream with a workspace of their own, and
    replayed on other inputs."""
    rng = np.random.default_rng(4)
    cache = random_cache(rng, 64, 2, 16, 64, "int8")
    pc = to_device(cache)
    rows, width = 6, 8
    lens = np.array([40, 33, 64, 1, 80, 17], np.int32)
    table = random_table(rng, lens, 16, 64, extra=3)
    t, ln, par = i32(table), i32(lens), i32(np.arange(rows))
    t2, l2, t3, used = i32(np.zeros((rows, width))), i32(np.zeros(rows)), i32(np.zeros((rows, width))), i32([0])
    ones, cu = i32(np.ones(rows)), i32(np.arange(rows + 1))
    k, _ = bf16(rng.standard_normal((rows, 2, 64)))
    q, _ = bf16(rng.standard_normal((rows, 4, 64)))
    o, z = torch.empty_like(q), torch.empty((rows, 4), device="cuda")
    need = max(pc.attend_bytes(4, rows, rows), pc.fork_bytes(rows, rows), pc.compact_bytes())
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def step():
        pc.fork(t, ln, par, ones, t2, l2, workspace=ws)
        pc.store(t2, l2, cu, k, k, max_n=1)
        pc.attend(t2, l2, cu, q, o, z, max_q=1, workspace=ws)
        pc.compact(t2, l2, t3, used, workspace=ws)
    with pytest.raises(xgr.XgrError) as e:
        pc.fork(t, ln, par, ones, t2, l2, workspace=ws[:256])
    assert e.value.status == xgr.XGR_ERR_CAPACITY
    step()
    torch.cuda.synchronize()
    for x, c in (("k", pc.k), ("v", pc.v)):
        c.view(torch.uint8).copy_(torch.from_numpy(cache[x]))
    pc.k_scale.copy_(torch.from_numpy(cache["ks"]))
    pc.v_scale.copy_(torch.from_numpy(cache["vs"]))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        parent = rng.integers(0, rows, rows).astype(np.int32)
        par.copy_(i32(parent))
        k2, k64 = bf16(rng.standard_normal((rows, 2, 64)))
        q2, q64 = bf16(rng.standard_normal((rows, 4, 64)))
        k.copy_(k2)
        q.copy_(q2)
        t.copy_(i32(table))
        ln.copy_(i32(lens))
        g.replay()
        torch.cuda.synchronize()
        want_t, want_l, _ = oc.fork(cache, table, lens, parent, np.ones(rows, np.int32))
        oc.store(cache, want_t, want_l, np.arange(rows + 1), k64, k64)
        ref, ref_lse = oc.attend(cache, want_t, want_l, np.arange(rows + 1), q64)
        close(o, z, ref, ref_lse, np.full((rows, 4, 1), 16.0), 64, 40.0)
        table, u = oc.compact(cache, want_t, want_l)
        lens = want_l
        assert np.array_equal(t3.cpu().numpy(), table) and used.item() == u
        same_cache(to_host(pc), cache)
    assert pc.device_status() == 0


def test_calls_from_two_threads():
    """Host threads with a stream each use one cache at the same time."""
    import threading
    rng = np.random.default_rng(4)
    cache = random_cache(rng, 300, 2, 32, 64, "int8")
    pc = to_device(cache)
    lens = np.array([3000, 2900])
    t, ln = i32(random_table(rng, lens, 32, 300)), i32(lens)
    q, _ = bf16(rng.standard_normal((80, 4, 64)))
    ref = {}
    for n in (1, 40):
        o, z = torch.empty_like(q[:2 * n]), torch.empty((2 * n, 4), device="cuda")
        pc.attend(t, ln, i32([0, n, 2 * n]), q[:2 * n], o, z, max_q=n)
        ref[n] = o
    torch.cuda.synchronize()
    bad = []

    def work(n):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            cu = i32([0, n, 2 * n])
            o, z = torch.empty_like(q[:2 * n]), torch.empty((2 * n, 4), device="cuda")
            for _ in range(50):
                o.zero_()
                pc.attend(t, ln, cu, q[:2 * n], o, z, max_q=n)
                s.synchronize()
                if not torch.equal(o, ref[n]):
                    bad.append(n)
    threads = [threading.Thread(target=work, args=(n,)) for n in (1, 40, 1, 40)]
    for x in threads:
        x.start()
    for x in threads:
        x.join()
    assert not bad and pc.device_status() == 0


def test_attend_strided_queries_and_spare_tokens():
    """q as a slice of a fused projection; tokens behind the last row stay as they are."""
    rng = np.random.default_rng(1)
    cache = random_cache(rng, 30, 2, 16, 64, "int8")
    lens, cu = np.array([50, 77, 20]), np.array([0, 1, 1, 6])
    table = random_table(rng, lens, 16, 30)
    T = 9
    fused, f64 = bf16(rng.standard_normal((T, 8 + 4, 64)))
    ref, ref_lse = oc.attend(cache, table, lens, cu, f64[:, 2:10])
    pc = to_device(cache)
    q = fused[:, 2:10]
    out, lse = torch.full((T, 8, 64), 3.0, dtype=torch.bfloat16, device="cuda"), torch.full((T, 8), 3.0, device="cuda")
    pc.attend(i32(table), i32(lens), i32(cu), q, out, lse, max_q=5)
    assert (out[6:] == 3).all() and (lse[6:] == 3).all()
    vmax = np.full((6, 8, 1), 127 * cache["vs"].max())
    close(out[:6], lse[:6], ref[:6], ref_lse[:6], vmax, 64, 40.0)


def test_attend_is_the_same_twice_and_on_other_streams():
    rng = np.random.default_rng(1)
    cache = random_cache(rng, 400, 2, 64, 128, "e4m3")
    lens = np.array([9000, 700, 9000])
    table = i32(random_table(rng, lens, 64, 400))
    pc = to_device(cache)
    for n in (1, 60):
        cu = i32([0, n, 2 * n, 3 * n])
        q, _ = bf16(rng.standard_normal((3 * n, 8, 128)))
        got = []
        streams = [torch.cuda.current_stream(), torch.cuda.Stream(), torch.cuda.Stream()]
        torch.cuda.synchronize()
        for s in streams:
            o, z = torch.empty_like(q), torch.empty((3 * n, 8), device="cuda")
            with torch.cuda.stream(s):
                for _ in range(3):
                    pc.attend(table, i32(lens), cu, q, o, z, max_q=n)
            got.append((o, z))
        torch.cuda.synchronize()
        for o, z in got[1:]:
            assert torch.equal(o, got[0][0]) and torch.equal(z, got[0][1])
    assert pc.device_status() == 0


@pytest.mark.parametrize("d,G,lo,hi", [(128, 2, 4, 14), (128, 2, 20, 40), (64, 2, 4, 16), (128, 4, 1, 4), (64, 4, 30, 200),
                                       (128, 4, 40, 300)])
def test_attend_is_the_same_every_time(d, G, lo, hi):
    """Ragged rows, many segments a CTA, cut ones among them, some hundred times: a race would show."""
    rng = np.random.default_rng(hi)
    n_rows, hkv, page = 99, 8, 128
    n = rng.integers(lo, hi + 1, n_rows)
    lens = np.maximum(n, rng.integers(18, 1815, n_rows))
    n_pages = int(sum(-(-int(x) // page) for x in lens)) + 4
    g = torch.Generator(device="cuda").manual_seed(1)
    from shared_prefix_decode_xattention_b200.cache import PagedCache
    k, v = (torch.randint(-127, 128, (n_pages, hkv, page, d), generator=g, device="cuda", dtype=torch.int8) for _ in range(2))
    ks, vs = (torch.rand((n_pages, hkv), generator=g, device="cuda") / 73 for _ in range(2))
    pc = PagedCache(k, v, ks, vs)
    t, ln, cu = i32(random_table(rng, lens, page, n_pages)), i32(lens), i32(np.concatenate([[0], np.cumsum(n)]))
    T = int(n.sum())
    q = torch.randn((T, hkv * G, d), generator=g, device="cuda").to(torch.bfloat16)
    o, z = torch.empty_like(q), torch.empty((T, hkv * G), device="cuda")
    pc.attend(t, ln, cu, q, o, z, max_q=hi)
    first = o.clone(), z.clone()
    same = torch.ones((), dtype=torch.bool, device="cuda")
    for _ in range(300):
        o.zero_()
        pc.attend(t, ln, cu, q, o, z, max_q=hi)
        same &= (o == first[0]).all() & (z == first[1]).all()
    assert same.item() and pc.device_status() == 0


def test_attend_captured_and_replayed():
    """A graph follows the lengths, tables and queries in its buffers; a capture without a workspace is refused."""
    rng = np.random.default_rng(1)
    cache = random_cache(rng, 60, 2, 32, 64, "int8")
    pc, fresh = to_device(cache), to_device(cache)
    lens = np.array([1300, 100])
    table = random_table(rng, lens, 32, 60)
    t, ln, cu = i32(table), i32(lens), i32([0, 1, 2])
    q, q64 = bf16(rng.standard_normal((2, 4, 64)))
    o, z = torch.empty_like(q), torch.empty((2, 4), device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        pc.attend(t, ln, cu, q, o, z, max_q=1)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        with pytest.raises(xgr.XgrError) as e:
            fresh.attend(t, ln, cu, q, o, z, max_q=1)
        pc.attend(t, ln, cu, q, o, z, max_q=1)
    assert e.value.status == xgr.XGR_ERR_STATE
    for L in ([1300, 100], [3, 77], [640, 1]):
        q2, q64 = bf16(rng.standard_normal((2, 4, 64)))
        q.copy_(q2)
        ln.copy_(i32(L))
        g.replay()
        torch.cuda.synchronize()
        ref, ref_lse = oc.attend(cache, table, L, [0, 1, 2], q64)
        close(o, z, ref, ref_lse, np.full((2, 4, 1), 127 * cache["vs"].max()), 64, 40.0)


@pytest.mark.parametrize("n", [1, 50])
def test_attend_reports_faults_and_goes_on(n):
    rng = np.random.default_rng(1)
    cache = random_cache(rng, 40, 1, 16, 64, "e4m3")
    lens = np.array([60, 60, 60, 60])
    lens[0] = max(n, 60)
    table = random_table(rng, lens, 16, 40)
    q, q64 = bf16(rng.standard_normal((4 * n, 2, 64)))
    good = np.array([0, n, 2 * n, 3 * n, 4 * n])

    def go(t, ln, cu, max_q=n, want=0):
        pc = to_device(cache)
        o = torch.full((4 * n, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda")
        z = torch.full((4 * n, 2), 5.0, device="cuda")
        pc.attend(i32(t), i32(ln), i32(cu), q, o, z, max_q=max_q)
        assert pc.device_status() == want
        return o.float().cpu().numpy(), z.cpu().numpy()
    base, base_z = go(table, lens, good)
    # a page that is not there: its keys are not attended
    for pid in (-1, 40, 1 << 30):
        t = table.copy()
        t[1, 1] = pid
        o, z = go(t, lens, good, want=xgr.XGR_DEV_INDEX)
        rows = np.r_[0:n, 2 * n:4 * n]
        assert np.array_equal(o[rows], base[rows]) and np.isfinite(o).all()
        k, v = oc.row_kv(cache, table[1], 60, 0)
        i = n - 1                                        # the row's last query sees all 60 keys but 16..31
        x = np.delete(k, np.s_[16:32], 0) @ q64[n + i].T * 64 ** -0.5
        w = np.exp(x - x.max(0))
        want = (w / w.sum(0)).T @ np.delete(v, np.s_[16:32], 0)
        assert np.abs(o[n + i] - want).max() <= (2.0 ** -8 + 2.0 ** -10) * np.abs(v).max()
    # lengths and token ranges that do not fit: the row has no tokens
    for bad_len, bad_cu in ((np.array([lens[0], -1, 60, 60]), good), (np.array([lens[0], 1 << 30, 60, 60]), good),
                            (np.array([lens[0], n - 1, 60, 60]), good)):
        o, z = go(table, bad_len, bad_cu, want=xgr.XGR_DEV_INDEX)
        assert (o[n:2 * n] == 5).all() and (z[n:2 * n] == 5).all()
        assert np.array_equal(np.delete(o, np.s_[n:2 * n], 0), np.delete(base, np.s_[n:2 * n], 0))
    go(table, lens, [0, n, 2 * n, 3 * n, 4 * n + 1], want=xgr.XGR_DEV_INDEX)
    go(table, lens, [0, -5, 2 * n, 3 * n, 4 * n], want=xgr.XGR_DEV_INDEX)
    if n > 1:
        go(table, lens, good, max_q=n - 1, want=xgr.XGR_DEV_CAPACITY)


def test_attend_pages_past_32_bit_offsets():
    """Page ids whose codes lie more than 2^31 bytes into the cache."""
    n_pages, hkv, page, d = 300000, 1, 64, 128
    from shared_prefix_decode_xattention_b200.cache import PagedCache
    pc = PagedCache.create(n_pages, hkv, page, d, torch.int8)
    rng = np.random.default_rng(1)
    ids = np.array([n_pages - 1, 5, 290000, 270001, n_pages - 2])
    small = random_cache(rng, 5, hkv, page, d, "int8")
    where = torch.tensor(ids, device="cuda")
    for x, t in (("k", pc.k), ("v", pc.v)):
        t.view(torch.uint8)[where] = torch.from_numpy(small[x]).cuda()
    pc.k_scale[where] = torch.from_numpy(small["ks"]).cuda()
    pc.v_scale[where] = torch.from_numpy(small["vs"]).cuda()
    L = 5 * page - 3
    for n in (1, 40):
        q, q64 = bf16(rng.standard_normal((n, 4, d)))
        o, z = torch.empty_like(q), torch.empty((n, 4), device="cuda")
        pc.attend(i32(ids[None]), i32([L]), i32([0, n]), q, o, z, max_q=n)
        ref, ref_lse = oc.attend(small, np.arange(5)[None], [L], [0, n], q64)
        close(o, z, ref, ref_lse, np.full((n, 4, 1), 127 * small["vs"].max()), d, 40.0)
    # the same tokens stored, forked and moved there
    k, k64 = bf16(rng.standard_normal((7, hkv, d)))
    oc.store(small, np.arange(5)[None], [L], [0, 7], k64, k64)
    pc.store(i32(ids[None]), i32([L]), i32([0, 7]), k, k, max_n=7)
    t2, l2 = i32(np.zeros((2, 5))), i32([0, 0])
    pc.fork(i32(ids[None]), i32([L]), i32([0, 0]), None, t2, l2)
    assert t2[1].tolist() == [*ids[:4], 0]
    t3, used = i32(np.zeros((2, 5))), i32([0])
    pc.compact(t2, l2, t3, used)
    assert used.item() == 6 and pc.device_status() == 0
    assert t3.tolist() == [[4, 5, 2, 1, 3], [4, 5, 2, 1, 0]]
    for j, pid in enumerate(t3[0].tolist()):
        assert np.array_equal(pc.k[pid].view(torch.uint8).cpu().numpy(), small["k"][j]), j
    assert np.array_equal(pc.v[t3[1, 4].item()].view(torch.uint8).cpu().numpy(), small["v"][4])


# ------------------------------------------------------------------ store

def store_case(rng, cache, table, lens, n, scale=1.0, edit=None, stride_extra=0):
    hkv, d = cache["k"].shape[1], cache["k"].shape[3]
    cu = np.concatenate([[0], np.cumsum(n)])
    T = int(cu[-1])
    x = rng.standard_normal((2, T, hkv + stride_extra, d)) * np.asarray(scale)
    if edit:
        edit(x)
    k, k64 = bf16(x[0])
    v, v64 = bf16(x[1])
    pc = to_device(cache)
    pc.store(i32(table), i32(lens), i32(cu), k[:, :hkv], v[:, :hkv], max_n=int(np.max(n)))
    oc.store(cache, table, lens, cu, k64[:, :hkv], v64[:, :hkv])
    assert pc.device_status() == 0
    same_cache(to_host(pc), cache)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_store_is_exact(page, d, fmt):
    rng = np.random.default_rng(page + d)
    lens = np.array([1, 40, 0, 129, 256, 333, 17, 2 * page, page + 1])
    n = np.array([1, 39, 0, 1, 256, 100, 0, page, 2])
    cache = random_cache(rng, 60, 3, page, d, fmt)
    for s in ("ks", "vs"):
        cache[s] = (2.0 ** np.round(np.log2(cache[s]))).astype(np.float32)
    table = random_table(rng, lens, page, 60)
    store_case(rng, cache, table, lens, n, stride_extra=2)
    # one more token a row (as a decode step appends), small, then large enough to make every scale grow
    for s in (0.01, 1000.0):
        lens = np.minimum(lens + 1, table.shape[1] * page)
        room = np.array([table[r, (lens[r] - 1) // page] >= 0 for r in range(len(lens))])
        store_case(rng, cache, table, np.where(room, lens, lens - 1), room.astype(int), s)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_store_values_at_the_edges(fmt):
    """Zeros, the smallest and largest numbers, ties, negative zeros; scales that are no powers of two."""
    rng = np.random.default_rng(0)

    def edit(x):
        x[:, :16] = 0
        x[:, 16:32] *= 2.0 ** -130
        x[:, 32:48] *= 2.0 ** 120
        x[:, 48:64] = np.round(x[:, 48:64] * 8) * 2.5
        x[:, 50, 0] = 448.0
        x[:, 64:80, :, ::2] = -0.0
        x[:, 96:112] = 127 * 2.0 ** rng.integers(-9, -7, x[:, 96:112].shape)
    cache = random_cache(rng, 12, 2, 16, 64, fmt)
    table = random_table(rng, [180], 16, 12)
    store_case(rng, cache, table, [115], [115], edit=edit)
    cache["ks"] *= np.float32(1.37)
    store_case(rng, cache, table, [120], [5])


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_store_marks_pages_that_get_no_number(fmt, bad):
    rng = np.random.default_rng(0)
    cache = random_cache(rng, 12, 2, 16, 64, fmt)
    table = random_table(rng, [64, 64], 16, 12)

    def edit(x):
        x[0, 20, 1, 3] = bad
        x[1, 45, 0, 63] = bad
    store_case(rng, cache, table, [40, 30], [40, 30], edit=edit)
    assert np.isnan(cache["ks"]).sum() == 1 and np.isnan(cache["vs"]).sum() == 1
    store_case(rng, cache, table, [44, 32], [4, 2])          # appended: stays marked
    assert np.isnan(cache["ks"]).sum() == 1
    store_case(rng, cache, table, [30, 32], [30, 0])         # begun anew
    assert np.isnan(cache["ks"]).sum() == 0


def test_store_faults():
    rng = np.random.default_rng(0)
    cache = random_cache(rng, 12, 2, 16, 64, "int8")
    lens, cu = np.array([40, 30]), np.array([0, 20, 35])
    table = random_table(rng, lens, 16, 12)
    k, _ = bf16(rng.standard_normal((35, 2, 64)))

    def go(t, ln, c, max_n=20, want=0):
        pc = to_device(cache)
        pc.store(i32(t), i32(ln), i32(c), k, k, max_n=max_n)
        assert pc.device_status() == want
        return to_host(pc)
    t = table.copy()
    t[0, 2] = 12
    got, base = go(t, lens, cu, want=xgr.XGR_DEV_INDEX), go(table, lens, cu)
    for x in ("k", "v", "ks", "vs"):
        base[x][table[0, 2]] = cache[x][table[0, 2]]
    same_cache(got, base)
    for ln, c, m, want in (([40, 14], cu, 20, xgr.XGR_DEV_INDEX), ([40, 1000], cu, 20, xgr.XGR_DEV_INDEX),
                           (lens, [0, 20, 36], 20, xgr.XGR_DEV_INDEX), (lens, [0, 15, 35], 19, xgr.XGR_DEV_CAPACITY),
                           (lens, [5, 1, 16], 20, xgr.XGR_DEV_INDEX)):
        go(table, ln, c, m, want)


# ------------------------------------------------------------------ fork, compact

def shared_tables(rng, cache_pages, page, width, n_rows):
    """Rows that share prompts: full pages in common, tails of their own."""
    order = rng.permutation(cache_pages)
    prompts, at = [], 0
    for _ in range(3):
        m = int(rng.integers(0, width - 3))
        prompts.append(order[at: at + m])
        at += m
    table, lens = np.full((n_rows, width), -1, dtype=np.int32), np.zeros(n_rows, dtype=np.int32)
    for r in range(n_rows):
        p = prompts[rng.integers(3)]
        own = int(rng.integers(0, 3))
        if at + own > cache_pages:
            own = 0
        table[r, :len(p)] = p
        table[r, len(p): len(p) + own] = order[at: at + own]
        at += own
        lens[r] = len(p) * page + (max(own - 1, 0) * page + int(rng.integers(1, page + 1)) if own else 0)
    return table, lens


@pytest.mark.parametrize("seed", range(8))
def test_fork_is_exact(seed):
    rng = np.random.default_rng(seed)
    page, d = [16, 32, 64, 128][seed % 4], [64, 128][seed // 4]
    fmt = "e4m3" if seed % 2 else "int8"
    n_rows, width = int(rng.integers(1, 40)), 8
    pages = [70, 200, 1100, 45][seed % 4]
    cache = random_cache(rng, pages, 1 + seed % 3, page, d, fmt)
    table, lens = shared_tables(rng, pages, page, width, n_rows)
    pc = to_device(cache)
    for step in range(4):
        n_out = int(rng.integers(1, 50))
        parent = rng.integers(-1, len(lens), n_out).astype(np.int32)
        n_new = rng.integers(0, 2 * page, n_out).astype(np.int32) if step != 2 else None
        t2, l2 = i32(np.zeros((n_out, width))), i32(np.zeros(n_out))
        pc.fork(i32(table), i32(lens), i32(parent), None if n_new is None else i32(n_new), t2, l2)
        want_t, want_l, st = oc.fork(cache, table, lens, parent, n_new)
        assert np.array_equal(t2.cpu().numpy(), want_t) and np.array_equal(l2.cpu().numpy(), want_l)
        same_cache(to_host(pc), cache)
        assert pc.device_status() == st
        table, lens = want_t, want_l


@pytest.mark.parametrize("pages", [70001, 800003])
def test_fork_many_pages_and_rows(pages):
    """More rows and pages than one share of the plan; more pages than its bitsets in shared memory hold (786432)."""
    rng = np.random.default_rng(0)
    page, width = 16, 5
    cache = random_cache(rng, pages, 1, page, 64, "int8")
    n = 2500
    lens = rng.integers(0, 3 * page, n).astype(np.int32)
    table = random_table(rng, lens, page, pages, extra=2)
    parent = rng.integers(0, n, n + 700).astype(np.int32)
    n_new = rng.integers(0, 20, n + 700).astype(np.int32)
    pc = to_device(cache)
    t2, l2 = i32(np.zeros((n + 700, width))), i32(np.zeros(n + 700))
    pc.fork(i32(table), i32(lens), i32(parent), i32(n_new), t2, l2)
    want_t, want_l, st = oc.fork(cache, table, lens, parent, n_new)
    assert np.array_equal(t2.cpu().numpy(), want_t) and np.array_equal(l2.cpu().numpy(), want_l) and st == 0
    same_cache(to_host(pc), cache)
    t3, used = torch.empty_like(t2), i32([0])
    pc.compact(t2, l2, t3, used)
    want, u = oc.compact(cache, want_t, want_l)
    assert np.array_equal(t3.cpu().numpy(), want) and used.item() == u
    same_cache(to_host(pc), cache)
    assert pc.device_status() == 0


def test_fork_faults():
    rng = np.random.default_rng(0)
    cache = random_cache(rng, 20, 1, 16, 64, "int8")
    lens = np.array([20, 33, 16], dtype=np.int32)
    table = random_table(rng, lens, 16, 20)
    t2, l2 = i32(np.zeros((3, table.shape[1]))), i32(np.zeros(3))

    def go(t, ln, parent, n_new, want):
        pc = to_device(cache)
        pc.fork(i32(t), i32(ln), i32(parent), i32(n_new), t2, l2)
        assert pc.device_status() == want
        return t2.cpu().numpy(), l2.cpu().numpy()
    t, ln = go(table, lens, [0, 3, -2], [1, 1, 1], xgr.XGR_DEV_INDEX)     # no such parents: empty rows
    assert ln.tolist() == [21, 0, 0] and (t[1:] == -1).all()
    bad = table.copy()
    bad[1, 0] = 20
    t, ln = go(bad, lens, [0, 1, 2], [0, 0, 0], xgr.XGR_DEV_INDEX)
    assert t[1, 0] == -1 and t[1, 1] == table[1, 1] and ln.tolist() == [20, 33, 16]
    t, ln = go(table, [20, 1000, 16], [0, 1, 2], [0, 0, 0], xgr.XGR_DEV_INDEX)
    assert ln.tolist() == [20, 0, 16]
    t, ln = go(table, lens, [0, 1, 2], [0, -4, 0], xgr.XGR_DEV_INDEX)
    assert ln.tolist() == [20, 33, 16]
    t, ln = go(table, lens, [0, 1, 2], [2 ** 31 - 1, 0, 0], xgr.XGR_DEV_CAPACITY)
    assert ln.tolist() == [table.shape[1] * 16, 33, 16]


@pytest.mark.parametrize("seed", range(6))
def test_compact_is_exact(seed):
    rng = np.random.default_rng(seed)
    page, d = [16, 128, 64][seed % 3], [64, 128][seed % 2]
    pages = [33, 64, 500, 1000, 40, 96][seed]
    cache = random_cache(rng, pages, 2, page, d, "int8" if seed % 2 else "e4m3")
    table, lens = shared_tables(rng, pages, page, 10, int(rng.integers(1, 30)))
    if seed == 4:
        lens[:] = 0
    pc = to_device(cache)
    out, used = i32(np.zeros_like(table)), i32([-1])
    pc.compact(i32(table), i32(lens), out, used)
    want, u = oc.compact(cache, table, lens)
    assert np.array_equal(out.cpu().numpy(), want) and used.item() == u and pc.device_status() == 0
    same_cache(to_host(pc), cache)


def test_refusals_of_the_wrapper():
    from shared_prefix_decode_xattention_b200.cache import PagedCache
    k = torch.zeros((4, 2, 16, 64), dtype=torch.int8, device="cuda")
    sc = torch.zeros((4, 2), device="cuda")
    for args in ((k.cpu(), k, sc, sc), (k, k[:3], sc, sc), (k.half(), k.half(), sc, sc), (k, k, sc[:3], sc),
                 (k.transpose(1, 2), k.transpose(1, 2), sc, sc), (k[..., :48].contiguous(),) * 2 + (sc, sc)):
        with pytest.raises(xgr.XgrError):
            PagedCache(*args)
    pc = PagedCache(k, k.clone(), sc, sc.clone())
    t, ln, cu = i32([[0, 1]]), i32([20]), i32([0, 1])
    q = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device="cuda")
    o, z = torch.empty_like(q), torch.empty((1, 4), device="cuda")
    for bad in (dict(q=q.float()), dict(q=q[:, :3]), dict(cu=i32([0, 1, 1])), dict(table=t.long()), dict(length=ln.cpu()),
                dict(out=o[:, :2]), dict(lse=z.double()), dict(mask="window"), dict(mask="prefix"), dict(prefix=ln),
                dict(first=i32([0, 0])), dict(slopes=z[0, :2]), dict(softcap=-1.0), dict(window=-2),
                dict(q=torch.zeros((1, 64, 4), dtype=torch.bfloat16, device="cuda").transpose(1, 2))):
        a = dict(table=t, length=ln, cu=cu, q=q, out=o, lse=z, max_q=1)
        a.update(bad)
        with pytest.raises(xgr.XgrError):
            pc.attend(**a)
    with pytest.raises(xgr.XgrError):
        pc.store(t, ln, cu, q, q, max_n=1)                      # four heads, the cache has two
    with pytest.raises(xgr.XgrError):
        pc.fork(t, ln, i32([0]), None, t, i32([0]))             # the table itself as the result
    with pytest.raises(xgr.XgrError):
        pc.compact(t, ln, t, i32([0]))
    assert pc.device_status() == 0


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("fmt,d,page", [("e4m3", 128, 16), ("int8", 64, 32)])
def test_beam_decode_over_the_cache(fmt, d, page):
    """Prompts stored once and shared by their beams; then steps of fork, store, attend and the masked beam
    top-K, whose parents are the next fork's; a compaction on the way; every step against the oracle."""
    rng = np.random.default_rng(7)
    B, BW, hkv, G, V, steps = 2, 6, 2, 2, 50, 4
    n_pages, width = 160, 12
    cache = random_cache(rng, n_pages, hkv, page, d, fmt)
    pc = to_device(cache)
    prompt = np.array([5 * page + 3, 2 * page])
    rows = B * BW
    # one row a request: its prompt
    table, lens, st = oc.fork(cache, np.full((B, width), -1, np.int32), np.zeros(B, np.int32), np.arange(B), prompt)
    t, ln = i32(np.zeros((B, width))), i32(np.zeros(B))
    pc.fork(i32(np.full((B, width), -1)), i32(np.zeros(B)), i32(np.arange(B)), i32(prompt), t, ln)
    cu = np.concatenate([[0], np.cumsum(prompt)])
    k, k64 = bf16(rng.standard_normal((cu[-1], hkv, d)))
    v, v64 = bf16(rng.standard_normal((cu[-1], hkv, d)))
    pc.store(t, ln, i32(cu), k, v, max_n=int(prompt.max()))
    oc.store(cache, table, lens, cu, k64, v64)
    same_cache(to_host(pc), cache)
    parent = np.repeat(np.arange(B), BW).astype(np.int32)
    cum = np.zeros((B, BW), np.float32)
    for s in range(steps):
        ones = np.ones(rows, np.int32)
        table, lens, st = oc.fork(cache, table, lens, parent, ones)
        t2, l2 = i32(np.zeros((rows, width))), i32(np.zeros(rows))
        pc.fork(t, ln, i32(parent), i32(ones), t2, l2)
        t, ln = t2, l2
        if s == 2:
            t3, used = torch.empty_like(t), i32([0])
            pc.compact(t, ln, t3, used)
            table, u = oc.compact(cache, table, lens)
            assert used.item() == u
            t = t3
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(ln.cpu().numpy(), lens) and st == 0
        cu = np.arange(rows + 1)
        k, k64 = bf16(rng.standard_normal((rows, hkv, d)) * (1 + s))
        v, v64 = bf16(rng.standard_normal((rows, hkv, d)) / (1 + s))
        q, q64 = bf16(rng.standard_normal((rows, hkv * G, d)))
        pc.store(t, ln, i32(cu), k, v, max_n=1)
        oc.store(cache, table, lens, cu, k64, v64)
        same_cache(to_host(pc), cache)
        out, lse = torch.empty_like(q), torch.empty((rows, hkv * G), device="cuda")
        pc.attend(t, ln, i32(cu), q, out, lse, max_q=1, softcap=30.0)
        ref, ref_lse = oc.attend(cache, table, lens, cu, q64, softcap=30.0)
        vmax = np.full((rows, hkv * G, 1), oc.QMAX[fmt] * np.nanmax(cache["vs"]))
        vmax = np.minimum(vmax, 16.0)
        close(out, lse, ref, ref_lse, vmax, d, 40.0)
        # the selection: a "model head" that takes the attention's output to scores
        scores = torch.log_softmax(out.float().reshape(B, BW, -1)[..., :V].contiguous(), -1)
        par, tok = (torch.empty((B, BW), dtype=torch.int32, device="cuda") for _ in range(2))
        cum_in = torch.tensor(cum, device="cuda")
        cum_out, n_out = torch.empty_like(cum_in), torch.empty(B, dtype=torch.int32, device="cuda")
        row_ptr = i32(np.arange(rows + 1) * V)
        cols = i32(np.tile(np.arange(V), rows))
        xgr.xgr_beam_topk_noalloc(B, BW, BW, V, scores, xgr.XGR_SCORES_LOGPROB, cum_in, i32([BW] * B), None,
                                  row_ptr, cols, par, tok, cum_out, n_out, torch.cuda.current_stream())
        cum = cum_out.cpu().numpy()
        p = par.cpu().numpy()
        assert (p >= 0).all()
        parent = (p + np.arange(B)[:, None] * BW).reshape(-1).astype(np.int32)
    # the beams of a finished request are given back: its pages are free
    dead = np.where(np.arange(rows) < BW, -1, np.arange(rows)).astype(np.int32)
    t2, l2 = i32(np.zeros((rows, width))), i32(np.zeros(rows))
    pc.fork(t, ln, i32(dead), None, t2, l2)
    t3, used = torch.empty_like(t), i32([0])
    pc.compact(t2, l2, t3, used)
    table, lens, st = oc.fork(cache, table, lens, dead)
    assert used.item() == oc.compact(cache, table, lens)[1]
    assert pc.device_status() == 0
