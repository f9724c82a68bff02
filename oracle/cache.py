"""The paged 8-bit KV cache by its definitions, in numpy and 64 bits: the
attention, the quantising store, the fork and the compaction of pages.  Plain
loops over rows, heads and pages; shares no code with the CUDA library.

A cache is a dict: k, v uint8 [n_pages][Hkv][page][D] (the codes' bits), ks, vs
float32 [n_pages][Hkv], fmt "e4m3" or "int8".  Tables are int32
[n_rows][max_pages], lengths int32 [n_rows], cu int32 [n_rows + 1].
"""
import numpy as np


def _e4m3_values():
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v[(b & 127) == 127] = np.nan
    return np.where(b >= 128, -v, v)


E4M3 = _e4m3_values()
QMAX = {"e4m3": 448.0, "int8": 127.0}


def decode(codes, fmt):
    """The codes' values (float64)."""
    codes = np.asarray(codes, dtype=np.uint8)
    return E4M3[codes] if fmt == "e4m3" else codes.view(np.int8).astype(np.float64)


def encode(x, fmt):
    """The code nearest to each finite x (ties to the even code), saturating."""
    x = np.asarray(x, dtype=np.float64)
    if fmt == "int8":
        return np.clip(np.rint(x), -127, 127).astype(np.int8).view(np.uint8)
    pos = E4M3[:127]                              # codes 0..126 ascend: 0 .. 448
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(pos, a), 1, 126)
    lo = hi - 1
    up = (pos[hi] - a) < (a - pos[lo])
    tie = (pos[hi] - a) == (a - pos[lo])
    code = np.where(up | (tie & (hi % 2 == 0)), hi, lo).astype(np.uint8)
    return np.where(np.signbit(x), code | 128, code).astype(np.uint8)


def row_kv(cache, table_row, length, g):
    """float64 k, v [length][D] of kv head g of one row."""
    page = cache["k"].shape[2]
    ids = np.asarray(table_row[: -(-length // page)], dtype=np.int64)
    out = []
    for c, s in (("k", "ks"), ("v", "vs")):
        x = decode(cache[c][ids, g], cache["fmt"]) * cache[s][ids, g].astype(np.float64)[:, None, None]
        out.append(x.reshape(-1, cache["k"].shape[3])[:length])
    return out


def visible(length, n, i, mask, window=0, prefix=None, first=None):
    """[lo, hi): the keys that query i of n (position length - n + i) sees."""
    pos = length - n + i
    hi = length if mask == "full" else pos + 1
    if prefix is not None:
        hi = max(hi, min(prefix, length))
    lo = 0 if first is None else max(0, first)
    if window:
        lo = max(lo, pos - window + 1)
    return lo, hi, pos


def attend(cache, table, length, cu, q, mask="causal", scale=0.0, softcap=0.0, window=0, slopes=None,
           prefix=None, first=None):
    """float64 out [T][Hq][D], lse [T][Hq] for q float64 [T][Hq][D]; rows of no query keep 0 / -inf."""
    T, hq, d = q.shape
    hkv = cache["k"].shape[1]
    out, lse = np.zeros((T, hq, d)), np.full((T, hq), -np.inf)
    sc = scale if scale else d ** -0.5
    for r in range(len(length)):
        t0, n = int(cu[r]), int(cu[r + 1] - cu[r])
        if n == 0:
            continue
        L = int(length[r])
        kv = [row_kv(cache, table[r], L, g) for g in range(hkv)]
        for i in range(n):
            lo, hi, pos = visible(L, n, i, mask, window, None if prefix is None else int(prefix[r]),
                                  None if first is None else int(first[t0 + i]))
            if lo >= hi:
                continue
            for h in range(hq):
                k, v = kv[h // (hq // hkv)]
                x = k[lo:hi] @ q[t0 + i, h] * sc
                if softcap:
                    x = softcap * np.tanh(x / softcap)
                if slopes is not None:
                    x = x - float(slopes[h]) * np.abs(pos - np.arange(lo, hi))
                m = x.max()
                w = np.exp(x - m)
                out[t0 + i, h] = w @ v[lo:hi] / w.sum()
                lse[t0 + i, h] = m + np.log(w.sum())
    return out, lse


def pow2_scale(absmax, fmt):
    """The smallest power of two s >= 2^-126 with absmax <= s * qmax."""
    e = -126
    while absmax > 2.0 ** e * QMAX[fmt]:
        e += 1
    return 2.0 ** e


def store(cache, table, length, cu, k, v):
    """Writes the rows' new tokens (k, v float64 [T][Hkv][D]) into the cache, in place."""
    page, hkv = cache["k"].shape[2], cache["k"].shape[1]
    fmt = cache["fmt"]
    for r in range(len(length)):
        n, L = int(cu[r + 1] - cu[r]), int(length[r])
        start = L - n
        for p in range(start // page, -(-L // page)) if n else ():
            a, b = max(start - p * page, 0), min(L - p * page, page)
            src = int(cu[r]) + p * page - start
            pid = int(table[r, p])
            for codes, scales, x in ((cache["k"], cache["ks"], k), (cache["v"], cache["vs"], v)):
                for g in range(hkv):
                    new = x[src + a: src + b, g]
                    was = float(scales[pid, g]) if a else 0.0
                    if not np.isfinite(new).all() or np.isnan(was):
                        s = np.nan
                        codes[pid, g, a:b] = 0
                        if a and not np.isnan(was):
                            codes[pid, g, :a] = 0
                    else:
                        s = max(pow2_scale(np.abs(new).max(), fmt), was)
                        if a and s != was:
                            codes[pid, g, :a] = encode(decode(codes[pid, g, :a], fmt) * was / s, fmt)
                        codes[pid, g, a:b] = encode(new / s, fmt)
                    scales[pid, g] = s


def fork(cache, table, length, parent, n_new=None):
    """(table_out, len_out, status bit 8 when pages ran out or a row was cut); copies pages in the cache."""
    n_pages, page, width = cache["k"].shape[0], cache["k"].shape[2], table.shape[1]
    n_out = len(parent)
    lens = [int(length[p]) if p >= 0 else 0 for p in parent]
    held, full_of, last_of = set(), set(), {}
    for r, p in enumerate(parent):
        for i in range(-(-lens[r] // page)):
            pid = int(table[p, i])
            held.add(pid)
            if i < lens[r] // page:
                full_of.add(pid)
            else:
                last_of.setdefault(pid, r)          # rows ascend: the lowest
    free = [p for p in range(n_pages) if p not in held]
    out = np.full((n_out, width), -1, dtype=np.int32)
    len_out = np.zeros(n_out, dtype=np.int32)
    status, at = 0, 0
    copies = []
    for r, p in enumerate(parent):
        L = lens[r]
        full, have = L // page, -(-L // page)
        copy = have > full and (int(table[p, full]) in full_of or last_of[int(table[p, full])] != r)
        want_len = L + (int(n_new[r]) if n_new is not None and p >= 0 else 0)
        if want_len > width * page:
            want_len, status = width * page, 8
        want = -(-want_len // page)
        begin = full if copy else have
        if begin:
            out[r, :begin] = table[p, :begin]
        need = want - begin
        got = max(0, min(need, len(free) - at))
        out[r, begin: begin + got] = free[at: at + got]
        if copy and got:
            copies.append((int(table[p, full]), free[at]))
        at += need
        if got < need:
            want_len, status = (begin + got) * page, 8
        len_out[r] = want_len
    for src, dst in copies:
        for x in ("k", "v", "ks", "vs"):
            cache[x][dst] = cache[x][src]
    return out, len_out, status


def compact(cache, table, length):
    """(table_out, pages in use); moves pages in the cache."""
    page, n_pages = cache["k"].shape[2], cache["k"].shape[0]
    used = sorted({int(table[r, i]) for r in range(len(length)) for i in range(-(-int(length[r]) // page))})
    U = len(used)
    far = [p for p in used if p >= U]
    hole = [p for p in range(U) if p not in set(used)]
    to = dict(zip(far, hole))
    out = np.full_like(table, -1)
    for r in range(len(length)):
        for i in range(-(-int(length[r]) // page)):
            out[r, i] = to.get(int(table[r, i]), int(table[r, i]))
    for src, dst in to.items():
        for x in ("k", "v", "ks", "vs"):
            cache[x][dst] = cache[x][src]
    return out, U
