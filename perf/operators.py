"""The paged 8-bit KV cache operators: what is timed, their plain forms, and their values in 64 bits.

A cache holds K and V as 8-bit codes (e4m3 or int8) in pages [n_pages][Hkv][page][D], with an fp32 scale for each page
and kv head.  A row (a sequence, or a request whose beams share its prompt) owns a line of a page table and a length.

  attend   attention of a row's query tokens over its pages; scores may be capped by a tanh, get a bias that falls with
           distance, and be masked (causal, a bidirectional prefix, a sliding window, the documents of a packed row)
  store    quantises new tokens into the last pages of their rows
  fork     the rows of the next step from their parents: shared pages, copies of partly filled ones, pages for new tokens
  compact  moves the pages in use to the front
"""
import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
QMAX = {"e4m3": 448.0, "int8": 127.0}
CODE = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


# ------------------------------------------------------------------ cases
def listed():
    base = dict(op="attend", q_lo=1, q_hi=1, mask="causal", window=0, doc=0, prefix=False, cap=0.0, alibi=False)
    return [
        # the smallest decode: 4 beams of one request over a 256-token history (latency)
        dict(base, name="attend-tiny-beams", rows=1, q_lo=4, q_hi=4, len_lo=256, len_hi=256, hq=8, hkv=2, d=64, page=16,
             fmt="e4m3", mask="full"),
        # one token for each of 64 requests with 8192-token prefixes and ragged suffixes (serving, memory bound), capped scores
        dict(base, name="attend-decode-64", rows=64, len_lo=8448, len_hi=10240, hq=32, hkv=8, d=128, page=64, fmt="e4m3",
             cap=30.0),
        # one token for each of three very long, very ragged histories, distance bias (work split along the cache)
        dict(base, name="attend-decode-long", rows=3, len_lo=9001, len_hi=180007, hq=32, hkv=4, d=128, page=128, fmt="int8",
             alibi=True),
        # 128 beams of 8 requests over 1024-token prompts (the candidate pool's step)
        dict(base, name="attend-beams-128", rows=8, q_lo=128, q_hi=128, len_lo=1024, len_hi=1024, hq=16, hkv=4, d=128, page=64,
             fmt="e4m3", mask="full"),
        # 512 beams of 16 requests over 4096-token prompts (the largest: compute bound)
        dict(base, name="attend-beams-512", rows=16, q_lo=512, q_hi=512, len_lo=4096, len_hi=4096, hq=32, hkv=8, d=128, page=64,
             fmt="e4m3", mask="full"),
        # chunks of packed histories beside short ones: causal, a bidirectional prefix, documents, capped scores
        dict(base, name="attend-chunks-packed", rows=7, q_lo=61, q_hi=1000, len_lo=1000, len_hi=6001, hq=32, hkv=8, d=128,
             page=32, fmt="int8", mask="prefix", prefix=True, doc=1733, cap=50.0),
        # one token of each of 8 x 128 beams appended after a fork
        dict(name="store-beam-tokens", op="store", rows=1024, n_lo=1, n_hi=1, len_lo=1025, len_hi=1040, hkv=4, d=128, page=16,
             fmt="int8"),
        # ragged prompts of 64 requests written after their prefill
        dict(name="store-prompts", op="store", rows=64, n_lo=2048, n_hi=16384, len_lo=2048, len_hi=16384, hkv=4, d=128, page=64,
             fmt="e4m3"),
        # the beams of 8 requests after a selection: about half of the parents survive
        dict(name="fork-beams-128", op="fork", groups=8, beams=128, live=61, prompt=1024, own_pages=2, hkv=4, d=128, page=16,
             fmt="e4m3", new=1),
        # the beams of 16 requests of the large pool, wide pages: the copies dominate
        dict(name="fork-beams-512", op="fork", groups=16, beams=512, live=200, prompt=4096, own_pages=1, hkv=8, d=128, page=32,
             fmt="int8", new=2),
        # a small cache moved together
        dict(name="compact-small", op="compact", rows=24, len_lo=100, len_hi=700, used=0.61, hkv=2, d=64, page=16, fmt="int8"),
        # the cache of 128 ragged requests, half of it free
        dict(name="compact-large", op="compact", rows=128, len_lo=500, len_hi=9000, used=0.5, hkv=4, d=128, page=64, fmt="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "store", "fork", "compact"])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    fmt = rng.choice(["e4m3", "int8"])
    hkv = rng.choice([1, 2, 4, 8])
    c = dict(op=op, d=d, page=page, fmt=fmt, hkv=hkv)
    if op == "attend":
        hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8])
        hi = _log(rng, 30, 120000)
        lo = _log(rng, 1, hi)
        rows = min(_log(rng, 1, 128), max(1, int(4.0e8 / (hi * hkv * d))))
        q_hi = rng.choice([1, 1, _log(rng, 2, 700)])
        pairs = rows * q_hi * hq * hi * d
        q_hi = max(1, min(q_hi, hi, int(q_hi * min(1.0, 6.0e10 / pairs))))
        mask = rng.choice(["full", "causal", "causal", "prefix"])
        return dict(c, rows=rows, q_lo=rng.randint(1, q_hi) if q_hi > 1 else rng.choice([0, 1, 1]), q_hi=q_hi, len_lo=lo, len_hi=hi,
                    hq=hq, mask=mask, prefix=mask == "prefix", window=rng.choice([0, 0, _log(rng, 1, hi)]),
                    doc=rng.choice([0, 0, 0, _log(rng, 7, 5000)]), cap=rng.choice([0.0, 0.0, 15.0, 30.0, 50.0]),
                    alibi=rng.random() < 0.3)
    if op == "store":
        n_hi = rng.choice([1, _log(rng, 2, 12000)])
        hi = n_hi + _log(rng, 1, 5000)
        rows = min(_log(rng, 1, 1024), max(1, int(4.0e8 / (hi * hkv * d))))
        return dict(c, rows=rows, n_lo=rng.randint(0, n_hi), n_hi=n_hi, len_lo=_log(rng, 1, hi), len_hi=hi)
    if op == "fork":
        beams = _log(rng, 1, 512)
        prompt = rng.randint(0, 4096 // page) * page
        own_pages = rng.randint(1, 3)
        groups = min(_log(rng, 1, 16), max(1, int(2.0e8 / (beams * own_pages * page * hkv * d))))
        return dict(c, groups=groups, beams=beams, live=rng.randint(1, beams), prompt=prompt, own_pages=own_pages,
                    new=rng.randint(0, 2 * page))
    hi = _log(rng, 20, 9000)
    rows = min(_log(rng, 1, 200), max(1, int(3.0e8 / (hi * hkv * d))))
    return dict(c, rows=rows, len_lo=_log(rng, 1, hi), len_hi=hi, used=round(rng.uniform(0.2, 0.95), 3))


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, ragged, the same ones for a case whatever the seed."""
    f = ((np.arange(n) + 1) * 0.6180339887498949) % 1.0
    v = np.floor(lo + f * (hi - lo + 1)).astype(np.int64)
    return np.clip(v, lo, hi)


def _pages(n, page):
    return -(-n // page)


def _attend_shape(c):
    """Per row: tokens, length, prefix; per token: position, its visible keys [lo, hi)."""
    n = _spread(c["rows"], c["q_lo"], c["q_hi"])
    length = np.maximum(_spread(c["rows"], c["len_lo"], c["len_hi"])[::-1], n)
    cu = np.concatenate([[0], np.cumsum(n)])
    row = np.repeat(np.arange(c["rows"]), n)
    pos = np.arange(cu[-1]) - cu[row] + length[row] - n[row]
    prefix = length // 3
    first = (pos // c["doc"]) * c["doc"] if c["doc"] else np.zeros_like(pos)
    lo, hi = first, length[row]
    if c["mask"] != "full":
        hi = pos + 1
    if c["mask"] == "prefix":
        hi = np.maximum(hi, prefix[row])
    if c["window"]:
        lo = np.maximum(lo, pos - c["window"] + 1)
    return dict(n=n, len=length, cu=cu, row=row, pos=pos, prefix=prefix, first=first, lo=lo, hi=hi)


def work(case):
    c, op = case, case["op"]
    line = c["hkv"] * c["d"]
    if op == "attend":
        s = _attend_shape(c)
        seen = np.maximum(s["hi"] - s["lo"], 0)
        lo = np.full(c["rows"], 1 << 60)
        hi = np.zeros(c["rows"], dtype=np.int64)
        np.minimum.at(lo, s["row"], s["lo"])
        np.maximum.at(hi, s["row"], s["hi"])
        keys = int(np.maximum(hi - lo, 0).sum())
        tokens = int(s["cu"][-1])
        return {"bytes": 2 * keys * line + 8 * keys // c["page"] * c["hkv"] + tokens * c["hq"] * (4 * c["d"] + 4),
                "flops": 4 * c["d"] * c["hq"] * int(seen.sum())}
    if op == "store":
        n = int(_spread(c["rows"], c["n_lo"], c["n_hi"]).sum())
        return {"bytes": max(1, 2 * n * line * 3), "flops": 0}
    if op == "fork":
        rows = c["groups"] * c["beams"]
        pages = c["prompt"] // c["page"] + c["own_pages"]
        copies = c["groups"] * (c["beams"] - c["live"])
        return {"bytes": 2 * rows * pages * 4 + copies * 4 * c["page"] * line, "flops": 0}
    s = _compact_shape(c)
    return {"bytes": 2 * int(s["need"].sum()) * 4 + int(s["moved"]) * 4 * c["page"] * line, "flops": 0}


def _compact_shape(c):
    length = _spread(c["rows"], c["len_lo"], c["len_hi"])
    need = _pages(length, c["page"])
    total = int(need.sum())
    n_pages = max(total + 1, int(round(total / c["used"])))
    return dict(len=length, need=need, total=total, n_pages=n_pages, moved=total * (n_pages - total) / n_pages)


# ------------------------------------------------------------------ inputs
def _i32(x):
    return torch.as_tensor(np.ascontiguousarray(x), dtype=torch.int32).to(DEV)


def _cache(g, n_pages, c):
    """Codes and scales of n_pages pages (and one spare page behind them, which no table names): normal values, as a
    quantiser with a scale for each page and head leaves them."""
    shape = (n_pages + 1, c["hkv"], c["page"], c["d"])

    def codes():
        x = torch.empty(shape, dtype=torch.float16, device=DEV).normal_(generator=g)
        if c["fmt"] == "e4m3":
            return (x * 110.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn)
        return (x * 32.0).round_().clamp_(-127.0, 127.0).to(torch.int8)

    def scales():
        x = torch.rand(shape[:2], generator=g, device=DEV) * 0.7 + 0.7
        return x / (110.0 if c["fmt"] == "e4m3" else 32.0)

    return dict(k=codes(), v=codes(), ks=scales(), vs=scales())


def _table(g, need, n_pages, width):
    """A table whose rows hold `need` pages each, drawn without repetition; -1 behind them."""
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    start = np.concatenate([[0], np.cumsum(need)[:-1]])
    idx = start[:, None] + np.arange(width)[None, :]
    held = np.arange(width)[None, :] < need[:, None]
    t = order[torch.as_tensor(np.where(held, idx, 0), device=DEV)]
    return torch.where(torch.as_tensor(held, device=DEV), t, torch.full_like(t, -1)).contiguous()


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    return {"attend": _prepare_attend, "store": _prepare_store, "fork": _prepare_fork,
            "compact": _prepare_compact}[c["op"]](c, g)


def _prepare_attend(c, g):
    s = _attend_shape(c)
    need = _pages(s["len"], c["page"])
    width = int(need.max()) + 3
    n_pages = int(need.sum()) + 5
    st = dict(case=c, n_pages=n_pages, **_cache(g, n_pages, c))
    st["table"] = _table(g, need, n_pages, width)
    st["len"], st["cu"] = _i32(s["len"]), _i32(s["cu"])
    tokens = int(s["cu"][-1])
    st["q"] = torch.empty((tokens, c["hq"], c["d"]), device=DEV).normal_(generator=g).to(torch.bfloat16)
    st["first"] = _i32(s["first"]) if c["doc"] else None
    st["prefix"] = _i32(s["prefix"]) if c["prefix"] else None
    st["slopes"] = (2.0 ** (-8.0 * torch.arange(1, c["hq"] + 1, device=DEV, dtype=torch.float32) / c["hq"])
                    if c["alibi"] else None)
    st["max_q"] = int(s["n"].max())
    st["max_len"] = int(s["len"].max())
    st["out"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty((tokens, c["hq"]), dtype=torch.float32, device=DEV)
    return st


def _prepare_store(c, g):
    n = _spread(c["rows"], c["n_lo"], c["n_hi"])
    length = np.maximum(_spread(c["rows"], c["len_lo"], c["len_hi"]), n)
    need = _pages(length, c["page"])
    n_pages = int(need.sum()) + 5
    st = dict(case=c, n_pages=n_pages, **_cache(g, n_pages, c))
    st["ks"] = torch.exp2(torch.floor(torch.log2(st["ks"])))   # as the operator itself leaves them: powers of two
    st["vs"] = torch.exp2(torch.floor(torch.log2(st["vs"])))
    st["table"] = _table(g, need, n_pages, int(need.max()) + 1)
    st["len"], st["cu"] = _i32(length), _i32(np.concatenate([[0], np.cumsum(n)]))
    tokens = int(n.sum())
    st["new_k"] = torch.empty((tokens, c["hkv"], c["d"]), device=DEV).normal_(generator=g).to(torch.bfloat16)
    st["new_v"] = (torch.empty((tokens, c["hkv"], c["d"]), device=DEV).normal_(generator=g) * 3.0).to(torch.bfloat16)
    st["max_n"] = int(n.max())
    return st


def _prepare_fork(c, g):
    rows, full = c["groups"] * c["beams"], c["prompt"] // c["page"]
    held = full + c["own_pages"]
    width = held + _pages(c["new"], c["page"]) + 1
    n_used = c["groups"] * full + rows * c["own_pages"]
    n_pages = n_used + rows * (2 + _pages(c["new"], c["page"])) // 2 + 3
    st = dict(case=c, n_pages=n_pages, **_cache(g, n_pages, c))
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    group = np.arange(rows) // c["beams"]
    idx = np.zeros((rows, width), dtype=np.int64)
    idx[:, :full] = group[:, None] * full + np.arange(full)[None, :]
    idx[:, full:held] = c["groups"] * full + np.arange(rows)[:, None] * c["own_pages"] + np.arange(c["own_pages"])[None, :]
    t = order[torch.as_tensor(idx, device=DEV)]
    t[:, held:] = -1
    st["table"] = t.contiguous()
    # the last of the own pages is partly filled, by the same number of tokens for every beam
    st["len"] = torch.full((rows,), held * c["page"] - 1 - c["page"] // 3, dtype=torch.int32, device=DEV)
    # `live` beams of each group have children; every one of those has one at least
    pick = torch.argsort(torch.rand((c["groups"], c["beams"]), generator=g, device=DEV), dim=1)[:, : c["live"]]
    more = torch.randint(0, c["live"], (c["groups"], c["beams"] - c["live"]), generator=g, device=DEV)
    par = torch.cat([pick, torch.gather(pick, 1, more)], dim=1)
    mix = torch.argsort(torch.rand(par.shape, generator=g, device=DEV), dim=1)
    par = torch.gather(par, 1, mix) + torch.arange(c["groups"], device=DEV)[:, None] * c["beams"]
    st["parent"] = par.reshape(-1).to(torch.int32).contiguous()
    st["n_new"] = torch.full((rows,), c["new"], dtype=torch.int32, device=DEV)
    st["table_out"] = torch.empty_like(st["table"])
    st["len_out"] = torch.empty_like(st["len"])
    return st


def _prepare_compact(c, g):
    s = _compact_shape(c)
    st = dict(case=c, n_pages=s["n_pages"], **_cache(g, s["n_pages"], c))
    st["table"] = _table(g, s["need"], s["n_pages"], int(s["need"].max()) + 2)
    st["len"] = _i32(s["len"])
    st["table_out"] = torch.empty_like(st["table"])
    st["n_used"] = torch.empty((1,), dtype=torch.int32, device=DEV)
    return st


# ------------------------------------------------------------------ the framework's calls
def _handle(s):
    """The cache's handle, made on the state's first pass and kept with it."""
    if "handle" not in s:
        from shared_prefix_decode_xattention_b200.cache import PagedCache
        n = s["n_pages"]
        s["handle"] = PagedCache(s["k"][:n], s["v"][:n], s["ks"][:n], s["vs"][:n])
    return s["handle"]


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        h = _handle(s)
        if op == "attend":
            c = s["case"]
            h.attend(s["table"], s["len"], s["cu"], s["q"], s["out"], s["lse"], max_q=s["max_q"], mask=c["mask"],
                     prefix=s["prefix"], first=s["first"], window=c["window"], softcap=c["cap"], slopes=s["slopes"])
            return s["out"], s["lse"]
        if op == "store":
            h.store(s["table"], s["len"], s["cu"], s["new_k"], s["new_v"], max_n=s["max_n"])
        elif op == "fork":
            h.fork(s["table"], s["len"], s["parent"], s["n_new"], s["table_out"], s["len_out"])
        else:
            h.compact(s["table"], s["len"], s["table_out"], s["n_used"])
    elif op == "attend":
        return _plain_attend(s)
    else:
        {"store": _plain_store, "fork": _plain_fork, "compact": _plain_compact}[op](s)
    n = s["n_pages"]
    cache = {"k": s["k"][:n], "v": s["v"][:n], "k_scale": s["ks"][:n], "v_scale": s["vs"][:n]}
    if op == "fork":
        return {**cache, "table": s["table_out"], "len": s["len_out"]}
    if op == "compact":
        return {**cache, "table": s["table_out"], "n_used": s["n_used"]}
    return cache


# ------------------------------------------------------------------ plain forms
def _gathered(codes, scales, table, n_keys):
    """fp32 [R][Hkv][n_keys][D]: the rows' pages, dequantised."""
    x = codes.view(torch.uint8)[table].view(codes.dtype).float() * scales[table][..., None, None]
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)[:, :, :n_keys]


def _plain_attend(s):
    c, n_keys, max_q = s["case"], s["max_len"], s["max_q"]
    hkv, d, group = c["hkv"], c["d"], c["hq"] // c["hkv"]
    table = s["table"].clamp(min=0).long()
    n, length = (s["cu"][1:] - s["cu"][:-1]).long(), s["len"].long()
    tokens = s["q"].shape[0]
    at = torch.arange(max_q, device=DEV)
    tok = (s["cu"][:-1, None].long() + at).clamp(max=max(tokens - 1, 0))
    q = s["q"][tok].float().reshape(c["rows"], max_q, hkv, group, d).permute(0, 2, 3, 1, 4)
    k = _gathered(s["k"], s["ks"], table, n_keys)
    v = _gathered(s["v"], s["vs"], table, n_keys)
    # a page behind a row's end may hold anything: its keys are left out before any product
    inside = (torch.arange(n_keys, device=DEV) < length[:, None])[:, None, :, None]
    k, v = torch.where(inside, k, 0.0), torch.where(inside, v, 0.0)
    x = torch.matmul(q.flatten(2, 3), k.transpose(2, 3)).view(c["rows"], hkv, group, max_q, n_keys) * (d ** -0.5)
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    pos = length[:, None] - n[:, None] + at
    key = torch.arange(n_keys, device=DEV)
    if s["slopes"] is not None:
        away = (pos[:, :, None] - key).abs().float()
        x = x - s["slopes"].view(1, hkv, group, 1, 1) * away[:, None, None]
    hi = length[:, None].expand_as(pos)
    if c["mask"] != "full":
        hi = pos + 1
    if s["prefix"] is not None:
        hi = torch.maximum(hi, torch.minimum(s["prefix"].long(), length)[:, None])
    lo = torch.zeros_like(pos)
    if s["first"] is not None:
        lo = s["first"].long()[tok]
    if c["window"]:
        lo = torch.maximum(lo, pos - c["window"] + 1)
    seen = (key >= lo[:, :, None]) & (key < hi[:, :, None])
    x = torch.where(seen[:, None, None], x, float("-inf"))
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.flatten(2, 3), v).view(c["rows"], hkv, group, max_q, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (m + torch.log(total))[..., 0]
    # back from [R][max_q] to the ragged tokens
    ids = torch.arange(tokens, device=DEV)
    row = torch.searchsorted(s["cu"][1:].long(), ids, right=True)
    back = ids - s["cu"][:-1].long()[row]
    o = o.permute(0, 3, 1, 2, 4)[row, back].reshape(tokens, c["hq"], d)
    lse = lse.permute(0, 3, 1, 2)[row, back].reshape(tokens, c["hq"])
    return o.to(torch.bfloat16), lse.contiguous()


def _pow2_scale(absmax, qmax):
    """The smallest power of two that brings absmax into the codes' range (2^-126 for zeros)."""
    frac, exp = torch.frexp(absmax / qmax)
    exp = torch.where(frac == 0.5, exp - 1, exp)
    exp = torch.where(absmax > 0, exp, torch.full_like(exp, -126)).clamp(min=-126)
    return torch.ldexp(torch.ones_like(absmax), exp)


def _plain_store(s):
    c = s["case"]
    page, d, hkv, rows, qmax = c["page"], c["d"], c["hkv"], c["rows"], QMAX[c["fmt"]]
    n, length = (s["cu"][1:] - s["cu"][:-1]).long(), s["len"].long()
    start = length - n
    p0 = start // page
    span = _pages(s["max_n"], page) + 1                       # pages that a row's new tokens can touch
    lane = torch.arange(span, device=DEV)
    touched = ((p0[:, None] + lane) * page < length[:, None]) & (n[:, None] > 0)
    idx = (p0[:, None] + lane).clamp(max=s["table"].shape[1] - 1)
    pages = torch.where(touched, torch.gather(s["table"].long(), 1, idx), s["n_pages"])   # else: the spare page
    pos = (p0[:, None] + lane)[..., None] * page + torch.arange(page, device=DEV)          # [R][span][page]
    new = (pos >= start[:, None, None]) & (pos < length[:, None, None])
    old = pos < start[:, None, None]
    tokens = s["new_k"].shape[0]
    tok = (s["cu"][:-1, None, None].long() + pos - start[:, None, None]).clamp(0, max(tokens - 1, 0))
    for codes, scales, x in ((s["k"], s["ks"], s["new_k"]), (s["v"], s["vs"], s["new_v"])):
        now = codes.view(torch.uint8)[pages].view(codes.dtype)
        was = now.float() * scales[pages][..., None, None]                                 # [R][span][Hkv][page][D]
        val = x[tok].float().permute(0, 1, 3, 2, 4)
        val = torch.where(new[:, :, None, :, None], val, 0.0)
        want = _pow2_scale(val.abs().amax((-1, -2)), qmax)
        keep = old.any(-1)[..., None]
        scale = torch.where(keep, torch.maximum(want, scales[pages]), want)
        val = torch.where(old[:, :, None, :, None], was, val) / scale[..., None, None]
        if c["fmt"] == "int8":
            val = torch.round(val)
        val = val.clamp(-qmax, qmax).to(codes.dtype)
        val = torch.where((new | old)[:, :, None, :, None], val.view(torch.uint8), now.view(torch.uint8))
        codes.view(torch.uint8)[pages] = val
        scales[pages] = scale


def _plain_fork(s):
    c = s["case"]
    page, n_pages, table = c["page"], s["n_pages"], s["table"].long()
    rows, width = table.shape
    parent = s["parent"].long()
    alive = parent >= 0
    length = torch.where(alive, s["len"].long()[parent.clamp(min=0)], 0)
    mine = table[parent.clamp(min=0)]
    col = torch.arange(width, device=DEV)
    full, held = length // page, (length + page - 1) // page
    is_full, partial = col < full[:, None], held > full
    spare = torch.full_like(mine, n_pages)
    holder = torch.zeros(n_pages + 1, dtype=torch.bool, device=DEV)
    holder[torch.where(is_full, mine, spare)] = True
    holder[n_pages] = False
    last = torch.gather(mine, 1, full.clamp(max=width - 1)[:, None])[:, 0]
    last = torch.where(partial, last, n_pages)
    ids = torch.arange(rows, device=DEV)
    lowest = torch.full((n_pages + 1,), rows, dtype=torch.long, device=DEV).scatter_reduce(0, last, ids, "amin")
    keep = partial & ~holder[last] & (lowest[last] == ids)
    copy = partial & ~keep
    holder[torch.where(keep, last, n_pages)] = True
    holder[n_pages] = True
    free_rank = torch.cumsum(~holder, 0) - 1
    free = torch.zeros(n_pages + 1, dtype=torch.long, device=DEV)
    free[torch.where(holder, n_pages, free_rank)] = torch.arange(n_pages + 1, device=DEV)
    grown = length + torch.where(alive, s["n_new"].long(), 0)
    want = (grown + page - 1) // page
    begin = torch.where(copy, full, held)
    stop = torch.maximum(want, held)
    need = (col >= begin[:, None]) & (col < stop[:, None])
    rank = (torch.cumsum(need.flatten(), 0) - 1).view(rows, width).clamp(min=0)
    out = torch.where(col < held[:, None], mine, -1)
    out = torch.where(need, free[rank], out)
    dst = torch.where(copy, torch.gather(out, 1, full.clamp(max=width - 1)[:, None])[:, 0], n_pages)
    src = torch.where(copy, last, n_pages)
    for x in (s["k"].view(torch.uint8), s["v"].view(torch.uint8), s["ks"], s["vs"]):
        x[dst] = x[src]
    s["table_out"].copy_(out)
    s["len_out"].copy_(grown)


def _plain_compact(s):
    c = s["case"]
    page, n_pages, table = c["page"], s["n_pages"], s["table"].long()
    col = torch.arange(table.shape[1], device=DEV)
    held = col < ((s["len"].long() + page - 1) // page)[:, None]
    used = torch.zeros(n_pages + 1, dtype=torch.bool, device=DEV)
    used[torch.where(held, table, n_pages)] = True
    used = used[:n_pages]
    total = used.sum()
    ids = torch.arange(n_pages, device=DEV)
    far, hole = used & (ids >= total), ~used & (ids < total)
    slot = torch.full((n_pages + 1,), n_pages, dtype=torch.long, device=DEV)
    slot[torch.where(hole, torch.cumsum(hole, 0) - 1, n_pages)] = ids
    dst = torch.where(far, slot[(torch.cumsum(far, 0) - 1).clamp(min=0)], n_pages)
    src = torch.where(far, ids, n_pages)
    for x in (s["k"].view(torch.uint8), s["v"].view(torch.uint8), s["ks"], s["vs"]):
        x[dst] = x[src]
    moved = torch.where(far, dst, ids)
    s["table_out"].copy_(torch.where(held, moved[table.clamp(min=0)], -1))
    s["n_used"].copy_(total.view(1))


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    """attend and store from their definitions, row by row; fork and compact only move what is there (no value to compute)."""
    c = case
    if c["op"] in ("fork", "compact"):
        return None
    s = prepare(c, seed)
    return _exact_attend(s) if c["op"] == "attend" else _exact_store(s)


def _exact_attend(s):
    c = s["case"]
    shape = _attend_shape(c)
    if float(np.maximum(shape["hi"] - shape["lo"], 0).sum()) * c["hq"] * c["d"] > 2.0e11:
        return None
    group, d = c["hq"] // c["hkv"], c["d"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["lse"].shape, dtype=torch.float64, device=DEV)
    for r in range(c["rows"]):
        a, b, length = int(shape["cu"][r]), int(shape["cu"][r + 1]), int(shape["len"][r])
        if a == b:
            continue
        ids = s["table"][r, : _pages(length, c["page"])].long()
        pos = torch.as_tensor(shape["pos"][a:b], device=DEV)[:, None]
        lo, hi = (torch.as_tensor(shape[w][a:b], device=DEV)[:, None] for w in ("lo", "hi"))
        key = torch.arange(length, device=DEV)[None]
        for g in range(c["hkv"]):
            kk, vv = ((s[x][ids, g].to(torch.float32).double() * s[y][ids, g].double()[:, None, None]).reshape(-1, d)[:length]
                      for x, y in (("k", "ks"), ("v", "vs")))
            for h in range(g * group, (g + 1) * group):
                x = s["q"][a:b, h].double() @ kk.T / d ** 0.5
                if c["cap"]:
                    x = c["cap"] * torch.tanh(x / c["cap"])
                if s["slopes"] is not None:
                    x -= s["slopes"][h].double() * (pos - key).abs()
                x.masked_fill_(~((key >= lo) & (key < hi)), -torch.inf)
                z = torch.logsumexp(x, 1, keepdim=True)
                w = torch.exp(x - torch.where(torch.isinf(z), torch.zeros_like(z), z))
                out[a:b, h] = w @ vv
                lse[a:b, h] = z[:, 0]
    return out, lse


def _exact_store(s):
    c = s["case"]
    page, qmax = c["page"], QMAX[c["fmt"]]
    n = _spread(c["rows"], c["n_lo"], c["n_hi"])
    if c["rows"] * int(_pages(n, page).max() + 1) > 40000:
        return None
    length = np.maximum(_spread(c["rows"], c["len_lo"], c["len_hi"]), n)
    cu = np.concatenate([[0], np.cumsum(n)])
    res = []
    for codes, scales, new in ((s["k"], s["ks"], s["new_k"]), (s["v"], s["vs"], s["new_v"])):
        val, sc = codes[: s["n_pages"]].float(), scales[: s["n_pages"]].clone()
        table = s["table"].cpu().numpy()
        for r in range(c["rows"]):
            begin = int(length[r] - n[r])
            for p in range(begin // page, _pages(int(length[r]), page) if n[r] else 0):
                a, b = max(begin, p * page), min(int(length[r]), (p + 1) * page)
                k = int(table[r, p])
                x = new[int(cu[r]) + a - begin: int(cu[r]) + b - begin].double().transpose(0, 1)     # [Hkv][.][D]
                most = x.abs().amax((1, 2)).clamp(min=1e-300)
                scale = torch.exp2(torch.ceil(torch.log2(most / qmax)).clamp(min=-126))
                scale = torch.where(most > scale * qmax, 2 * scale, scale)
                scale = torch.where((most <= scale * qmax / 2) & (scale > 2.0 ** -126), scale / 2, scale)
                if a > p * page:
                    scale = torch.maximum(scale, sc[k].double())
                    val[k, :, : a - p * page] = _code64(val[k, :, : a - p * page].double() * (sc[k].double() / scale)[:, None, None], c)
                val[k, :, a - p * page: b - p * page] = _code64(x / scale[:, None, None], c)
                sc[k] = scale.float()
        res += [val if c["fmt"] == "e4m3" else None, sc]
    return {"k": res[0], "v": res[2], "k_scale": res[1], "v_scale": res[3]}


def _code64(x, c):
    """x rounded to the nearest code's value (ties to even), in 64 bits."""
    if c["fmt"] == "int8":
        return torch.round(x).clamp(-127, 127).float()
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448).float()
