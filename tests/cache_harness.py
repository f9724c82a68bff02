"""Shared by the tests of the paged 8-bit cache: small caches on the host (as
the oracle takes them) and their copies on the device."""
import numpy as np
import torch

import oracle.cache as oc

DT = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def random_codes(rng, shape, fmt):
    if fmt == "int8":
        return rng.integers(-127, 128, shape, dtype=np.int8).view(np.uint8)
    return oc.encode(np.clip(rng.standard_normal(shape) * 110, -448, 448), "e4m3")


def random_cache(rng, n_pages, hkv, page, d, fmt, spread=1.0):
    """Codes and scales of normal values; `spread`: the scales' range, as a factor 2^+-spread."""
    shape = (n_pages, hkv, page, d)
    c = {"fmt": fmt, "k": random_codes(rng, shape, fmt), "v": random_codes(rng, shape, fmt)}
    for s in ("ks", "vs"):
        c[s] = ((1 / (110.0 if fmt == "e4m3" else 73.0)) *
                2.0 ** rng.uniform(-spread, spread, shape[:2])).astype(np.float32)
    return c


def random_table(rng, lens, page, n_pages, extra=2, junk=-1):
    """Distinct pages for every row; `junk` behind them."""
    need = [-(-int(x) // page) for x in lens]
    order = rng.permutation(n_pages)
    t = np.full((len(lens), max(need + [1]) + extra), junk, dtype=np.int32)
    at = 0
    for r, n in enumerate(need):
        t[r, :n] = order[at: at + n]
        at += n
    assert at <= n_pages
    return t


def to_device(cache):
    from shared_prefix_decode_xattention_b200.cache import PagedCache
    t = [torch.from_numpy(cache[x].copy()).cuda().view(DT[cache["fmt"]]) for x in ("k", "v")]
    t += [torch.from_numpy(cache[x].copy()).cuda() for x in ("ks", "vs")]
    return PagedCache(*t)


def to_host(pc):
    fmt = "int8" if pc.k.dtype == torch.int8 else "e4m3"
    c = {"fmt": fmt}
    for x, t in (("k", pc.k), ("v", pc.v)):
        c[x] = t.view(torch.uint8).cpu().numpy()
    c["ks"], c["vs"] = pc.k_scale.cpu().numpy(), pc.v_scale.cpu().numpy()
    return c


def same_cache(a, b):
    for x in ("k", "v", "ks", "vs"):
        u, w = a[x], b[x]
        if x in ("ks", "vs"):
            u, w = u.view(np.uint32).copy(), w.view(np.uint32).copy()
            u[np.isnan(a[x])] = w[np.isnan(b[x])] = 0x7fc00000
        assert np.array_equal(u, w), (x, np.argwhere(u != w)[:5])


def i32(x):
    return torch.tensor(np.ascontiguousarray(x), dtype=torch.int32, device="cuda")


def bf16(x):
    """Rounded to bf16: the device tensor and its exact values."""
    t = torch.tensor(np.ascontiguousarray(x), dtype=torch.float32).to(torch.bfloat16)
    return t.cuda(), t.double().numpy()


def close(out, lse, ref, ref_lse, vmax, D, qk):
    """out bf16, lse fp32 against 64 bits.

    out: its own rounding is at most 2^-8 |o| (half a bf16 step, relative).  Each
    weight is rounded to fp16, 2^-11 relative at most, which moves the mean of
    the values by at most 2^-11 max |v|; the exponentials, sums and scores add
    less than half of that again.
    lse: a score is a sum of D exact products in fp32, each of the D additions
    off by at most 2^-24 of the running sum, which stays below qk = scale max_j sum_d |q_d k_jd|;
    eight more roundings of the score and the result (scale, cap, bias, logarithm)."""
    o, z = out.double().cpu().numpy(), lse.double().cpu().numpy()
    seen = np.isfinite(ref_lse)
    assert np.array_equal(np.isneginf(z), np.isneginf(ref_lse))
    assert np.array_equal(o[~seen], np.zeros_like(o[~seen]))
    err = np.abs(o - ref)
    tol = 2.0 ** -8 * np.abs(ref) + 1.5 * 2.0 ** -11 * vmax
    assert (err <= tol).all(), (err - tol).max()
    if seen.any():
        tol = 2.0 ** -24 * ((D + 8) * qk + 16 * np.abs(ref_lse[seen]).max() + 32)
        off = np.abs(z[seen] - ref_lse[seen]).max()
        assert off <= tol, (off, tol)
