"""The paged 8-bit KV cache (include/xgr_cache.h) over torch tensors.

``PagedCache`` checks the tensors it is given, keeps the workspaces and the
status word, and calls the library; every computation runs in its kernels.
The order of a decode step: ``fork`` (the rows' new parents, pages for the
tokens to come), ``store``, ``attend``, a selection.

Streams: a call runs on ``stream``, or on torch's current stream of the cache's
device.  Each stream has workspaces of its own, so calls on two streams may
overlap; a captured graph keeps using the workspaces of the stream it was
captured on, so two graphs that may run at the same time are captured on two
streams, or with a PagedCache each (over the same tensors).  A workspace is made
by the first call that needs it and never freed before the PagedCache; a call
under capture that would have to make one raises, so make the call once before
the capture, on the capturing stream.
"""
from __future__ import annotations

import ctypes
from typing import Optional

from . import xgr

_MASKS = {"full": xgr.XGR_ATTN_FULL, "causal": xgr.XGR_ATTN_CAUSAL, "prefix": xgr.XGR_ATTN_CAUSAL}


def _bad(fn: str, why: str, status: int = xgr.XGR_ERR_ARG):
    raise xgr.XgrError(f"{fn}({why})", status)


class PagedCache:
    """K and V codes [n_pages][Hkv][page][D] (torch.float8_e4m3fn or torch.int8)
    with fp32 scales [n_pages][Hkv], all contiguous on one CUDA device."""

    def __init__(self, k, v, k_scale, v_scale):
        import torch
        self._torch = torch
        fmt = {torch.float8_e4m3fn: xgr.XGR_CACHE_E4M3, torch.int8: xgr.XGR_CACHE_INT8}
        if k.dim() != 4 or k.dtype not in fmt or v.dtype != k.dtype or v.shape != k.shape:
            _bad("PagedCache", "k, v: two [n_pages][Hkv][page][D] tensors of float8_e4m3fn or int8")
        for t in (k_scale, v_scale):
            if t.dtype != torch.float32 or tuple(t.shape) != tuple(k.shape[:2]):
                _bad("PagedCache", "scales: fp32 [n_pages][Hkv]")
        for t in (k, v, k_scale, v_scale):
            if not t.is_cuda or t.device != k.device or not t.is_contiguous():
                _bad("PagedCache", "tensors: contiguous, on one CUDA device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device = k.device
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self._c = xgr.xgr_cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                self.n_pages, self.page_size, self.n_kv_heads, self.head_dim,
                                fmt[k.dtype])
        xgr.xgr_cache_compact_bytes(self._c)      # refuses shapes the library does not take
        self._status = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._ws = {}                             # stream handle -> its workspace
        self._old = []                            # outgrown workspaces: a captured graph may use them
        self._need = {}                           # (call, sizes) -> bytes

    @classmethod
    def create(cls, n_pages: int, n_kv_heads: int, page_size: int, head_dim: int, dtype=None,
               device: str = "cuda"):
        """A cache of its own (contents undefined until stored); dtype float8_e4m3fn by default."""
        import torch
        shape = (n_pages, n_kv_heads, page_size, head_dim)
        dt = torch.float8_e4m3fn if dtype is None else dtype
        codes = [torch.zeros(shape, dtype=torch.uint8, device=device).view(dt) for _ in range(2)]
        scales = [torch.zeros(shape[:2], dtype=torch.float32, device=device) for _ in range(2)]
        return cls(*codes, *scales)

    # ------------------------------------------------------------------ checks
    def _i32(self, fn, name, t, shape):
        if t.dtype != self._torch.int32 or t.device != self.device or tuple(t.shape) != shape \
                or not t.is_contiguous():
            _bad(fn, f"{name}: contiguous int32 {list(shape)} on {self.device}")

    def _rows(self, fn, table, length):
        if table.dim() != 2:
            _bad(fn, "table: int32 [n_rows][max_pages]")
        n_rows, width = table.shape
        self._i32(fn, "table", table, (n_rows, width))
        self._i32(fn, "length", length, (n_rows,))
        return xgr.xgr_cache_rows(n_rows, width, table.data_ptr(), length.data_ptr())

    def _tokens(self, fn, name, t, heads):
        """Packed tokens [n][heads][D] bf16, each token's heads contiguous; the token stride."""
        if t.dim() != 3 or t.dtype != self._torch.bfloat16 or t.device != self.device \
                or t.shape[2] != self.head_dim or (heads is not None and t.shape[1] != heads):
            _bad(fn, f"{name}: bf16 [n_tokens][{heads or 'heads'}][{self.head_dim}] on {self.device}")
        line = t.shape[1] * t.shape[2]
        stride = t.stride(0) if t.shape[0] > 1 else line
        if t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != t.shape[2]) or stride < line:
            _bad(fn, f"{name}: the heads of a token contiguous", xgr.XGR_ERR_SHAPE)
        return stride

    def _stream(self, stream):
        if stream is None:
            return self._torch.cuda.current_stream(self.device).cuda_stream
        return stream if isinstance(stream, int) else stream.cuda_stream

    def _workspace(self, fn, stream, need):
        ws = self._ws.get(stream)
        if ws is None or ws.numel() < need:
            torch = self._torch
            if torch.cuda.is_current_stream_capturing():
                _bad(fn, "no workspace of this size on the capturing stream yet: make the call once "
                         "before the capture", xgr.XGR_ERR_STATE)
            if ws is not None:
                self._old.append(ws)
                need = max(need, 2 * ws.numel())
            ws = torch.empty(need, dtype=torch.uint8, device=self.device)
            self._ws[stream] = ws
        return ws

    def _guard(self):
        return self._torch.cuda.device(self.device)

    # ------------------------------------------------------------------ calls
    def attend(self, table, length, cu, q, out, lse, *, max_q: int, scale: float = 0.0, softcap: float = 0.0,
               mask: str = "causal", window: int = 0, slopes=None, prefix=None, first=None, stream=None):
        """Attention of packed query tokens q [T][Hq][D] (bf16) over the rows' pages into out
        [T][Hq][D] (bf16) and lse [T][Hq] (fp32); cu int32 [n_rows + 1].  mask: "full", "causal",
        or "prefix" (causal beside a bidirectional prefix of prefix[r] tokens).  See
        xgr_cache_attend."""
        fn, torch = "PagedCache.attend", self._torch
        rows = self._rows(fn, table, length)
        n_rows = rows.n_rows
        if mask not in _MASKS or (mask == "prefix") != (prefix is not None):
            _bad(fn, "mask: 'full', 'causal', or 'prefix' with prefix int32 [n_rows]")
        stride = self._tokens(fn, "q", q, None)
        n_tokens, hq = q.shape[0], q.shape[1]
        self._i32(fn, "cu", cu, (n_rows + 1,))
        if out.dtype != torch.bfloat16 or out.shape != q.shape or not out.is_contiguous() \
                or out.device != self.device:
            _bad(fn, "out: contiguous bf16 of q's shape")
        if lse.dtype != torch.float32 or tuple(lse.shape) != (n_tokens, hq) or not lse.is_contiguous() \
                or lse.device != self.device:
            _bad(fn, "lse: contiguous fp32 [n_tokens][Hq]")
        if slopes is not None and (slopes.dtype != torch.float32 or tuple(slopes.shape) != (hq,)
                                   or not slopes.is_contiguous() or slopes.device != self.device):
            _bad(fn, "slopes: contiguous fp32 [Hq]")
        if prefix is not None:
            self._i32(fn, "prefix", prefix, (n_rows,))
        if first is not None:
            self._i32(fn, "first", first, (n_tokens,))
        opts = xgr.xgr_attn_opts(scale, softcap, _MASKS[mask], window,
                                 None if slopes is None else slopes.data_ptr(),
                                 None if prefix is None else prefix.data_ptr(),
                                 None if first is None else first.data_ptr())
        key = ("attend", hq, n_rows, n_tokens)
        need = self._need.get(key)
        if need is None:
            need = self._need[key] = xgr.xgr_cache_attend_bytes(self._c, hq, n_rows, n_tokens)
        with self._guard():
            st = self._stream(stream)
            ws = self._workspace(fn, st, need)
            xgr.xgr_cache_attend(self._c, rows, cu, n_tokens, max_q, hq, q, stride, opts, out, lse, ws,
                                 ws.numel(), self._status, st)

    def store(self, table, length, cu, k, v, *, max_n: int, stream=None):
        """Quantises the rows' new tokens k, v [T][Hkv][D] (bf16) into their pages; length counts
        them already.  See xgr_cache_store."""
        fn = "PagedCache.store"
        rows = self._rows(fn, table, length)
        stride = self._tokens(fn, "k", k, self.n_kv_heads)
        if v.shape != k.shape or self._tokens(fn, "v", v, self.n_kv_heads) != stride:
            _bad(fn, "k, v: the same shape and token stride", xgr.XGR_ERR_SHAPE)
        self._i32(fn, "cu", cu, (rows.n_rows + 1,))
        with self._guard():
            xgr.xgr_cache_store(self._c, rows, cu, k.shape[0], max_n, k, v, stride, self._status,
                                self._stream(stream))

    def fork(self, table, length, parent, n_new, table_out, len_out, *, stream=None):
        """The rows of the next step from their parents (-1: none), with pages for n_new[r] more
        tokens (None: none).  See xgr_cache_fork."""
        fn = "PagedCache.fork"
        rows = self._rows(fn, table, length)
        n_out = parent.shape[0] if parent.dim() == 1 else -1
        self._i32(fn, "parent", parent, (n_out,))
        if n_new is not None:
            self._i32(fn, "n_new", n_new, (n_out,))
        self._i32(fn, "table_out", table_out, (n_out, rows.max_pages))
        self._i32(fn, "len_out", len_out, (n_out,))
        key = ("fork", n_out)
        need = self._need.get(key)
        if need is None:
            need = self._need[key] = xgr.xgr_cache_fork_bytes(self._c, n_out)
        with self._guard():
            st = self._stream(stream)
            ws = self._workspace(fn, st, need)
            xgr.xgr_cache_fork(self._c, rows, n_out, parent, n_new, table_out, len_out, ws, ws.numel(),
                               self._status, st)

    def compact(self, table, length, table_out, n_used, *, stream=None):
        """Moves the pages that the rows hold to the front; n_used int32 [1].  See
        xgr_cache_compact."""
        fn = "PagedCache.compact"
        rows = self._rows(fn, table, length)
        self._i32(fn, "table_out", table_out, tuple(table.shape))
        self._i32(fn, "n_used", n_used, (1,))
        need = self._need.get("compact")
        if need is None:
            need = self._need["compact"] = xgr.xgr_cache_compact_bytes(self._c)
        with self._guard():
            st = self._stream(stream)
            ws = self._workspace(fn, st, need)
            xgr.xgr_cache_compact(self._c, rows, table_out, n_used, ws, ws.numel(), self._status, st)

    def device_status(self) -> int:
        """Waits for the cache's device, returns the status word's bits (XGR_DEV_*) and clears them."""
        self._torch.cuda.synchronize(self.device)
        code = int(self._status.item())
        if code:
            self._status.zero_()
        return code
