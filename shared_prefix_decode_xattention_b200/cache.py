"""The paged 8-bit KV cache (include/xgr_cache.h) over torch tensors.

``PagedCache`` checks the tensors it is given, keeps the workspaces and the
status word, and calls the library; every computation runs in its kernels.
The order of a decode step: ``fork`` (the rows' new parents, pages for the
tokens to come), ``store``, ``attend``, a selection.

Streams: a call runs on ``stream``, or on torch's current stream of the cache's
device; the tensors it is given have to be ready there.  Each stream has a
workspace of its own, so calls on two streams may overlap.  It is made by the
first call that needs it, from that stream's memory, and never freed before the
PagedCache.  A captured graph keeps using the workspace of the stream it was
captured on; a call under capture that would have to make one raises.  So either
make the call once before the capture, on the capturing stream, or give the
captured calls a ``workspace`` of their own (a uint8 tensor of attend_bytes /
fork_bytes / compact_bytes; calls of one graph may share it), which is also the
way for graphs that may run at the same time.
"""
from __future__ import annotations

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
        self.device, self._index = k.device, k.get_device()
        self._i32, self._bf16, self._f32 = torch.int32, torch.bfloat16, torch.float32
        self.n_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self._c = xgr.xgr_cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                self.n_pages, self.page_size, self.n_kv_heads, self.head_dim,
                                fmt[k.dtype])
        xgr.xgr_cache_compact_bytes(self._c)      # refuses shapes the library does not take
        if torch.cuda.is_current_stream_capturing():
            _bad("PagedCache", "made under a capture: make it before", xgr.XGR_ERR_STATE)
        self._status = torch.zeros(1, dtype=torch.int32, device=self.device)
        torch.cuda.current_stream(self._index).synchronize()     # calls on any stream may set bits of it
        self._d_status = self._status.data_ptr()
        self._ws = {}                             # stream handle -> its workspace (tensor, bytes, address)
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
    def _int32(self, fn, name, t, shape):
        if t.dtype is not self._i32 or t.shape != shape or t.get_device() != self._index or not t.is_contiguous():
            _bad(fn, f"{name}: contiguous int32 {list(shape)} on {self.device}")
        return t.data_ptr()

    def _rows(self, fn, table, length):
        if table.dim() != 2:
            _bad(fn, "table: int32 [n_rows][max_pages]")
        n_rows, width = table.shape
        return xgr.xgr_cache_rows(n_rows, width, self._int32(fn, "table", table, table.shape),
                                  self._int32(fn, "length", length, (n_rows,)))

    def _tokens(self, fn, name, t, heads):
        """Packed tokens [n][heads][D] bf16, each token's heads contiguous; the token stride."""
        if t.dim() != 3 or t.dtype is not self._bf16 or t.get_device() != self._index:
            _bad(fn, f"{name}: bf16 [n_tokens][heads][{self.head_dim}] on {self.device}")
        n, h, d = t.shape
        if d != self.head_dim or (heads is not None and h != heads):
            _bad(fn, f"{name}: bf16 [n_tokens][{heads or 'heads'}][{self.head_dim}]")
        if t.is_contiguous():
            return h * d
        stride, across, along = t.stride()
        if n <= 1:
            stride = max(stride, h * d)
        if along != 1 or (h > 1 and across != d) or stride < h * d:
            _bad(fn, f"{name}: the heads of a token contiguous", xgr.XGR_ERR_SHAPE)
        return stride

    def _stream(self, stream):
        if stream is None:
            return self._torch.cuda.current_stream(self._index).cuda_stream
        return stream if isinstance(stream, int) else stream.cuda_stream

    def _bytes(self, key, size):
        need = self._need.get(key)
        if need is None:
            if len(self._need) >= 256:
                self._need.clear()
            need = self._need[key] = size()
        return need

    def _workspace(self, fn, stream, need, given):
        if given is not None:
            if given.dtype is not self._torch.uint8 or given.get_device() != self._index or not given.is_contiguous():
                _bad(fn, f"workspace: contiguous uint8 on {self.device}")
            return given, given.numel(), given.data_ptr()     # (the library checks size and alignment)
        ws = self._ws.get(stream)
        if ws is None or ws[1] < need:
            torch = self._torch
            own = (torch.cuda.ExternalStream(stream, device=self.device) if stream
                   else torch.cuda.default_stream(self._index))
            with torch.cuda.stream(own):      # memory of the stream that uses it, which orders its reuse
                if torch.cuda.is_current_stream_capturing():
                    _bad(fn, "no workspace of this size on the capturing stream yet: make the call once on it "
                             "before the capture, or pass workspace", xgr.XGR_ERR_STATE)
                if ws is not None:
                    self._old.append(ws[0])
                    need = max(need, 2 * ws[1])
                t = torch.empty(need, dtype=torch.uint8, device=self.device)
            ws = self._ws[stream] = (t, need, t.data_ptr())
        return ws

    def _run(self, call, *args):
        """The C call on the cache's device (a context's current device is the thread's)."""
        cuda = self._torch.cuda
        if cuda.current_device() == self._index:
            return call(*args)
        with cuda.device(self._index):
            return call(*args)

    # ------------------------------------------------------------------ calls
    def attend_bytes(self, n_q_heads: int, n_rows: int, n_tokens: int) -> int:
        """Bytes of the workspace of an attend call."""
        return self._bytes(("attend", n_q_heads, n_rows, n_tokens),
                           lambda: xgr.xgr_cache_attend_bytes(self._c, n_q_heads, n_rows, n_tokens))

    def fork_bytes(self, n_rows: int, n_out: int) -> int:
        """Bytes of the workspace of a fork of n_rows rows into n_out."""
        return self._bytes(("fork", n_rows, n_out), lambda: xgr.xgr_cache_fork_bytes(self._c, n_rows, n_out))

    def compact_bytes(self) -> int:
        """Bytes of the workspace of a compaction."""
        return self._bytes("compact", lambda: xgr.xgr_cache_compact_bytes(self._c))

    def attend(self, table, length, cu, q, out, lse, *, max_q: int, scale: float = 0.0, softcap: float = 0.0,
               mask: str = "causal", window: int = 0, slopes=None, prefix=None, first=None, stream=None,
               workspace=None):
        """Attention of packed query tokens q [T][Hq][D] (bf16) over the rows' pages into out
        [T][Hq][D] (bf16) and lse [T][Hq] (fp32); cu int32 [n_rows + 1].  mask: "full", "causal",
        or "prefix" (causal beside a bidirectional prefix of prefix[r] tokens).  The beams of a
        request over its prompt are one row under "full", however many (without slopes and window,
        which go by position).  See xgr_cache_attend."""
        self._run(self._attend, table, length, cu, q, out, lse, max_q, scale, softcap, mask, window, slopes,
                  prefix, first, stream, workspace)

    def _attend(self, table, length, cu, q, out, lse, max_q, scale, softcap, mask, window, slopes, prefix,
                first, stream, workspace):
        fn, index = "PagedCache.attend", self._index
        rows = self._rows(fn, table, length)
        n_rows = rows.n_rows
        if mask not in _MASKS or (mask == "prefix") != (prefix is not None):
            _bad(fn, "mask: 'full', 'causal', or 'prefix' with prefix int32 [n_rows]")
        stride = self._tokens(fn, "q", q, None)
        n_tokens, hq, _ = q.shape
        d_cu = self._int32(fn, "cu", cu, (n_rows + 1,))
        if out.dtype is not self._bf16 or out.shape != q.shape or not out.is_contiguous() \
                or out.get_device() != index:
            _bad(fn, "out: contiguous bf16 of q's shape")
        if lse.dtype is not self._f32 or lse.shape != (n_tokens, hq) or not lse.is_contiguous() \
                or lse.get_device() != index:
            _bad(fn, "lse: contiguous fp32 [n_tokens][Hq]")
        opts = xgr.xgr_attn_opts(scale, softcap, _MASKS[mask], window)
        if slopes is not None:
            if slopes.dtype is not self._f32 or slopes.shape != (hq,) or not slopes.is_contiguous() \
                    or slopes.get_device() != index:
                _bad(fn, "slopes: contiguous fp32 [Hq]")
            opts.d_slopes = slopes.data_ptr()
        if prefix is not None:
            opts.d_prefix = self._int32(fn, "prefix", prefix, (n_rows,))
        if first is not None:
            opts.d_first = self._int32(fn, "first", first, (n_tokens,))
        st = self._stream(stream)
        _, size, d_ws = self._workspace(fn, st, self.attend_bytes(hq, n_rows, n_tokens), workspace)
        xgr.xgr_cache_attend(self._c, rows, d_cu, n_tokens, max_q, hq, q.data_ptr(), stride, opts,
                             out.data_ptr(), lse.data_ptr(), d_ws, size, self._d_status, st)

    def store(self, table, length, cu, k, v, *, max_n: int, stream=None):
        """Quantises the rows' new tokens k, v [T][Hkv][D] (bf16) into their pages; length counts
        them already.  See xgr_cache_store."""
        self._run(self._store, table, length, cu, k, v, max_n, stream)

    def _store(self, table, length, cu, k, v, max_n, stream):
        fn = "PagedCache.store"
        rows = self._rows(fn, table, length)
        stride = self._tokens(fn, "k", k, self.n_kv_heads)
        if v.shape != k.shape or self._tokens(fn, "v", v, self.n_kv_heads) != stride:
            _bad(fn, "k, v: the same shape and token stride", xgr.XGR_ERR_SHAPE)
        d_cu = self._int32(fn, "cu", cu, (rows.n_rows + 1,))
        xgr.xgr_cache_store(self._c, rows, d_cu, k.shape[0], max_n, k.data_ptr(), v.data_ptr(), stride,
                            self._d_status, self._stream(stream))

    def fork(self, table, length, parent, n_new, table_out, len_out, *, stream=None, workspace=None):
        """The rows of the next step from their parents (-1: none), with pages for n_new[r] more
        tokens (None: none).  Pages of rows without children are free in this very call: a row to
        come back to is kept as its own parent, before its other children.  See xgr_cache_fork."""
        self._run(self._fork, table, length, parent, n_new, table_out, len_out, stream, workspace)

    def _fork(self, table, length, parent, n_new, table_out, len_out, stream, workspace):
        fn = "PagedCache.fork"
        rows = self._rows(fn, table, length)
        if parent.dim() != 1:
            _bad(fn, "parent: int32 [n_out]")
        n_out = parent.shape[0]
        d_parent = self._int32(fn, "parent", parent, (n_out,))
        d_new = None if n_new is None else self._int32(fn, "n_new", n_new, (n_out,))
        d_table = self._int32(fn, "table_out", table_out, (n_out, rows.max_pages))
        d_len = self._int32(fn, "len_out", len_out, (n_out,))
        st = self._stream(stream)
        _, size, d_ws = self._workspace(fn, st, self.fork_bytes(rows.n_rows, n_out), workspace)
        xgr.xgr_cache_fork(self._c, rows, n_out, d_parent, d_new, d_table, d_len, d_ws, size, self._d_status, st)

    def compact(self, table, length, table_out, n_used, *, stream=None, workspace=None):
        """Moves the pages that the rows hold to the front; n_used int32 [1].  See
        xgr_cache_compact."""
        self._run(self._compact, table, length, table_out, n_used, stream, workspace)

    def _compact(self, table, length, table_out, n_used, stream, workspace):
        fn = "PagedCache.compact"
        rows = self._rows(fn, table, length)
        d_table = self._int32(fn, "table_out", table_out, table.shape)
        d_used = self._int32(fn, "n_used", n_used, (1,))
        st = self._stream(stream)
        _, size, d_ws = self._workspace(fn, st, self.compact_bytes(), workspace)
        xgr.xgr_cache_compact(self._c, rows, d_table, d_used, d_ws, size, self._d_status, st)

    def device_status(self) -> int:
        """Waits for the cache's device, returns the status word's bits (XGR_DEV_*) and clears them.  (Bits of calls
        that another thread makes meanwhile stay, unless they are the same.)"""
        self._torch.cuda.synchronize(self.device)
        code = int(self._status.item())
        if code:
            self._status.bitwise_and_(~code)
            self._torch.cuda.current_stream(self._index).synchronize()
        return code
