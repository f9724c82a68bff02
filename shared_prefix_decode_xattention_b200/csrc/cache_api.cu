// cache_api.cu -- the C ABI of the paged 8-bit KV cache (declared in
// include/xgr_cache.h): argument validation, workspace layout, launches.
#include <cmath>

#include "cache.cuh"

using namespace xgr;

namespace {

constexpr size_t kAlign = 256;
constexpr int kMaxPages = 1 << 30;
constexpr int kMaxRows = 1 << 22;

size_t up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

// XGR_OK, or why this cache cannot be used; its page's shift in *shift
xgr_status check_cache(const xgr_cache *c, int *shift) {
    if (!c) return XGR_ERR_ARG;
    if (c->format != XGR_CACHE_E4M3 && c->format != XGR_CACHE_INT8) return XGR_ERR_ARG;
    if (c->n_pages < 1 || c->n_pages > kMaxPages || c->n_kv_heads < 1 || c->n_kv_heads > 1024) return XGR_ERR_SHAPE;
    // (blocks of 16 keys of a head are counted in 32 bits)
    if ((int64_t)c->n_pages * c->n_kv_heads * (c->page_size / 16) > 0x7fffffffll) return XGR_ERR_SHAPE;
    if (c->head_dim != 64 && c->head_dim != 128) return XGR_ERR_UNIMPLEMENTED;
    switch (c->page_size) {
        case 16: *shift = 4; break;
        case 32: *shift = 5; break;
        case 64: *shift = 6; break;
        case 128: *shift = 7; break;
        default: return XGR_ERR_UNIMPLEMENTED;
    }
    return XGR_OK;
}

xgr_status check_call(const xgr_cache *c, const xgr_cache_rows *rows, int32_t *d_status, CacheArgs *a) {
    int shift = 0;
    const xgr_status st = check_cache(c, &shift);
    if (st != XGR_OK) return st;
    if (!al(c->d_k, 16) || !al(c->d_v, 16) || !al(c->d_k_scale, 4) || !al(c->d_v_scale, 4) || !al(d_status, 4))
        return XGR_ERR_ARG;
    if (!rows) return XGR_ERR_ARG;
    if (rows->n_rows < 0 || rows->n_rows > kMaxRows || rows->max_pages < 1) return XGR_ERR_SHAPE;
    if ((int64_t)rows->max_pages * c->page_size > 0x7fffffffll - 4096) return XGR_ERR_SHAPE;
    if (rows->n_rows > 0 && (!al(rows->d_table, 4) || !al(rows->d_len, 4))) return XGR_ERR_ARG;
    *a = CacheArgs{};
    a->k = static_cast<uint8_t *>(c->d_k);
    a->v = static_cast<uint8_t *>(c->d_v);
    a->ks = c->d_k_scale;
    a->vs = c->d_v_scale;
    a->table = rows->d_table;
    a->len = rows->d_len;
    a->status = d_status;
    a->n_pages = c->n_pages;
    a->page = c->page_size;
    a->page_shift = shift;
    a->Hkv = c->n_kv_heads;
    a->D = c->head_dim;
    a->fmt = c->format;
    a->n_rows = rows->n_rows;
    a->max_pages = rows->max_pages;
    return XGR_OK;
}

bool overlaps(const void *p, size_t n, const void *q, size_t m) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + m && b < a + n;
}

size_t words_of(const xgr_cache *c) { return ((size_t)c->n_pages + 31) / 32; }

}  // namespace

extern "C" xgr_status xgr_cache_attend_bytes(const xgr_cache *cache, int32_t n_q_heads, int32_t n_rows,
                                             int32_t n_tokens, size_t *bytes) {
    int shift = 0;
    const xgr_status st = check_cache(cache, &shift);
    if (st != XGR_OK) return st;
    if (!bytes) return XGR_ERR_ARG;
    if (n_q_heads < 1 || n_q_heads % cache->n_kv_heads || n_rows < 0 || n_tokens < 0) return XGR_ERR_SHAPE;
    *bytes = attend_ws_bytes(cache->head_dim, n_q_heads / cache->n_kv_heads, n_rows, n_tokens);
    return XGR_OK;
}

extern "C" xgr_status xgr_cache_attend(const xgr_cache *cache, const xgr_cache_rows *rows, const int32_t *d_cu,
                                       int32_t n_tokens, int32_t max_q, int32_t n_q_heads, const void *d_q,
                                       int64_t q_stride, const xgr_attn_opts *opts, void *d_out, float *d_lse,
                                       void *d_ws, size_t ws_bytes, int32_t *d_status, xgr_stream_t stream) {
    AttendArgs a{};
    xgr_status st = check_call(cache, rows, d_status, &a.c);
    if (st != XGR_OK) return st;
    if (!opts) return XGR_ERR_ARG;
    if (opts->mask != XGR_ATTN_FULL && opts->mask != XGR_ATTN_CAUSAL) return XGR_ERR_ARG;
    if (opts->d_prefix && opts->mask != XGR_ATTN_CAUSAL) return XGR_ERR_ARG;
    if (!std::isfinite(opts->scale) || opts->scale < 0.f || !std::isfinite(opts->softcap) || opts->softcap < 0.f)
        return XGR_ERR_ARG;
    if ((opts->d_slopes && !al(opts->d_slopes, 4)) || (opts->d_prefix && !al(opts->d_prefix, 4)) ||
        (opts->d_first && !al(opts->d_first, 4)))
        return XGR_ERR_ARG;
    if (n_tokens < 0 || max_q < 0 || opts->window < 0 || n_q_heads < 1 || n_q_heads % cache->n_kv_heads)
        return XGR_ERR_SHAPE;
    if (rows->n_rows == 0 || n_tokens == 0 || max_q == 0) return XGR_OK;
    const int G = n_q_heads / cache->n_kv_heads;
    if (q_stride < (int64_t)n_q_heads * cache->head_dim || q_stride % 8) return XGR_ERR_SHAPE;
    if ((int64_t)n_tokens * n_q_heads > 0x7fffffffll || (int64_t)max_q * G > 0x3fffffffll) return XGR_ERR_SHAPE;
    if (!al(d_cu, 4) || !al(d_q, 16) || !al(d_out, 16) || !al(d_lse, 4) || !al(d_ws, kAlign)) return XGR_ERR_ARG;
    // (the query of a token is read by whoever takes a part of its keys)
    const size_t q_bytes = ((size_t)(n_tokens - 1) * q_stride + (size_t)n_q_heads * cache->head_dim) * 2;
    if (overlaps(d_out, (size_t)n_tokens * n_q_heads * cache->head_dim * 2, d_q, q_bytes)) return XGR_ERR_ARG;
    if (ws_bytes < attend_ws_bytes(cache->head_dim, G, rows->n_rows, n_tokens)) return XGR_ERR_CAPACITY;
    a.c.cu = d_cu;
    a.c.n_tokens = n_tokens;
    a.q = static_cast<const __nv_bfloat16 *>(d_q);
    a.q_stride = q_stride;
    a.out = static_cast<__nv_bfloat16 *>(d_out);
    a.lse = d_lse;
    a.Hq = n_q_heads;
    a.G = G;
    a.max_q = max_q;
    a.scale = opts->scale > 0.f ? opts->scale : 1.f / std::sqrt((float)cache->head_dim);
    a.softcap = opts->softcap;
    a.causal = opts->mask == XGR_ATTN_CAUSAL;
    a.c.beams = !a.causal;
    a.window = opts->window;
    a.slopes = opts->d_slopes;
    a.prefix = opts->d_prefix;
    a.first = opts->d_first;
    a.ws = static_cast<uint8_t *>(d_ws);
    return launch_cache_attend(a, (cudaStream_t)stream) == cudaSuccess ? XGR_OK : XGR_ERR_CUDA;
}

extern "C" xgr_status xgr_cache_store(const xgr_cache *cache, const xgr_cache_rows *rows, const int32_t *d_cu,
                                      int32_t n_tokens, int32_t max_n, const void *d_k, const void *d_v,
                                      int64_t token_stride, int32_t *d_status, xgr_stream_t stream) {
    StoreArgs a{};
    xgr_status st = check_call(cache, rows, d_status, &a.c);
    if (st != XGR_OK) return st;
    if (n_tokens < 0 || max_n < 0) return XGR_ERR_SHAPE;
    if (rows->n_rows == 0 || n_tokens == 0 || max_n == 0) return XGR_OK;
    if (token_stride < (int64_t)cache->n_kv_heads * cache->head_dim || token_stride % 8) return XGR_ERR_SHAPE;
    // (the grid: a slot for each page that a row can touch, for each kv head)
    const int64_t slots = n_tokens / cache->page_size + 2ll * rows->n_rows;
    if (slots * cache->n_kv_heads > 0x7fffffffll) return XGR_ERR_SHAPE;
    if (!al(d_cu, 4) || !al(d_k, 16) || !al(d_v, 16)) return XGR_ERR_ARG;
    a.c.cu = d_cu;
    a.c.n_tokens = n_tokens;
    a.k = static_cast<const __nv_bfloat16 *>(d_k);
    a.v = static_cast<const __nv_bfloat16 *>(d_v);
    a.stride = token_stride;
    a.max_n = max_n;
    return launch_cache_store(a, (cudaStream_t)stream) == cudaSuccess ? XGR_OK : XGR_ERR_CUDA;
}

namespace {

struct ForkWs {
    size_t used, full, lowest, owner, need, copy, list, sums, total;
};
ForkWs fork_ws(const xgr_cache *c, int32_t n_rows, int32_t n_out) {
    ForkWs w{};
    w.used = 0;
    w.full = up(words_of(c) * 4);
    w.lowest = w.full + up(words_of(c) * 4);
    w.owner = w.lowest + up((size_t)c->n_pages * 4);
    w.need = w.owner + up((size_t)n_rows * 4);
    w.copy = w.need + up((size_t)n_out * 4);
    w.list = w.copy + up((size_t)n_out * 4);
    w.sums = w.list + up((size_t)c->n_pages * 4);       // 16 sums, the number of free pages
    w.total = w.sums + kAlign;
    return w;
}

struct CompactWs {
    size_t used, prefix, hole, far, sums, total;
};
CompactWs compact_ws(const xgr_cache *c) {
    CompactWs w{};
    w.used = 0;
    w.prefix = up(words_of(c) * 4);
    w.hole = w.prefix + up(words_of(c) * 4);
    w.far = w.hole + up((size_t)c->n_pages * 4);
    w.sums = w.far + up((size_t)c->n_pages * 4);        // 8 sums, the held pages below U
    w.total = w.sums + kAlign;
    return w;
}

}  // namespace

extern "C" xgr_status xgr_cache_fork_bytes(const xgr_cache *cache, int32_t n_rows, int32_t n_out,
                                           size_t *bytes) {
    int shift = 0;
    const xgr_status st = check_cache(cache, &shift);
    if (st != XGR_OK) return st;
    if (!bytes) return XGR_ERR_ARG;
    if (n_rows < 0 || n_out < 0) return XGR_ERR_SHAPE;
    *bytes = fork_ws(cache, n_rows, n_out).total;
    return XGR_OK;
}

extern "C" xgr_status xgr_cache_fork(const xgr_cache *cache, const xgr_cache_rows *rows, int32_t n_out,
                                     const int32_t *d_parent, const int32_t *d_n_new, int32_t *d_table_out,
                                     int32_t *d_len_out, void *d_ws, size_t ws_bytes, int32_t *d_status,
                                     xgr_stream_t stream) {
    ForkArgs a{};
    const xgr_status st = check_call(cache, rows, d_status, &a.c);
    if (st != XGR_OK) return st;
    if (n_out < 0 || n_out > kMaxRows) return XGR_ERR_SHAPE;
    if (n_out == 0) return XGR_OK;
    if ((int64_t)n_out * 64 > 0x7fffffffll || (int64_t)n_out * rows->max_pages > 0x7fffffffll) return XGR_ERR_SHAPE;
    if (!al(d_parent, 4) || (d_n_new && !al(d_n_new, 4)) || !al(d_table_out, 4) || !al(d_len_out, 4) ||
        !al(d_ws, kAlign))
        return XGR_ERR_ARG;
    const size_t line = (size_t)rows->max_pages * 4;
    const void *out[2] = {d_table_out, d_len_out};
    const size_t out_n[2] = {n_out * line, (size_t)n_out * 4};
    const void *in[4] = {rows->d_table, rows->d_len, d_parent, d_n_new};
    const size_t in_n[4] = {rows->n_rows * line, (size_t)rows->n_rows * 4, (size_t)n_out * 4,
                            d_n_new ? (size_t)n_out * 4 : 0};
    for (int o = 0; o < 2; ++o)
        for (int i = 0; i < 4; ++i)
            if (in_n[i] && overlaps(out[o], out_n[o], in[i], in_n[i])) return XGR_ERR_ARG;
    const ForkWs w = fork_ws(cache, rows->n_rows, n_out);
    if (ws_bytes < w.total) return XGR_ERR_CAPACITY;
    uint8_t *ws = static_cast<uint8_t *>(d_ws);
    a.n_out = n_out;
    a.parent = d_parent;
    a.n_new = d_n_new;
    a.table_out = d_table_out;
    a.len_out = d_len_out;
    a.used = reinterpret_cast<uint32_t *>(ws + w.used);
    a.full = reinterpret_cast<uint32_t *>(ws + w.full);
    a.lowest = reinterpret_cast<int32_t *>(ws + w.lowest);
    a.owner = reinterpret_cast<int32_t *>(ws + w.owner);
    a.row_need = reinterpret_cast<int32_t *>(ws + w.need);
    a.row_copy = reinterpret_cast<int32_t *>(ws + w.copy);
    a.free_list = reinterpret_cast<int32_t *>(ws + w.list);
    a.sums = reinterpret_cast<int32_t *>(ws + w.sums);
    a.n_free = a.sums + 32;
    return launch_cache_fork(a, (cudaStream_t)stream) == cudaSuccess ? XGR_OK : XGR_ERR_CUDA;
}

extern "C" xgr_status xgr_cache_compact_bytes(const xgr_cache *cache, size_t *bytes) {
    int shift = 0;
    const xgr_status st = check_cache(cache, &shift);
    if (st != XGR_OK) return st;
    if (!bytes) return XGR_ERR_ARG;
    *bytes = compact_ws(cache).total;
    return XGR_OK;
}

extern "C" xgr_status xgr_cache_compact(const xgr_cache *cache, const xgr_cache_rows *rows, int32_t *d_table_out,
                                        int32_t *d_n_used, void *d_ws, size_t ws_bytes, int32_t *d_status,
                                        xgr_stream_t stream) {
    CompactArgs a{};
    const xgr_status st = check_call(cache, rows, d_status, &a.c);
    if (st != XGR_OK) return st;
    if (!al(d_n_used, 4) || !al(d_ws, kAlign)) return XGR_ERR_ARG;
    const size_t table = (size_t)rows->n_rows * rows->max_pages * 4;
    if (rows->n_rows > 0 && (!al(d_table_out, 4) || overlaps(d_table_out, table, rows->d_table, table) ||
                             overlaps(d_table_out, table, rows->d_len, (size_t)rows->n_rows * 4)))
        return XGR_ERR_ARG;
    const CompactWs w = compact_ws(cache);
    if (ws_bytes < w.total) return XGR_ERR_CAPACITY;
    uint8_t *ws = static_cast<uint8_t *>(d_ws);
    a.table_out = d_table_out;
    a.n_used = d_n_used;
    a.used = reinterpret_cast<uint32_t *>(ws + w.used);
    a.prefix = reinterpret_cast<int32_t *>(ws + w.prefix);
    a.hole = reinterpret_cast<int32_t *>(ws + w.hole);
    a.far = reinterpret_cast<int32_t *>(ws + w.far);
    a.sums = reinterpret_cast<int32_t *>(ws + w.sums);
    a.below = a.sums + 32;
    return launch_cache_compact(a, (cudaStream_t)stream) == cudaSuccess ? XGR_OK : XGR_ERR_CUDA;
}
