/*
 * xgr_cache.h -- C ABI of the paged 8-bit KV cache of libxgr.so: attention
 * over a cache held in 8 bits with a scale for each page and kv head, the
 * store that quantises tokens into it, and the life of its pages (fork, free,
 * copy, compact).  Context-free calls beside the staged decode of xgr.h: a
 * prompt held here takes half the bytes of the bf16 prompt store, its pages
 * can be shared, copied and given back one by one, and scores may be capped,
 * biased and masked.
 *
 * The cache (caller-owned device memory; n_pages pages of page_size tokens):
 *   codes   d_k, d_v            [n_pages][n_kv_heads][page_size][head_dim], 8 bits each
 *   scales  d_k_scale, d_v_scale  fp32 [n_pages][n_kv_heads]
 *   value = code * scale.  format XGR_CACHE_E4M3: codes are e4m3 (finite codes
 *   only: the two NaN codes are no valid contents).  XGR_CACHE_INT8: codes are
 *   two's complement.  xgr_cache_store writes powers of two as scales; the
 *   attention takes any finite non-negative scale (softmax weights below 2^-100
 *   of a query's largest may count as none, whatever their page's scale).
 *
 * Rows: row r (a sequence, a beam, or a request whose beams share a prompt)
 * owns line r of a page table, d_table int32 [n_rows][max_pages], and a length
 * d_len int32 [n_rows] in tokens.  Its token j lies in page
 * d_table[r][j / page_size] at slot j % page_size.  Entries from
 * ceil(len / page_size) on are not read (xgr_cache_fork and xgr_cache_compact
 * write -1 there).  Rows may share pages.
 *
 * Ragged tokens: a call on new tokens takes them packed, row r's tokens being
 * d_cu[r] .. d_cu[r + 1] - 1 (d_cu int32 [n_rows + 1], ascending from 0,
 * d_cu[n_rows] <= n_tokens; tokens behind d_cu[n_rows] belong to no row and
 * are neither read nor written).  They are the last of their row: token i of
 * n stands at position len - n + i, d_len counting them already.  A row may
 * have none.  (Beams over a prompt, XGR_ATTN_FULL, are none of its tokens, and
 * may outnumber them.)
 *
 * The order of a decode step: xgr_cache_fork (the rows' new parents, and pages
 * for the tokens to come), xgr_cache_store, xgr_cache_attend, a selection.
 *
 * Conventions are those of xgr.h: caller-owned buffers, device pointers 16-byte
 * aligned (the int32 arrays d_cu, d_len, d_table, d_parent, d_n_new, d_prefix,
 * d_first, d_n_used, d_status and the fp32 d_slopes, scales and d_lse: 4), host-side
 * errors returned at once with nothing enqueued, no synchronisation, no device
 * allocation.  Every call runs on the current device, which must be the
 * buffers'.  Faults found on the device (a page id outside [0, n_pages), a
 * length outside [0, max_pages * page_size], d_cu out of order or past
 * n_tokens, a row with more tokens than its length but under XGR_ATTN_FULL:
 * XGR_DEV_INDEX; no free page, a row longer than max_pages or with more tokens
 * than max_n / max_q: XGR_DEV_CAPACITY) set bits in the caller's status word (d_status, int32,
 * never cleared by these calls), and the faulty element is skipped: a key in a
 * page that is not there is not attended, a token without a page is not
 * stored, a row whose length is at fault has no tokens.  Where d_cu is out of
 * order or past n_tokens anywhere, no row of an xgr_cache_attend has tokens, and
 * rows of an xgr_cache_store may be left out, each whole (XGR_DEV_INDEX in any
 * case).
 * XGR_DEV_TIMEOUT, as in xgr.h: a bounded wait inside xgr_cache_attend gave up,
 * and its results are not to be used.
 * The workspace of a call (d_ws, 256-byte aligned, at least the bytes its
 * _bytes function gives) needs no initial contents and holds nothing between
 * calls, so calls on one stream may share it; calls that may overlap on the
 * GPU (two streams, two captured graphs) need one each.
 */
#ifndef XGR_CACHE_H_
#define XGR_CACHE_H_

#include "xgr.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
    XGR_CACHE_E4M3 = 0,
    XGR_CACHE_INT8 = 1
};

typedef struct {
    void *d_k;
    void *d_v;
    float *d_k_scale;
    float *d_v_scale;
    int32_t n_pages;
    int32_t page_size;      /* 16, 32, 64 or 128 tokens */
    int32_t n_kv_heads;
    int32_t head_dim;       /* 64 or 128 */
    int32_t format;         /* XGR_CACHE_E4M3 or XGR_CACHE_INT8 */
} xgr_cache;

typedef struct {
    int32_t n_rows;         /* up to 4194304 */
    int32_t max_pages;
    const int32_t *d_table; /* [n_rows][max_pages] */
    const int32_t *d_len;   /* [n_rows] */
} xgr_cache_rows;

/* Which keys a query at position pos of a row of length len may see. */
enum {
    XGR_ATTN_FULL = 0,      /* every key of the row */
    XGR_ATTN_CAUSAL = 1     /* keys up to pos; with d_prefix also the row's first d_prefix[r] keys */
};

typedef struct {
    float scale;              /* of q.k; 0: 1 / sqrt(head_dim) */
    float softcap;            /* c > 0: scores become c * tanh(score / c); 0: none */
    int32_t mask;             /* XGR_ATTN_FULL or XGR_ATTN_CAUSAL */
    int32_t window;           /* w > 0: only keys j > pos - w; 0: none */
    const float *d_slopes;    /* fp32 [n_q_heads] or NULL: - slope_h * |pos - j| after the cap */
    const int32_t *d_prefix;  /* [n_rows] or NULL: a bidirectional prefix (with the causal mask) */
    const int32_t *d_first;   /* [n_tokens] or NULL: first visible key of each query, e.g. the start
                                 of its document in a row of packed documents */
} xgr_attn_opts;

/* Attention of the rows' new tokens over the rows' pages:
 *   d_q    bf16, query head h of token t at d_q + t * q_stride + h * head_dim
 *          (q_stride in elements, a multiple of 8, >= n_q_heads * head_dim);
 *          head h reads kv head h / (n_q_heads / n_kv_heads)
 *   d_out  bf16 [n_tokens][n_q_heads][head_dim]; d_lse fp32 [n_tokens][n_q_heads]; neither
 *          overlaps an input
 * Query i of a row sees the keys lo <= j < hi: hi = len (full), pos + 1
 * (causal), max(pos + 1, min(prefix, len)) (causal with a prefix); lo = the
 * largest of 0, d_first and pos - window + 1.  A query that sees none gets 0
 * and LSE -inf.  x_j = cap(scale * q.k_j) - slope * |pos - j|;
 * out = sum_j softmax(x)_j v_j; LSE = ln sum_j exp(x_j).
 * max_q: no row has more tokens than this (a row that does is skipped, and
 * XGR_DEV_CAPACITY set; with 0 the call does nothing).  The beams of a request over its shared prompt are
 * one row with a token for each beam and XGR_ATTN_FULL, as many as there are;
 * slopes and window go by position under this mask too, where query i of n
 * stands at len - n + i (below 0 where n > len), not all beams at the end.
 * n_q_heads: a multiple of n_kv_heads.  Contents behind a row's length are
 * never used, whatever bits are there. */
xgr_status xgr_cache_attend_bytes(const xgr_cache *cache, int32_t n_q_heads, int32_t n_rows,
                                  int32_t n_tokens, size_t *bytes);
xgr_status xgr_cache_attend(const xgr_cache *cache, const xgr_cache_rows *rows, const int32_t *d_cu,
                            int32_t n_tokens, int32_t max_q, int32_t n_q_heads, const void *d_q,
                            int64_t q_stride, const xgr_attn_opts *opts, void *d_out, float *d_lse,
                            void *d_ws, size_t ws_bytes, int32_t *d_status, xgr_stream_t stream);

/* Quantises the rows' new tokens into their pages (which they own: no other
 * row may hold a page that a call writes):
 *   d_k, d_v  bf16, kv head g of token t at d + t * token_stride + g * head_dim
 *             (token_stride in elements, a multiple of 8, >= n_kv_heads * head_dim)
 * For each page and kv head written, K and V apart: the scale becomes the
 * smallest power of two s (2^-126 at least) with max |x| <= s * 448 (e4m3) or
 * s * 127 (int8) over the new tokens, or stays where tokens before the new
 * ones lie in the page and its scale is larger; the codes are x / s rounded to
 * nearest (ties to even).  Where such a page's scale grows, its older tokens
 * are rounded again from their old values.  Slots behind the new tokens keep
 * their bits.  A NaN or infinity among a page and head's new values makes its
 * scale NaN and its codes 0, and it stays so until the page is begun anew (a
 * store from its first slot): every query that sees a key of that page and
 * head gets NaN, whether in its K or its V; queries that see none are not
 * touched by it.
 * max_n: no row has more tokens than this (a row that does is skipped, and
 * XGR_DEV_CAPACITY set; with 0 the call does nothing). */
xgr_status xgr_cache_store(const xgr_cache *cache, const xgr_cache_rows *rows, const int32_t *d_cu,
                           int32_t n_tokens, int32_t max_n, const void *d_k, const void *d_v,
                           int64_t token_stride, int32_t *d_status, xgr_stream_t stream);

/* The rows of the next step, from their parents: out row r continues row
 * d_parent[r] of `rows` with room for d_n_new[r] more tokens (NULL: none);
 * parent -1 makes an empty row without pages.  With p the parent's length:
 *   d_len_out[r] = p + d_n_new[r]
 *   full pages (p / page_size of them) are shared with the parent;
 *   a partly filled last page stays with the lowest out row that has it, unless
 *     another out row has it as a full page; every other row gets a copy of it
 *     (codes and scales of all kv heads, K and V);
 *   pages for the new tokens follow; the rest of the line is -1.
 * A page is free when no out row holds one of its parent's pages there, so
 * pages are freed by having no children, and one call forks, grows and frees:
 * `rows` has to list every holder of pages of this cache (a row is kept by
 * being its own parent).  New pages are the free ones in ascending order, given
 * out row by row, the copy first.  Where pages run out, or a row would pass
 * max_pages, the row ends before the first page it did not get, d_len_out says
 * so, and XGR_DEV_CAPACITY is set.  A parent outside [-1, n_rows) is taken for
 * -1 (XGR_DEV_INDEX).
 * d_table_out int32 [n_out][max_pages] and d_len_out [n_out] must not overlap
 * the arrays read.  Pages of rows without children are free in this very call:
 * it may copy into them and hand them out, and a partly filled page that a row
 * kept is written by that row's next store.  So `rows` is not to be gone on from
 * afterwards.  A row to come back to is kept: its own parent, listed before its
 * other children (who then get the copies), and not stored into. */
xgr_status xgr_cache_fork_bytes(const xgr_cache *cache, int32_t n_rows, int32_t n_out,
                                size_t *bytes);
xgr_status xgr_cache_fork(const xgr_cache *cache, const xgr_cache_rows *rows, int32_t n_out,
                          const int32_t *d_parent, const int32_t *d_n_new, int32_t *d_table_out,
                          int32_t *d_len_out, void *d_ws, size_t ws_bytes, int32_t *d_status,
                          xgr_stream_t stream);

/* Moves the pages that `rows` holds to the front of the cache: with U pages
 * held, the held pages from U on, in ascending order, go to the free slots
 * below U, in ascending order; pages below U stay.  d_table_out
 * [n_rows][max_pages] is the table after the move (-1 behind a row's pages;
 * must not overlap d_table), *d_n_used = U.  Lengths stay as they are. */
xgr_status xgr_cache_compact_bytes(const xgr_cache *cache, size_t *bytes);
xgr_status xgr_cache_compact(const xgr_cache *cache, const xgr_cache_rows *rows,
                             int32_t *d_table_out, int32_t *d_n_used, void *d_ws, size_t ws_bytes,
                             int32_t *d_status, xgr_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* XGR_CACHE_H_ */
