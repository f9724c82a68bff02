// cache.cuh -- what the kernels of the paged 8-bit KV cache share (internal).
#pragma once

#include <cuda_fp16.h>

#include <algorithm>

#include "../../include/xgr_cache.h"
#include "async.cuh"
#include "common.cuh"
#include "kernels.h"

namespace xgr {

constexpr int kMaxDevices = 64;
constexpr int kSms = 148;   // SMs of the one GPU this is built for; grids are multiples of it

// Rows and the pages behind them, as every kernel of the cache gets them.
struct CacheArgs {
    uint8_t *k, *v;              // [n_pages][Hkv][page][D]
    float *ks, *vs;              // [n_pages][Hkv]
    const int32_t *table;        // [n_rows][max_pages]
    const int32_t *len;          // [n_rows]
    const int32_t *cu;           // [n_rows + 1]
    int32_t *status;
    int n_pages, page, page_shift, Hkv, D, fmt;
    int n_rows, max_pages, n_tokens;
    int beams;                   // 1: a row may have more tokens than its length (beams over a prompt)
};

// A row's new tokens [t0, t0 + n) and its length; n = 0 and len = 0 where they do not fit together.
struct RowSpan {
    int t0, n, len;
};

__device__ __forceinline__ RowSpan row_span(const CacheArgs &a, int r, int max_n) {
    const int t0 = a.cu[r], t1 = a.cu[r + 1], len = a.len[r];
    RowSpan s{t0, t1 - t0, len};
    const bool bad = t0 < 0 || t1 < t0 || t1 > a.n_tokens || len < 0 ||
                     len > (int64_t)a.max_pages * a.page || (t1 - t0 > len && !a.beams);
    if (bad || s.n > max_n) {
        set_status(a.status, bad ? XGR_DEV_INDEX : XGR_DEV_CAPACITY);
        s.n = 0;
        s.len = 0;
    }
    return s;
}

// d_cu[i] and d_cu[i + 1], read here and now: their checks may stand behind other work.  (Rows are found by a search in
// d_cu, which misses some and finds others twice where it does not ascend.)
struct CuPair {
    int a, b;
};
__device__ __forceinline__ CuPair cu_pair(const CacheArgs &c, int i) {
    CuPair p;
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(p.a) : "l"(c.cu + i));
    asm volatile("ld.global.b32 %0, [%1];" : "=r"(p.b) : "l"(c.cu + i + 1));
    return p;
}
__device__ __forceinline__ bool out_of_order(const CacheArgs &c, const CuPair &p) {
    return p.a < 0 || p.a > p.b || p.b > c.n_tokens;
}

// Validation and the launches' arguments (cache_api.cu).
inline bool al(const void *p, size_t n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct AttendArgs {
    CacheArgs c;
    const __nv_bfloat16 *q;
    int64_t q_stride;
    __nv_bfloat16 *out;
    float *lse;
    int Hq, G;
    int max_q;
    float scale, softcap;
    int causal, window;
    const float *slopes;
    const int32_t *prefix;
    const int32_t *first;
    int whole;                  // 1: a work unit is a whole segment (every row is short)
    int lead;                   // units that stand for a segment's cost beside its keys
    int32_t *tile_lo;           // lowest visible key of each tile (with first)
    uint8_t *ws;
};

struct ForkArgs {
    CacheArgs c;                // rows: the parents'
    int n_out;
    const int32_t *parent, *n_new;
    int32_t *table_out, *len_out;
    uint32_t *used, *full;      // [words] pages some out row holds, and holds as a full page
    int32_t *sums;              // [16] the plan's CTAs' sums
    int32_t *lowest;            // [n_pages] lowest out row with the page as its partly filled last one
    int32_t *owner;             // [n_rows] the child that marks a parent's pages
    int32_t *row_need;          // [n_out] pages handed out before the row
    int32_t *row_copy;          // [n_out] 1: the row's first new page takes a copy
    int32_t *free_list;         // [n_pages] free pages, ascending
    int32_t *n_free;            // [1]
};

struct CompactArgs {
    CacheArgs c;
    int32_t *table_out, *n_used;
    uint32_t *used;             // [words] pages that rows hold
    int32_t *sums;              // [8] the plan's CTAs' sums
    int32_t *below;             // [1] held pages below U
    int32_t *prefix;            // [words] pages held before the word
    int32_t *hole;              // [n_pages] free slots below U, ascending
    int32_t *far;               // [n_pages] held pages from U on, ascending
};

struct StoreArgs {
    CacheArgs c;
    const __nv_bfloat16 *k, *v;
    int64_t stride;
    int max_n;
};

size_t attend_ws_bytes(int D, int G, int n_rows, int n_tokens);
cudaError_t launch_cache_attend(const AttendArgs &a, cudaStream_t s);
cudaError_t launch_cache_store(const StoreArgs &a, cudaStream_t s);
cudaError_t launch_cache_fork(const ForkArgs &a, cudaStream_t s);
cudaError_t launch_cache_compact(const CompactArgs &a, cudaStream_t s);

}  // namespace xgr
