// cache_pages.cu -- the life of the paged cache's pages: xgr_cache_fork (rows
// from their parents, copies of partly filled pages, new pages, freed pages)
// and xgr_cache_compact (pages in use to the front).
//
// Nothing about pages is kept between calls: which pages are in use follows
// from the tables, as a bitset built by each call (one bit a page, set by
// atomicOr, so the order does not matter), and every choice (which row keeps a
// shared partial page, which free page goes where) is by lowest index.  So the
// result is a function of the tables alone, the calls can be captured and
// replayed, and a page cannot be freed twice.
//
// Both are bound by the copies of whole pages (each page's K and V are two
// contiguous blocks of Hkv * page * D bytes); small calls by their four
// dependent launches, which overlap by programmatic launch.
#include "cache.cuh"

namespace xgr {

namespace {

constexpr int kScanThreads = 1024;   // the scan: one word of the bitset a thread, 32768 pages a block
constexpr int kCopyThreads = 256;
constexpr int64_t kPartBytes = 32768;   // bytes of one block's share of a page copy

// Exclusive block scan of one int per thread (block of kScanThreads); *total gets the sum.
__device__ __forceinline__ int block_scan(int v, int *total) {
    __shared__ int part[33];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) part[warp] = x;
    __syncthreads();
    if (warp == 0) {
        const int p = part[lane];
        int z = p;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, z, o);
            if (lane >= o) z += y;
        }
        part[lane] = z - p;
        if (lane == 31) part[32] = z;
    }
    __syncthreads();
    *total = part[32];
    return part[warp] + x - v;
}

// words before `w` of a bitset: their set bits (every thread of the block gets the sum)
__device__ __forceinline__ int bits_before(const uint32_t *bits, int w) {
    int n = 0;
    for (int i = threadIdx.x; i < w; i += kScanThreads) n += __popc(bits[i]);
    int total;
    block_scan(n, &total);
    return total;
}

// An out row of a fork: its parent's line and what it keeps of it.
struct Child {
    const int32_t *line;   // the parent's table line
    int len, full, held;   // the parent's length, its full pages, its pages
};

__device__ __forceinline__ Child child_of(const ForkArgs &a, int r) {
    int p = a.parent[r];
    if (p < -1 || p >= a.c.n_rows) {
        set_status(a.c.status, XGR_DEV_INDEX);
        p = -1;
    }
    Child c{nullptr, 0, 0, 0};
    if (p < 0) return c;
    int len = a.c.len[p];
    if (len < 0 || len > (int64_t)a.c.max_pages * a.c.page) {
        set_status(a.c.status, XGR_DEV_INDEX);
        len = 0;
    }
    c.line = a.c.table + (int64_t)p * a.c.max_pages;
    c.len = len;
    c.full = len >> a.c.page_shift;
    c.held = (int)(((int64_t)len + a.c.page - 1) >> a.c.page_shift);
    return c;
}

__device__ __forceinline__ bool page_ok(const CacheArgs &c, int id) { return id >= 0 && id < c.n_pages; }

// ---------------------------------------------------------------- fork

__global__ void __launch_bounds__(256) fork_clear_kernel(ForkArgs a, int words) {
    griddep_wait();
    griddep_launch_dependents();
    const int stride = gridDim.x * 256;
    for (int i = blockIdx.x * 256 + threadIdx.x; i < words; i += stride) a.used[i] = 0;
    // `lowest` is read at the rows' partly filled pages only
    for (int r = blockIdx.x * 256 + threadIdx.x; r < a.n_out; r += stride) {
        const Child c = child_of(a, r);
        if (c.held > c.full) {
            const int id = c.line[c.full];
            if (page_ok(a.c, id)) a.lowest[id] = 0x7fffffff;
        }
    }
}

// A warp per out row marks the row's pages as used.  A prompt's pages are
// marked by every beam that shares it: a plain load first keeps all but the
// first few of the atomics away (a stale value only costs one more).
__global__ void __launch_bounds__(256) fork_mark_kernel(ForkArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x % 32;
    for (int r = blockIdx.x * 8 + threadIdx.x / 32; r < a.n_out; r += gridDim.x * 8) {
        const Child c = child_of(a, r);
        for (int i = lane; i < c.held; i += 32) {
            const int id = c.line[i];
            if (!page_ok(a.c, id)) {
                set_status(a.c.status, XGR_DEV_INDEX);
                continue;
            }
            const uint32_t bit = 1u << (id & 31);
            if (!(__ldcg(a.used + (id >> 5)) & bit)) atomicOr(a.used + (id >> 5), bit);
            const int mine = i < c.full ? -1 : r;   // -1: a full page of some row, nobody's to write
            if (__ldcg(a.lowest + id) > mine) atomicMin(a.lowest + id, mine);
        }
    }
}

// Block 0: pages each out row needs, as a prefix over the rows.  Blocks 1..:
// the free pages in ascending order (each block its 32768 pages; the free ones
// before them are counted from the bitset again, so no block waits).
__global__ void __launch_bounds__(kScanThreads) fork_scan_kernel(ForkArgs a, int words) {
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x == 0) {
        int base = 0;
        for (int r0 = 0; r0 < a.n_out; r0 += kScanThreads) {
            const int r = r0 + threadIdx.x;
            int need = 0, copy = 0;
            if (r < a.n_out) {
                const Child c = child_of(a, r);
                if (c.held > c.full) {
                    const int id = c.line[c.full];
                    copy = page_ok(a.c, id) && a.lowest[id] != r;
                }
                int more = a.n_new ? a.n_new[r] : 0;
                if (!c.line) more = 0;
                if (more < 0) {
                    set_status(a.c.status, XGR_DEV_INDEX);
                    more = 0;
                }
                const int64_t grown = std::min((int64_t)c.len + more, (int64_t)a.c.max_pages << a.c.page_shift);
                const int want = (int)((grown + a.c.page - 1) >> a.c.page_shift);
                need = want - c.held + copy;
                a.row_copy[r] = copy;
            }
            int total;
            const int before = block_scan(need, &total);
            if (r < a.n_out) a.row_need[r] = base + before;
            base += total;
        }
        return;
    }
    const int w0 = (blockIdx.x - 1) * kScanThreads;
    const int free_before = w0 * 32 - bits_before(a.used, w0);
    const int w = w0 + threadIdx.x;
    uint32_t bits = 0;
    if (w < words) {
        bits = ~a.used[w];
        if ((w + 1) * 32 > a.c.n_pages) bits &= (1u << (a.c.n_pages & 31)) - 1u;   // (n_pages not a multiple of 32)
    }
    int total;
    int at = free_before + block_scan(__popc(bits), &total);
    for (; bits; bits &= bits - 1) a.free_list[at++] = w * 32 + __ffs(bits) - 1;
    if (w0 + kScanThreads >= words && threadIdx.x == 0) *a.n_free = free_before + total;
}

// 16-byte copy of `bytes` (a multiple of 16) by the block, eight loads in flight a thread
__device__ __forceinline__ void block_copy(uint8_t *dst, const uint8_t *src, int64_t bytes) {
    const uint4 *s = reinterpret_cast<const uint4 *>(src);
    uint4 *d = reinterpret_cast<uint4 *>(dst);
    const int64_t n = bytes / 16;
    for (int64_t i = threadIdx.x; i < n; i += 8 * kCopyThreads) {
        uint4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (i + u * kCopyThreads < n) v[u] = __ldcs(s + i + u * kCopyThreads);
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (i + u * kCopyThreads < n) __stcs(d + i + u * kCopyThreads, v[u]);
    }
}

// Part `part` of `parts` of the copy of a page (K and V codes, and by part 0 the scales).
__device__ __forceinline__ void copy_page(const CacheArgs &c, int dst, int src, int part, int parts) {
    const int64_t block = (int64_t)c.Hkv * c.page * c.D;   // bytes of a page's K (a multiple of 1024)
    const int64_t share = ((2 * block / 16 + parts - 1) / parts) * 16;
    const int64_t b0 = part * share, b1 = min(b0 + share, 2 * block);
    if (b0 < block) {
        const int64_t e = min(b1, block);
        block_copy(c.k + dst * block + b0, c.k + src * block + b0, e - b0);
    }
    if (b1 > block) {
        const int64_t s = max(b0, block) - block;
        block_copy(c.v + dst * block + s, c.v + src * block + s, b1 - block - s);
    }
    if (part == 0)
        for (int g = threadIdx.x; g < 2 * c.Hkv; g += kCopyThreads) {
            float *p = g < c.Hkv ? c.ks : c.vs;
            const int h = g < c.Hkv ? g : g - c.Hkv;
            p[(int64_t)dst * c.Hkv + h] = p[(int64_t)src * c.Hkv + h];
        }
}

// A block per (out row, part): part 0 writes the row's line, all parts copy its partial page.
__global__ void __launch_bounds__(kCopyThreads) fork_apply_kernel(ForkArgs a, int parts) {
    griddep_wait();
    griddep_launch_dependents();
    const int r = blockIdx.x / parts, part = blockIdx.x % parts;
    const int copy = a.row_copy[r];
    if (part > 0 && !copy) return;
    const Child c = child_of(a, r);
    const int need0 = a.row_need[r];
    const int n_free = *a.n_free;
    if (copy && need0 < n_free) copy_page(a.c, a.free_list[need0], c.line[c.full], part, parts);
    if (part > 0) return;
    int more = a.n_new && c.line ? max(a.n_new[r], 0) : 0;
    const int64_t cap = (int64_t)a.c.max_pages << a.c.page_shift;
    int64_t grown = (int64_t)c.len + more;
    bool cut = grown > cap;
    grown = min(grown, cap);
    const int want = (int)((grown + a.c.page - 1) >> a.c.page_shift);
    const int begin = copy ? c.full : c.held;            // the first new page's column
    const int have = max(0, min(want - begin, n_free - need0));
    if (begin + have < want) {                            // pages ran out
        grown = (int64_t)(begin + have) << a.c.page_shift;
        cut = true;
    }
    int32_t *out = a.table_out + (int64_t)r * a.c.max_pages;
    for (int i = threadIdx.x; i < a.c.max_pages; i += kCopyThreads) {
        int id = -1;
        if (i < begin) {
            id = c.line[i];
            if (!page_ok(a.c, id)) id = -1;
        } else if (i < begin + have) {
            id = a.free_list[need0 + i - begin];
        }
        out[i] = id;
    }
    if (threadIdx.x == 0) {
        a.len_out[r] = (int)grown;
        if (cut) set_status(a.c.status, XGR_DEV_CAPACITY);
    }
}

// ---------------------------------------------------------------- compact

__global__ void __launch_bounds__(256) compact_clear_kernel(CompactArgs a, int words) {
    griddep_wait();
    griddep_launch_dependents();
    for (int i = blockIdx.x * 256 + threadIdx.x; i < words; i += gridDim.x * 256) a.used[i] = 0;
}

__device__ __forceinline__ int pages_of(const CacheArgs &c, int r) {
    const int len = c.len[r];
    if (len < 0 || len > (int64_t)c.max_pages * c.page) {
        set_status(c.status, XGR_DEV_INDEX);
        return 0;
    }
    return (int)(((int64_t)len + c.page - 1) >> c.page_shift);
}

__global__ void __launch_bounds__(256) compact_mark_kernel(CompactArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x % 32;
    for (int r = blockIdx.x * 8 + threadIdx.x / 32; r < a.c.n_rows; r += gridDim.x * 8) {
        const int held = pages_of(a.c, r);
        const int32_t *line = a.c.table + (int64_t)r * a.c.max_pages;
        for (int i = lane; i < held; i += 32) {
            const int id = line[i];
            if (!page_ok(a.c, id)) {
                set_status(a.c.status, XGR_DEV_INDEX);
                continue;
            }
            const uint32_t bit = 1u << (id & 31);
            if (!(__ldcg(a.used + (id >> 5)) & bit)) atomicOr(a.used + (id >> 5), bit);
        }
    }
}

// Each block its 32768 pages: held pages before each word, the free slots below
// U and the held pages from U on, both ascending.
__global__ void __launch_bounds__(kScanThreads) compact_scan_kernel(CompactArgs a, int words) {
    griddep_wait();
    griddep_launch_dependents();
    const int U = bits_before(a.used, words);
    const int w0 = blockIdx.x * kScanThreads;
    const int before = bits_before(a.used, w0);
    const int w = w0 + threadIdx.x;
    const uint32_t bits = w < words ? a.used[w] : 0u;
    int total;
    const int mine = before + block_scan(__popc(bits), &total);   // held pages before word w
    if (w < words) a.prefix[w] = mine;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.n_used = U;
    // held pages below U: the far pages' ranks start there
    const int uw = U >> 5;
    int below = bits_before(a.used, uw);
    if (uw < words) below += __popc(a.used[uw] & ((1u << (U & 31)) - 1u));
    if (w >= words) return;
    for (uint32_t b = bits; b; b &= b - 1) {
        const int j = __ffs(b) - 1, id = w * 32 + j;
        if (id >= U) a.far[mine + __popc(bits & ((1u << j) - 1u)) - below] = id;
    }
    for (uint32_t b = ~bits; b; b &= b - 1) {
        const int j = __ffs(b) - 1, id = w * 32 + j;
        if (id < U) a.hole[id - mine - __popc(bits & ((1u << j) - 1u))] = id;
    }
}

__global__ void __launch_bounds__(kCopyThreads) compact_apply_kernel(CompactArgs a, int parts) {
    griddep_wait();
    griddep_launch_dependents();
    const int U = *a.n_used;
    auto before = [&](int id) {   // held pages before page id
        return a.prefix[id >> 5] + __popc(a.used[id >> 5] & ((1u << (id & 31)) - 1u));
    };
    const int below = U < a.c.n_pages ? before(U) : U;
    const int64_t moves = (int64_t)(U - below) * parts;
    for (int64_t m = blockIdx.x; m < moves; m += gridDim.x) {
        const int k = (int)(m / parts);
        copy_page(a.c, a.hole[k], a.far[k], (int)(m % parts), parts);
    }
    for (int r = blockIdx.x; r < a.c.n_rows; r += gridDim.x) {
        const int held = pages_of(a.c, r);
        const int32_t *line = a.c.table + (int64_t)r * a.c.max_pages;
        int32_t *out = a.table_out + (int64_t)r * a.c.max_pages;
        for (int i = threadIdx.x; i < a.c.max_pages; i += kCopyThreads) {
            int id = i < held ? line[i] : -1;
            if (!page_ok(a.c, id)) id = -1;
            if (id >= U) id = a.hole[before(id) - below];
            out[i] = id;
        }
    }
}

int copy_parts(const CacheArgs &c) {
    const int64_t bytes = 2ll * c.Hkv * c.page * c.D;
    return (int)std::min<int64_t>(64, (bytes + kPartBytes - 1) / kPartBytes);
}

}  // namespace

cudaError_t launch_cache_fork(const ForkArgs &a, cudaStream_t s) {
    const int words = (a.c.n_pages + 31) / 32;
    const int warps = std::min((a.n_out + 7) / 8, kSms * 8);
    const int clear = std::min((std::max(words, a.n_out) + 255) / 256, kSms * 4);
    cudaError_t e = launch_pdl(fork_clear_kernel, dim3(clear), dim3(256), 0, s, a, words);
    if (e == cudaSuccess) e = launch_pdl(fork_mark_kernel, dim3(warps), dim3(256), 0, s, a);
    const int blocks = 1 + (words + kScanThreads - 1) / kScanThreads;
    if (e == cudaSuccess) e = launch_pdl(fork_scan_kernel, dim3(blocks), dim3(kScanThreads), 0, s, a, words);
    const int parts = copy_parts(a.c);
    if (e == cudaSuccess)
        e = launch_pdl(fork_apply_kernel, dim3(a.n_out * parts), dim3(kCopyThreads), 0, s, a, parts);
    return e;
}

cudaError_t launch_cache_compact(const CompactArgs &a, cudaStream_t s) {
    const int words = (a.c.n_pages + 31) / 32;
    cudaError_t e = launch_pdl(compact_clear_kernel, dim3(std::min((words + 255) / 256, kSms)), dim3(256), 0, s, a, words);
    if (e == cudaSuccess)
        e = launch_pdl(compact_mark_kernel, dim3(std::min((a.c.n_rows + 7) / 8, kSms * 8)), dim3(256), 0, s, a);
    const int blocks = (words + kScanThreads - 1) / kScanThreads;
    if (e == cudaSuccess)
        e = launch_pdl(compact_scan_kernel, dim3(blocks), dim3(kScanThreads), 0, s, a, words);
    if (e == cudaSuccess)
        e = launch_pdl(compact_apply_kernel, dim3(kSms * 8), dim3(kCopyThreads), 0, s, a, copy_parts(a.c));
    return e;
}

}  // namespace xgr
