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
// Each call is two kernels.  The plan runs on one cluster of eight CTAs, whose
// hardware barrier separates its phases (clear, mark, count and place), so a
// small call costs two launches instead of four; every CTA marks pages in a
// bitset of its own in shared memory first (the beams of a request all hold
// its prompt's pages, and that many atomics on one word took 120 us for 8192
// rows of 129 pages).  The second kernel is bound by the copies of whole pages:
// each page's K and V are two contiguous blocks of Hkv * page * D bytes.
#include "cache.cuh"

namespace xgr {

namespace {

constexpr int kPlanCtas = 8;
constexpr int kPlanThreads = 1024;
constexpr int kPlan = kPlanCtas * kPlanThreads;
constexpr int kSmemWords = 24576;       // two bitsets of up to 786432 pages in shared memory; above, in global memory
constexpr int kCopyThreads = 256;
constexpr int64_t kPartBytes = 32768;   // bytes of one block's share of a page copy

// Every thread of the cluster gets here before any goes on, and sees what the others wrote before.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Exclusive block scan of one int per thread (block of kPlanThreads); *total gets the sum.
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

// [b, e) of n things for this CTA, and of those for this thread (contiguous)
__device__ __forceinline__ void my_share(int n, int &b, int &e) {
    const int per = (n + kPlan - 1) / kPlan;
    b = min((int)(blockIdx.x * kPlanThreads + threadIdx.x) * per, n);
    e = min(b + per, n);
}

__device__ __forceinline__ bool page_ok(const CacheArgs &c, int id) { return id >= 0 && id < c.n_pages; }

// A bitset that marks go to: this CTA's own in shared memory, or the one in global memory.
__device__ __forceinline__ void mark(uint32_t *bits, int id) {
    const uint32_t bit = 1u << (id & 31);
    volatile uint32_t *w = bits + (id >> 5);
    if (!(*w & bit)) atomicOr(bits + (id >> 5), bit);
}

// A warp marks the pages of a line's first `held` entries in `used`, and of its
// first `full` ones in `whole`.  Eight entries a lane are read before the first
// is marked: the marks' atomics would hold back every later read, and a line
// would take a round trip per 32 entries.
__device__ __forceinline__ void mark_line(const CacheArgs &c, const int32_t *line, int held, int full,
                                          uint32_t *used, uint32_t *whole) {
    const int lane = threadIdx.x % 32;
    for (int i0 = lane; i0 < held; i0 += 256) {
        int id[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) id[k] = i0 + 32 * k < held ? line[i0 + 32 * k] : 0x7fffffff;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (i0 + 32 * k >= held) break;
            if (!page_ok(c, id[k])) {
                set_status(c.status, XGR_DEV_INDEX);
                continue;
            }
            mark(used, id[k]);
            if (i0 + 32 * k < full) mark(whole, id[k]);
        }
    }
}

// Adds this CTA's marks to the bitset in global memory.
__device__ __forceinline__ void flush_marks(uint32_t *to, const uint32_t *from, int words) {
    for (int w = threadIdx.x; w < words; w += kPlanThreads)
        if (from[w]) atomicOr(to + w, from[w]);
}

// the bits of word w that stand for pages
__device__ __forceinline__ uint32_t word_mask(const CacheArgs &c, int w) {
    const int n = c.n_pages - w * 32;
    return n >= 32 ? 0xffffffffu : (1u << n) - 1u;
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

// ---------------------------------------------------------------- fork

// Out row r's pages beyond its parent's, and whether the first takes a copy.
__device__ __forceinline__ int row_need(const ForkArgs &a, int r, int &copy) {
    const Child c = child_of(a, r);
    copy = 0;
    if (c.held > c.full) {
        const int id = c.line[c.full];
        copy = page_ok(a.c, id) && ((a.full[id >> 5] >> (id & 31) & 1) || a.lowest[id] != r);
    }
    int more = a.n_new && c.line ? a.n_new[r] : 0;
    if (more < 0) {
        set_status(a.c.status, XGR_DEV_INDEX);
        more = 0;
    }
    const int64_t grown = min((int64_t)c.len + more, (int64_t)a.c.max_pages << a.c.page_shift);
    return (int)((grown + a.c.page - 1) >> a.c.page_shift) - c.held + copy;
}

// Phases: clear; mark the pages that out rows hold; then the pages each row
// needs and the free pages, each as its share's sum, and after one more barrier
// in place.
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(ForkArgs a, int words) {
    extern __shared__ uint32_t own[];
    griddep_wait();
    griddep_launch_dependents();
    const bool in_smem = words <= kSmemWords;
    const int tid = blockIdx.x * kPlanThreads + threadIdx.x, lane = threadIdx.x % 32;
    for (int i = tid; i < words; i += kPlan) a.used[i] = a.full[i] = 0;
    if (in_smem)
        for (int i = threadIdx.x; i < 2 * words; i += kPlanThreads) own[i] = 0;
    for (int r = tid; r < a.n_out; r += kPlan) {     // `lowest` is read at partly filled pages only
        const Child c = child_of(a, r);
        if (c.held > c.full) {
            const int id = c.line[c.full];
            if (page_ok(a.c, id)) a.lowest[id] = 0x7fffffff;
        }
        if (c.line) a.owner[a.parent[r]] = r;        // of several children any one: it marks the parent's pages for all
    }
    cluster_sync();
    uint32_t *used = in_smem ? own : a.used, *full = in_smem ? own + words : a.full;
    // a warp takes up to 32 rows at a time: their parents and lengths are read at once, then their lines
    const int rows = min(32, (a.n_out + kPlan / 32 - 1) / (kPlan / 32));
    for (int r0 = tid / 32 * rows; r0 < a.n_out; r0 += kPlan / 32 * rows) {
        Child c{nullptr, 0, 0, 0};
        if (lane < rows && r0 + lane < a.n_out) {
            const int r = r0 + lane;
            c = child_of(a, r);
            if (c.held > c.full) {
                const int id = c.line[c.full];
                if (page_ok(a.c, id)) atomicMin(a.lowest + id, r);
            }
            if (c.line && a.owner[a.parent[r]] != r) c.held = 0;
        }
        for (int j = 0; j < rows; ++j) {
            const int32_t *line = reinterpret_cast<const int32_t *>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(c.line), j));
            const int held = __shfl_sync(0xffffffffu, c.held, j);
            mark_line(a.c, line, held, __shfl_sync(0xffffffffu, c.full, j), used, full);
            __syncwarp();
        }
    }
    if (in_smem) {
        __syncthreads();
        flush_marks(a.used, own, words);
        flush_marks(a.full, own + words, words);
    }
    cluster_sync();
    int r0, r1, w0, w1, need = 0, copy, free = 0;
    my_share(a.n_out, r0, r1);
    my_share(words, w0, w1);
#pragma unroll 4
    for (int r = r0; r < r1; ++r) {
        const int n = row_need(a, r, copy);
        a.row_copy[r] = copy;
        a.row_need[r] = n;
        need += n;
    }
    for (int w = w0; w < w1; ++w) free += __popc(~a.used[w] & word_mask(a.c, w));
    int all_need, all_free;
    need = block_scan(need, &all_need);
    free = block_scan(free, &all_free);
    if (threadIdx.x == 0) {
        a.sums[blockIdx.x] = all_need;
        a.sums[kPlanCtas + blockIdx.x] = all_free;
    }
    cluster_sync();
    for (int i = 0; i < (int)blockIdx.x; ++i) {
        need += a.sums[i];
        free += a.sums[kPlanCtas + i];
    }
    for (int r = r0; r < r1; ++r) {
        const int n = a.row_need[r];
        a.row_need[r] = need;
        need += n;
    }
    for (int w = w0; w < w1; ++w)
        for (uint32_t b = ~a.used[w] & word_mask(a.c, w); b; b &= b - 1) a.free_list[free++] = w * 32 + __ffs(b) - 1;
    if (tid == kPlan - 1) *a.n_free = free;          // (the last share ends at the last word)
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

__device__ __forceinline__ int pages_of(const CacheArgs &c, int r) {
    const int len = c.len[r];
    if (len < 0 || len > (int64_t)c.max_pages * c.page) {
        set_status(c.status, XGR_DEV_INDEX);
        return 0;
    }
    return (int)(((int64_t)len + c.page - 1) >> c.page_shift);
}

// Phases: clear; mark the pages that rows hold; their sums; then held pages
// before each word, the free slots below U and the held pages from U on, both
// ascending.
__global__ void __launch_bounds__(kPlanThreads) compact_plan_kernel(CompactArgs a, int words) {
    extern __shared__ uint32_t own[];
    griddep_wait();
    griddep_launch_dependents();
    const bool in_smem = words <= kSmemWords;
    const int tid = blockIdx.x * kPlanThreads + threadIdx.x;
    for (int i = tid; i < words; i += kPlan) a.used[i] = 0;
    if (in_smem)
        for (int i = threadIdx.x; i < words; i += kPlanThreads) own[i] = 0;
    cluster_sync();
    uint32_t *used = in_smem ? own : a.used;
    for (int r = tid / 32; r < a.c.n_rows; r += kPlan / 32) {
        mark_line(a.c, a.c.table + (int64_t)r * a.c.max_pages, pages_of(a.c, r), 0, used, used);
    }
    if (in_smem) {
        __syncthreads();
        flush_marks(a.used, own, words);
    }
    cluster_sync();
    int w0, w1, held = 0, all;
    my_share(words, w0, w1);
    for (int w = w0; w < w1; ++w) held += __popc(a.used[w]);
    held = block_scan(held, &all);
    if (threadIdx.x == 0) a.sums[blockIdx.x] = all;
    cluster_sync();
    int U = 0;
    for (int i = 0; i < kPlanCtas; ++i) {
        if (i < (int)blockIdx.x) held += a.sums[i];
        U += a.sums[i];
    }
    for (int w = w0; w < w1; ++w) {
        a.prefix[w] = held;
        const uint32_t bits = a.used[w];
        if (U >= w * 32 && U < w * 32 + 32) *a.below = held + __popc(bits & ((1u << (U & 31)) - 1u));
        held += __popc(bits);
    }
    if (tid == 0) {
        *a.n_used = U;
        if (U >= words * 32) *a.below = U;           // (every page is held)
    }
    cluster_sync();
    const int below = *a.below;                      // held pages below U: the far pages' ranks start there
    for (int w = w0; w < w1; ++w) {
        const uint32_t bits = a.used[w];
        const int before = a.prefix[w];
        for (uint32_t b = bits; b; b &= b - 1) {
            const int j = __ffs(b) - 1, id = w * 32 + j;
            if (id >= U) a.far[before + __popc(bits & ((1u << j) - 1u)) - below] = id;
        }
        for (uint32_t b = ~bits; b; b &= b - 1) {
            const int j = __ffs(b) - 1, id = w * 32 + j;
            if (id < U) a.hole[id - before - __popc(bits & ((1u << j) - 1u))] = id;
        }
    }
}

__global__ void __launch_bounds__(kCopyThreads) compact_apply_kernel(CompactArgs a, int parts) {
    griddep_wait();
    griddep_launch_dependents();
    const int U = *a.n_used;
    auto before = [&](int id) {   // held pages before page id
        return a.prefix[id >> 5] + __popc(a.used[id >> 5] & ((1u << (id & 31)) - 1u));
    };
    const int below = *a.below;
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

// one cluster of kPlanCtas CTAs, as a programmatic dependent of the kernel before
template <typename Args>
static cudaError_t launch_plan(void (*kernel)(Args, int), const Args &a, int words, int sets, cudaStream_t s) {
    static bool ready[kMaxDevices] = {};   // (one instance a kernel: their argument types differ)
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sets * kSmemWords * 4);
        if (e != cudaSuccess) return e;
        ready[dev] = true;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kPlanCtas);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = words <= kSmemWords ? (size_t)sets * words * 4 : 0;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kPlanCtas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a, words);
}

cudaError_t launch_cache_fork(const ForkArgs &a, cudaStream_t s) {
    const cudaError_t e = launch_plan(fork_plan_kernel, a, (a.c.n_pages + 31) / 32, 2, s);
    if (e != cudaSuccess) return e;
    const int parts = copy_parts(a.c);
    return launch_pdl(fork_apply_kernel, dim3(a.n_out * parts), dim3(kCopyThreads), 0, s, a, parts);
}

cudaError_t launch_cache_compact(const CompactArgs &a, cudaStream_t s) {
    const cudaError_t e = launch_plan(compact_plan_kernel, a, (a.c.n_pages + 31) / 32, 1, s);
    if (e != cudaSuccess) return e;
    const int parts = copy_parts(a.c);
    const int64_t most = std::max<int64_t>(a.c.n_rows, (int64_t)a.c.n_pages / 2 * parts);   // (moves fill free slots)
    return launch_pdl(compact_apply_kernel, dim3((unsigned)std::min<int64_t>(kSms * 8, std::max<int64_t>(most, 1))),
                      dim3(kCopyThreads), 0, s, a, parts);
}

}  // namespace xgr
