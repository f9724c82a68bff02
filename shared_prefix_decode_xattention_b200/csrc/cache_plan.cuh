// cache_plan.cuh -- how the attention over the paged cache is cut into work
// (internal; shared by its kernels).
//
// A row's query rows (new tokens x query heads of a kv head, token-major) are
// cut into tiles of R; a segment is (row, tile, kv head) and its keys are cut
// into units of kUnitKeys.  All units of all segments form one line, and CTA c
// of N takes units [c * per, (c + 1) * per): rows of any raggedness load the
// CTAs evenly, however few they are.  A segment cut by a CTA's end leaves
// partial results (O relative to its reference, m, l) in the workspace, at most
// two a CTA (the segment it continues, slot 0, and the one it leaves
// unfinished, slot 1), and the join kernel folds them: every cut segment is the
// one that some CTA begins in the middle of, so it runs over the CTAs' first
// cursors.  Lengths are read on the device, so nothing waits for the host;
// every CTA works the plan out anew from d_cu and d_len.
//
// In "whole" mode (every row is short) a unit is a whole segment: nothing is
// cut and no join runs.
//
// A segment also costs something before its first key (its query rows, its
// result): AttendArgs::lead units of it stand for that, at its front, without
// keys.  A CTA's end that would fall into them, or leave or take fewer than that
// many units of keys, moves to the segment's edge.  Where such segments are at
// most half as many as the CTAs, every segment is cut into equal parts of its
// own instead, a CTA a part (a unit is then a part).
#pragma once

#include "cache.cuh"
#include "tcgen.cuh"

namespace xgr {

constexpr int kUnitKeys = 128;

// Where a CTA stands in the line.
struct Cursor {
    int r, t, g;     // segment
    int u;           // unit within it
    int units;       // its units
};

// Results of parts of segments, for the join (null in whole mode).
struct PlanOut {
    Cursor *first;       // [N] each CTA's first cursor (u = 0: it cuts nothing)
    float *o;            // [N][2][R][D]
    float2 *ml;          // [N][2][R]
};

struct KeyRange {
    int lo, hi;
};

// The tiles of all rows are numbered with gaps: row r's begin at tile_slot (no
// row has more tiles than the gap to the next row's), so a slot's row is found
// from d_cu alone and the plan runs over slots, one or a few a thread, however
// the tokens are spread.  R is a power of two.
__device__ __forceinline__ int64_t tile_slot(const AttendArgs &a, int r, int R) {
    return ((int64_t)a.c.cu[r] * a.G >> (31 - __clz(R))) + r;
}
__device__ __forceinline__ int64_t tile_slots(const AttendArgs &a, int R) {
    return ((int64_t)a.c.n_tokens * a.G >> (31 - __clz(R))) + a.c.n_rows;
}

// First key of the window of a query at pos (below 0 where beams outnumber the row's keys).
__device__ __forceinline__ int window_lo(const AttendArgs &a, int pos) { return pos >= a.window ? pos - a.window + 1 : 0; }

// The keys [lo, hi) that some query of tile t of a row with span s may see.
__device__ __forceinline__ KeyRange tile_keys(const AttendArgs &a, const RowSpan &s, int r, int R, int t) {
    KeyRange k{0, s.len};
    const int i0 = t * R / a.G, i1 = (min((t + 1) * R, s.n * a.G) - 1) / a.G;   // its tokens
    const int p0 = s.len - s.n;
    if (a.causal) {
        k.hi = p0 + i1 + 1;
        if (a.prefix) k.hi = max(k.hi, min(a.prefix[r], s.len));
    }
    if (a.window > 0) k.lo = window_lo(a, p0 + i0);
    if (a.first) k.lo = max(k.lo, a.tile_lo[tile_slot(a, r, R) + t]);
    return k;
}

// chunks of kUnitKeys keys that a range touches
__device__ __forceinline__ int range_chunks(const KeyRange &k) {
    return max(0, (k.hi + kUnitKeys - 1) / kUnitKeys - k.lo / kUnitKeys);
}

// What a unit is.  NoParts: kUnitKeys keys (or one of the lead).  Parts, with parts > 0: a part of a segment, `parts` of
// them shared out beside one a segment, in proportion to its share of all `chunks`.
struct NoParts {
    static constexpr bool kParts = false;
    static constexpr int parts = 0, chunks = 1;
};
struct Parts {
    static constexpr bool kParts = true;
    int parts, chunks;
};

template <typename U>
__device__ __forceinline__ int range_units(const AttendArgs &a, const U &w, const KeyRange &k) {
    if (a.whole) return 1;
    const int n = range_chunks(k);
    if (U::kParts && w.parts > 0) return (int)max((int64_t)1, min((int64_t)n / 2, 1 + (int64_t)n * w.parts / w.chunks));
    return max(1, a.lead + n);
}

__device__ __forceinline__ int row_tiles(const AttendArgs &a, const RowSpan &s, int R) {
    return (int)(((int64_t)s.n * a.G + R - 1) / R);
}

// The row and tile of a slot (t past the row's tiles: an empty slot).
__device__ __forceinline__ RowSpan slot_tile(const AttendArgs &a, int R, int64_t slot, int &r, int64_t &t) {
    int lo = 0, hi = a.c.n_rows - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (tile_slot(a, mid, R) <= slot) lo = mid;
        else hi = mid - 1;
    }
    r = lo;
    t = slot - tile_slot(a, lo, R);
    return row_span(a.c, lo, a.max_q);
}

// The keys of a slot's tile (false: an empty slot).
__device__ __forceinline__ bool slot_keys(const AttendArgs &a, int R, int64_t slot, int &r, int64_t &t, KeyRange &k) {
    const RowSpan s = slot_tile(a, R, slot, r, t);
    if (t < 0 || t >= row_tiles(a, s, R)) return false;
    k = tile_keys(a, s, r, R, (int)t);
    return true;
}

// The segment after cur; cur.r = n_rows behind the last one.
template <typename U>
__device__ __forceinline__ void plan_next(const AttendArgs &a, const U &w, int R, Cursor &cur) {
    cur.u = 0;
    if (++cur.g < a.c.Hkv) return;
    cur.g = 0;
    ++cur.t;
    for (; cur.r < a.c.n_rows; ++cur.r, cur.t = 0) {
        const RowSpan s = row_span(a.c, cur.r, a.max_q);
        if (cur.t >= row_tiles(a, s, R)) continue;
        cur.units = range_units(a, w, tile_keys(a, s, cur.r, R, cur.t));
        return;
    }
}

// Shared memory of plan_begin.
template <int T>
struct PlanSmem {
    int64_t base[T / 32 + 1];
    int64_t edge[2];
    Cursor first;
};

// Exclusive sum over the block's threads; the sum of all is sm.base[T / 32].  `any`: whether it was set in any thread.
template <int T>
__device__ __forceinline__ int64_t plan_scan(PlanSmem<T> &sm, int64_t v, bool &any) {
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    any = __syncthreads_or(any);
    if (lane == 31) sm.base[warp + 1] = x;
    if (threadIdx.x == 0) sm.base[0] = 0;
    __syncthreads();
    if (threadIdx.x == 0)
        for (int i = 0; i < T / 32; ++i) sm.base[i + 1] += sm.base[i];
    __syncthreads();
    return sm.base[warp] + x - v;
}

// Every thread of the block gets the block's first cursor and [begin, end)
// (false: no work).  T = threads of the block; w: shared memory where it is Parts.
template <int T, typename U>
__device__ __forceinline__ bool plan_begin(const AttendArgs &a, int R, int min_units, PlanSmem<T> &sm,
                                           const PlanOut &p, U &w, Cursor &cur, int64_t &begin, int64_t &end) {
    const int64_t slots = tile_slots(a, R), spt = (slots + T - 1) / T;
    const int64_t s0 = min(threadIdx.x * spt, slots), s1 = min(s0 + spt, slots);
    const CuPair pair = cu_pair(a.c, min((int)threadIdx.x, a.c.n_rows - 1));
    bool bad = false;
    for (int i = threadIdx.x + T; i < a.c.n_rows; i += T) bad |= out_of_order(a.c, cu_pair(a.c, i));
    int units = 0, r = 0;
    int64_t t = 0;
    KeyRange k{0, 0};
    if constexpr (U::kParts) {   // chunks and segments in all
        int64_t both = 0;
        bool unused = false;
        if (!a.whole)
            for (int64_t s = s0; s < s1; ++s)
                if (slot_keys(a, R, s, r, t, k)) both += ((int64_t)range_chunks(k) << 24) + 1;
        plan_scan<T>(sm, both, unused);
        const int64_t segs = (sm.base[T / 32] & 0xffffff) * a.c.Hkv, chunks = (sm.base[T / 32] >> 24) * a.c.Hkv;
        const bool few = segs > 0 && segs * 2 <= gridDim.x && chunks < 0x7fffffff;
        if (threadIdx.x == 0) {
            w.parts = few ? (int)(gridDim.x - segs) : 0;
            w.chunks = few ? max((int)chunks, 1) : 1;
        }
        __syncthreads();
        if (few) min_units = 1;
    }
    int64_t mine = 0;
    for (int64_t s = s0; s < s1; ++s) {
        units = 0;
        if (slot_keys(a, R, s, r, t, k)) units = range_units(a, w, k);
        mine += (int64_t)units * a.c.Hkv;
    }
    bad |= out_of_order(a.c, pair);
    const int64_t from = plan_scan<T>(sm, mine, bad);     // first unit of this thread's slots
    if (bad) mine = 0;                                // (of every block: there is no work)
    const int64_t total = bad ? 0 : sm.base[T / 32];
    const int64_t per = max((int64_t)min_units, (total + gridDim.x - 1) / gridDim.x);
    // the block's two edges, each found by the thread whose slots hold it
#pragma unroll 1
    for (int e = 1; e >= 0; --e) {
        const int64_t edge = min((blockIdx.x + e) * per, total);
        if (edge == total && threadIdx.x == 0) sm.edge[e] = total;
        if (from > edge || edge >= from + mine) continue;
        int64_t left = edge - from;
        if (spt > 1)                              // (one slot: it is at hand)
            for (int64_t s = s0; s < s1; ++s) {
                units = 0;
                if (slot_keys(a, R, s, r, t, k)) units = range_units(a, w, k);
                if (left < (int64_t)units * a.c.Hkv) break;
                left -= (int64_t)units * a.c.Hkv;
            }
        units = max(units, 1);
        int u = (int)(left % units);
        if (!U::kParts || w.parts == 0) {
            if (u > 0 && u - a.lead < a.lead) u = 0;
            if (u > 0 && units - u < a.lead) u = units;
        }
        sm.edge[e] = edge - left % units + u;
        if (e == 0) sm.first = Cursor{r, (int)t, min((int)(left / units), a.c.Hkv - 1), u, units};
    }
    __syncthreads();
    begin = sm.edge[0];
    end = sm.edge[1];
    if (begin < end) {
        cur = sm.first;
        if (cur.u == cur.units) plan_next(a, w, R, cur);
    } else {
        cur = Cursor{0, 0, 0, 0, 0};
    }
    if (threadIdx.x == 0 && bad) set_status(a.c.status, XGR_DEV_INDEX);
    if (threadIdx.x == 0 && p.first) p.first[blockIdx.x] = cur;
    return begin < end;
}

// Query i of row span s at position pos sees [lo, hi).
__device__ __forceinline__ KeyRange query_keys(const AttendArgs &a, const RowSpan &s, int r, int i) {
    const int pos = s.len - s.n + i;
    KeyRange k{0, s.len};
    if (a.causal) {
        k.hi = pos + 1;
        if (a.prefix) k.hi = max(k.hi, min(a.prefix[r], s.len));
    }
    if (a.window > 0) k.lo = window_lo(a, pos);
    if (a.first) k.lo = max(k.lo, a.first[s.t0 + i]);
    return k;
}

// The keys of units [cur.u, u1) of segment cur (hi <= lo: none).
template <typename U>
__device__ __forceinline__ KeyRange segment_keys(const AttendArgs &a, const U &w, const RowSpan &s,
                                                 const Cursor &cur, int u1, int R) {
    const KeyRange k = tile_keys(a, s, cur.r, R, cur.t);
    if (a.whole) return k;
    const int c0 = k.lo / kUnitKeys;
    int b = max(cur.u - a.lead, 0), e = max(u1 - a.lead, 0);        // chunks of the range
    if (U::kParts && w.parts > 0) {
        const int64_t n = range_chunks(k);
        b = (int)(cur.u * n / cur.units);
        e = (int)(u1 * n / cur.units);
    }
    return KeyRange{max(k.lo, (c0 + b) * kUnitKeys), min(k.hi, (c0 + e) * kUnitKeys)};
}

__device__ __forceinline__ float exp2_fast(float x) {   // one MUFU op; tiny results flush to 0
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float log2_fast(float x) {   // one MUFU op and the scaling of tiny arguments
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// c * tanh(y) with tanh from one exponential and one reciprocal: 1 - 2 / (1 + e^2y).
// Its error is a few 2^-24 absolute, which is what counts in an exponent; the
// hardware's own tanh (about 2^-11) would put 2 % on a weight at a cap of 50.
__device__ __forceinline__ float tanh_score(float y2) {   // y2 = 2 log2(e) y
    return 1.f - __fdividef(2.f, 1.f + exp2_fast(y2));
}

// The same for a pair of small arguments, |y| <= 1/2 (kTanhNear in y2's units):
// tanh y = y P(y^2) with P of degree 4, a Chebyshev fit of tanh(y) / y on
// [0, 1/4] whose relative error is 2.7e-8 (1.3e-7 with the roundings of its
// evaluation in fp32).  Scores are mostly this far inside their cap, and two
// MUFU operations a score (8 cycles of a warp's scheduler each) cost more than
// the polynomial's packed FMAs.
constexpr float kTanhNear = kLog2e;
constexpr double tanh_coef(double c, int i) {   // c y^(2i + 1) as a factor of y2^(2i + 1)
    double f = c;
    for (int k = 0; k < 2 * i + 1; ++k) f /= 2.0 * 1.4426950408889634;
    return f;
}
__device__ __forceinline__ float2 tanh_near(float2 y2) {
    constexpr float c0 = (float)tanh_coef(1.0, 0), c1 = (float)tanh_coef(-0x1.5554a60000000p-2, 1),
                    c2 = (float)tanh_coef(0x1.10e47a0000000p-3, 2), c3 = (float)tanh_coef(-0x1.b2167e0000000p-5, 3),
                    c4 = (float)tanh_coef(0x1.18d7e80000000p-6, 4);
    const float2 u = tc::fmul2(y2, y2);
    float2 r = tc::ffma2(u, make_float2(c4, c4), make_float2(c3, c3));
    r = tc::ffma2(r, u, make_float2(c2, c2));
    r = tc::ffma2(r, u, make_float2(c1, c1));
    r = tc::ffma2(r, u, make_float2(c0, c0));
    return tc::fmul2(r, y2);
}

// V scales and K scales: finite and non-negative, or NaN for a page that got a
// NaN or an infinity; an infinite one counts as NaN.
__device__ __forceinline__ float clean_scale(float s) {
    return fabsf(s) < INFINITY ? s : __int_as_float(0x7fc00000);
}

// The weights are kept as 2^14 p (fp16 in the products): p <= 1 leaves the top
// of fp16's range, so a weight as small as 2^-38 of the row's largest still counts.
constexpr float kBias = 14.f;
constexpr float kTcBias = 7.f;   // of the tcgen05 kernel, whose reference lags by up to 2^8

// cache_attend_tc.cu: 256-row tiles, one CTA an SM
cudaError_t launch_attend_tc(const AttendArgs &a, const PlanOut &po, int ctas, int min_units, cudaStream_t s);

}  // namespace xgr
