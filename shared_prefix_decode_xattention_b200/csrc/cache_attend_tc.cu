// cache_attend_tc.cu -- attention over the paged 8-bit cache for rows with
// many query rows (a chunk of a prompt, the beams of a request over its shared
// prompt), on the 5th-generation tensor cores.
//
// The mathematics is that of cache_attend.cu: the products take the codes
// themselves as fp16 numbers, the scales stay outside.  Here the exponent of
// the V scale joins the score: t_j = x_j log2 e + log2 b_j is the exponent of
// the weight w_j = b_j p_j, one lazily raised reference M per row bounds it
// (raised when a chunk passes it by more than 2^8), and l sums w_j / b_j, so
// neither scale costs an instruction per score.  That is sound while the V scales
// lie between 2^-60 and 2^30: beyond, a b_j far from the others would push w_j or
// l out of fp32's range.  From a segment's first chunk with such a scale on (pages
// of zeros have the smallest) l is summed from the scores themselves, 2^(x_j log2 e - P)
// with a reference P of its own.  Rounded are the weights (fp16) and the output
// (bf16); all else is fp32.
//
// One CTA per SM, persistent over its share of the work line (cache_plan.cuh);
// a tile is 256 query rows, two products of 128 rows; 16 warps:
//   warps 0-7    two softmax warpgroups, a query row a thread: scores from
//                tensor memory, cap, bias, mask, weights back over the scores'
//                buffer as fp16, and at a segment's end the output;
//   warp 8       issues the products: S_h = Q_h K^T, O_h += W_h V, whichever of
//                the two tiles is ready, so one tile's softmax runs beside the
//                other's products;
//   warps 9-15   the codes of each 128-key chunk, 16 bytes a copy from the pages
//                one chunk ahead, converted and written as the
//                128-byte-swizzled operands of K and V (rings of two).
// A conversion serves 256 query rows.  With 128 rows or fewer (a "narrow"
// segment) both warpgroups take the same rows and alternate chunks, and the
// first one folds the second's result in at the end.
// Registers: 512 threads start with 128 each; the softmax warpgroups take 192,
// the other two keep 64 (their sum is what the block has).
//
// What bounds it: a tile's chain of softmax, W V and the next Q K^T, whose
// scores may only be written once W V has read the weights over the old ones
// (tensor memory is full: two S, two O of 128 columns); two tiles overlap their
// chains.  Measured at 512 beams x 32 heads over 4096 keys, 16 requests (550
// GFLOP; 1692 TFLOP/s of bf16 would take 325 us): 713 us in ten passes after a
// pause, 771 TFLOP/s, 0.46 of the measured bf16 rate; 759 where hundreds run back to
// back and the clock settles lower.  Other forms, measured beside 692 us (without the
// way for far V scales, which costs its code 2 to 3 %): four conversion warps 696 us,
// three 870; weights through shared memory, so that the next scores need not wait, 740
// (the writes, and single operand buffers for want of room); the scores read in two
// rolled passes 790; spills in the issuing warp (48 registers) 822.
// Every wait is bounded (XGR_DEV_TIMEOUT and an unwound CTA, no hang).
#include "cache_codes.cuh"
#include "cache_plan.cuh"
#include "tcgen.cuh"

namespace xgr {

namespace {

constexpr int kThreads = 512;
constexpr int kConvWarps = 7;
constexpr int kConvThreads = 32 * kConvWarps;
constexpr int kIssueWarp = 8;
constexpr int kSoftmaxRegs = 192, kOtherRegs = 64;
constexpr int kChunk = 128;                    // keys of a chunk
constexpr int kRing = 4;                       // chunks whose scales are at hand
constexpr uint32_t kTmemCols = 512;            // S0 [0,128) S1 [128,256) O0 [256,384) O1 [384,512)
constexpr float kZeroLogV = -150.f;            // log2 of a V scale of 0, as good as it: 448 * 2^-150 is 0 in bf16
constexpr float kLowV = 0x1p-60f, kHighV = 0x1p30f;   // scales for which l may be summed from the weights
constexpr int kFar = 256;                      // of Scales::bad: the segment has met scales past those, or that are NaN

struct Scales {
    float2 k[8];                // by 16 keys: K scale, log2 V scale (0 where far)
    float iv[8];                // 1 / V scale (0 where far)
    float lv[8];                // log2 V scale
    int bad;                    // bit g: group g lies in a page that is not there; kFar (both take the slow way)
    int pad[3];
};

template <int D>
struct Lay {
    static constexpr uint32_t kHalf = 16384;                  // 128 rows x 64 fp16
    static constexpr uint32_t kTile = 128 * D * 2;
    static constexpr uint32_t q = 0;                          // two tiles
    static constexpr uint32_t k = 2 * kTile;                  // two stages
    static constexpr uint32_t v = 4 * kTile;
    static constexpr uint32_t raw = 6 * kTile;                // codes of the next K and V chunk (first the plan's scratch)
    static constexpr uint32_t sc = raw + 2 * kChunk * D;
    static constexpr uint32_t unit = sc + kRing * sizeof(Scales);
    static constexpr uint32_t x = kTile;                      // [128] (M, l) of a narrow segment's second half: it has no
                                                              // second Q tile
    static constexpr uint32_t bar = unit + 64;
    static constexpr uint32_t misc = bar + 256;
    static constexpr uint32_t total = misc + 16 + 1024;       // with room to align the window
};

enum { B_KFULL = 0, B_KEMPTY = 2, B_VFULL = 4, B_VEMPTY = 6, B_SFULL = 8, B_PFULL = 10, B_PVDONE = 12, B_QFULL = 14,
       B_SC = 16, B_XCH = B_SC + kRing, B_XDONE, B_DONE, B_COUNT };
static_assert(B_COUNT * 8 <= 256, "barrier area");

// byte offset of 16-byte chunk c of row `row` in a 128-row operand of 64-column swizzled halves
template <int D>
__device__ __forceinline__ uint32_t sw128(int row, int c) {
    return (uint32_t)(c >> 3) * Lay<D>::kHalf + (uint32_t)row * 128u + (uint32_t)(((c & 7) ^ (row & 7)) << 4);
}

// Softmax and conversion warps go on from a bounded wait whatever its verdict, and ask at the end of a segment whether one
// gave up: a lane that left a loop alone would leave the others in instructions that take all 32.  Until then they work on
// what is there; later waits end soon, as the flag is up, and nothing of the segment is written.  (A vote in the loops
// over chunks instead: 512 beams 722 us, 696 without, ten passes after a pause.)
__device__ __forceinline__ bool went_well(volatile int *abort) { return __all_sync(0xffffffffu, *abort == 0); }

// A segment as every role sees it.
struct Seg {
    RowSpan row;
    int u1, kb0, ke, chunks, rows;
    bool narrow;
    __device__ int tile_chunks(int h) const {   // chunks of S_h
        return narrow ? (chunks + 1 - h) / 2 : h == 0 || rows > 128 ? chunks : 0;
    }
    __device__ int chunk_of(int h, int i) const { return narrow ? 2 * i + h : i; }
};

__device__ __forceinline__ Seg segment(const AttendArgs &a, const Parts &w, const Cursor &cur, int left) {
    constexpr int R = 256;
    Seg s;
    s.row = row_span(a.c, cur.r, a.max_q);
    s.u1 = min(cur.units, cur.u + left);
    const KeyRange k = segment_keys(a, w, s.row, cur, s.u1, R);
    s.kb0 = k.lo & ~(kChunk - 1);
    s.ke = k.hi;
    s.chunks = k.hi > k.lo ? (k.hi - s.kb0 + kChunk - 1) / kChunk : 0;
    s.rows = min(R, s.row.n * a.G - cur.t * R);
    s.narrow = s.rows <= 128;
    return s;
}

// A row's state past the scales' limits, on the thread's stack: P (infinite before), and l relative to 2^P.
struct Far {
    float P, l;
};

// A chunk past the limits: its scores, log2 units without the V scales, into far.l (which takes over l, relative to 2^M, at
// the first), and the V scales onto them.  Called by whole warps; not inlined, as with far_mean: the loop around it rarely
// comes here and has no register to spare.
__device__ __noinline__ void far_sum(uint32_t ts, const Scales &sc, Far &far, float M, float l) {
    const bool begun = far.P != INFINITY;
    float P = begun ? far.P : M;
    if (begun) l = far.l;
#pragma unroll 1
    for (int p = 0; p < 4; ++p) {
        float x[32], top = -INFINITY, sum = 0.f;
        tc::ld32(ts + 32u * p, x);
        tc::wait_ld_into(x);
#pragma unroll
        for (int e = 0; e < 32; ++e) top = fmaxf(top, x[e]);
        const float up_to = fmaxf(P, top), ref = up_to == -INFINITY ? 0.f : up_to;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
            sum += exp2_fast(x[e] - ref + kTcBias);
            x[e] = x[e] == -INFINITY ? x[e] : x[e] + sc.lv[2 * p + e / 16];
        }
        l = l * exp2_fast(P - ref) + sum;
        P = up_to;
        __syncwarp();
        tc::st32(ts + 32u * p, reinterpret_cast<const uint32_t *>(x));
    }
    tc::wait_st();
    far = Far{fminf(P, 0x1.fffffep127f), l};   // (infinite stands for no such chunk, in every thread alike)
}

// The result of such a segment in the usual form, O and l relative to the same 2^M.  Any M would do but for fp32's range:
// with O the mean, l = 1, the parts of the row that others hold may be 2^-126 of it and still matter, if its own values are
// that small.  So l is up to 2^60, as far as O is below the mean's usual size: then whatever is lost where parts meet weighs
// less than 2^-100 of the row, or is less than 2^-40 of it beside larger values.
template <int D>
__device__ __noinline__ void far_mean(uint32_t to, const Far &far, float &M, float &l) {
    tc::fence_after();
    const float all = far.l + l * 0.f;        // (l has met the NaNs of V scales)
    const float top = far.P + log2f(all), k = rintf(fminf(fmaxf(top - M, 0.f), 60.f));
    const float mean = all == 0.f ? 0.f : 1.f / all, f = M == -INFINITY ? 0.f : exp2f(M - far.P + k);
#pragma unroll 1
    for (int p = 0; p < D / 32; ++p) {
        float o[32];
        tc::ld32(to + 32u * p, o);
        tc::wait_ld_into(o);
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = o[e] * mean * f;
        __syncwarp();
        tc::st32(to + 32u * p, reinterpret_cast<const uint32_t *>(o));
    }
    tc::wait_st();
    M = top - k;
    l = all == 0.f ? 0.f : exp2f(k);
}

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, 1) cache_attend_tc_kernel(AttendArgs a, PlanOut po, int min_units) {
    using L = Lay<D>;
    constexpr int R = 256;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const uint32_t sb = smem_u32(base);
    auto bar = [&](int i) { return sb + L::bar + 8u * (uint32_t)i; };
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(base + L::misc);
    volatile int *abort = reinterpret_cast<int *>(base + L::misc + 4);
    Scales *ring = reinterpret_cast<Scales *>(base + L::sc);
    float2 *xch = reinterpret_cast<float2 *>(base + L::x);
    float2 *unit = reinterpret_cast<float2 *>(base + L::unit);   // [8] (1, 0)
    const CacheArgs &c = a.c;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_KFULL + i), kConvThreads);
            mbar_init(bar(B_VFULL + i), kConvThreads);
            mbar_init(bar(B_KEMPTY + i), 2);      // a commit for each tile (two for a chunk of one tile)
            mbar_init(bar(B_VEMPTY + i), 2);
            mbar_init(bar(B_SFULL + i), 1);
            mbar_init(bar(B_PFULL + i), 128);
            mbar_init(bar(B_PVDONE + i), 1);
            mbar_init(bar(B_QFULL + i), 128);
        }
        for (int i = 0; i < kRing; ++i) mbar_init(bar(B_SC + i), 1);
        mbar_init(bar(B_XCH), 128);
        mbar_init(bar(B_XDONE), 128);
        mbar_init(bar(B_DONE), 1);
        for (int i = 0; i < 8; ++i) unit[i] = make_float2(1.f, 0.f);
        *abort = 0;
        fence_mbar_init();
    }
    griddep_wait();
    griddep_launch_dependents();
    Cursor cur;
    Parts &units = *reinterpret_cast<Parts *>(base + L::misc + 8);
    int64_t begin, end;
    if (!plan_begin<kThreads>(a, R, min_units, *reinterpret_cast<PlanSmem<kThreads> *>(base + L::raw), po, units, cur, begin, end)) return;   // (of the whole block)
    const int share = (int)(end - begin);            // units of this CTA
    if (warp == kIssueWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc::fence_before();
    __syncthreads();
    tc::fence_after();
    const uint32_t tmem = *tmem_holder;
    // a warpgroup's warps all take the same one: the last two warpgroups hold both of the other roles
    static_assert(256 * kSoftmaxRegs + (kThreads - 256) * kOtherRegs <= kThreads * 128, "no more than the block has");
    static_assert(kIssueWarp == 8 && kIssueWarp + 1 + kConvWarps == kThreads / 32, "two warpgroups and two");
    if (warp < 8) tc::regs_up<kSoftmaxRegs>();
    else tc::regs_down<kOtherRegs>();

    if (warp < 8) {
        // ------------------------------------------------------------ softmax
        const int h = warp / 4;
        const int tr = tid % 128;                                     // row of the tile, TMEM lane
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t ts = tmem + 128u * h + lanes, to = tmem + 256u + 128u * h + lanes;
        const bool capped = a.softcap > 0.f;
        int gc = 0;        // chunks of the segments before
        int cnt = 0;       // of them, this warpgroup's
        int nx = 0;        // narrow segments before
        for (int left = share; left > 0 && cur.r < c.n_rows;) {
            const Seg s = segment(a, units, cur, left);
            const int ia = cur.t * R + tr + (s.narrow ? 0 : 128 * h);
            const bool valid = ia < s.row.n * a.G;
            const int tok = valid ? ia / a.G : 0, head = cur.g * a.G + (valid ? ia % a.G : 0);
            KeyRange vis = query_keys(a, s.row, cur.r, tok);
            if (!valid) vis = KeyRange{0, 0x7fffffff};                // a row of zeros, never written
            const int n = s.tile_chunks(h);
            const float slope = a.slopes ? a.slopes[head] * kLog2e : 0.f;
            const int pos = s.row.len - s.row.n + tok;
            // ---- the warp's 32 query rows as fp16, near 1: copied into their places in the operand (D / 8 lanes a row,
            // whole lines), then scaled there.  (Loops stay mostly rolled: this code runs once a segment, and fetching
            // instructions that are not in the caches costs more than they do.)
            float fac = 0.f;
            if (s.chunks > 0 && (n > 0 || s.narrow)) {
                constexpr int kPer = 256 / D;          // rows of one copy of the warp
                const int64_t q_off = valid ? (int64_t)(s.row.t0 + tok) * a.q_stride + (int64_t)head * D : -1;
                const int ln = lane % (D / 8);
                const uint32_t qt = (s.narrow ? 0 : h) * L::kTile;
                if (!s.narrow || h == 0) {
#pragma unroll 4
                    for (int i = 0; i < 32 / kPer; ++i) {
                        const int rr = i * kPer + lane / (D / 8);
                        const int64_t off = __shfl_sync(0xffffffffu, q_off, rr);
                        cp_async16_zfill(sb + L::q + qt + sw128<D>(32 * (warp & 3) + rr, ln), a.q + (off >= 0 ? off + 8 * ln : 0),
                                         off >= 0);
                    }
                    cp_async_commit();
                    cp_async_wait_all();
                    __syncwarp();
                }
#pragma unroll 4
                for (int i = 0; i < 32 / kPer; ++i) {
                    const int rr = i * kPer + lane / (D / 8);
                    uint4 v;
                    if (!s.narrow || h == 0) {
                        v = *reinterpret_cast<const uint4 *>(base + L::q + qt + sw128<D>(32 * (warp & 3) + rr, ln));
                    } else {   // (the other warpgroup's rows: only their scale is needed)
                        const int64_t off = __shfl_sync(0xffffffffu, q_off, rr);
                        v = off >= 0 ? *reinterpret_cast<const uint4 *>(a.q + off + 8 * ln) : make_uint4(0, 0, 0, 0);
                    }
                    float f[8], top = 0.f;
                    unpack8(v, f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
#pragma unroll
                    for (int o = 1; o < D / 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                    const int ex = query_exp(top);
                    const float mine = __shfl_sync(0xffffffffu, a.scale * pow2i(ex), (lane % kPer) * (D / 8));
                    if (lane / kPer == i) fac = mine;
                    if (!s.narrow || h == 0) {
                        const float down = pow2i(-ex);
                        *reinterpret_cast<uint4 *>(base + L::q + qt + sw128<D>(32 * (warp & 3) + rr, ln)) =
                            make_uint4(pack_f16(f[0] * down, f[1] * down), pack_f16(f[2] * down, f[3] * down),
                                       pack_f16(f[4] * down, f[5] * down), pack_f16(f[6] * down, f[7] * down));
                    }
                }
                if (!s.narrow || h == 0) {
                    fence_async_smem();
                    mbar_arrive(bar(B_QFULL + h));
                }
            }
            // what one factor can hold of a score's way to log2 units
            const float f0 = capped ? fac * (2.f * kLog2e / a.softcap) : fac * kLog2e;
            const int lo_max = __reduce_max_sync(0xffffffffu, valid ? vis.lo : 0);
            const int hi_min = __reduce_min_sync(0xffffffffu, vis.hi);

            float M = -INFINITY, l = 0.f;
            Far far{INFINITY, 0.f};   // (of a segment with chunks marked kFar)
            for (int i = 0; i < n; ++i) {
                const int ch = s.chunk_of(h, i), gi = gc + ch;
                mbar_wait(bar(B_SC + gi % kRing), (gi / kRing) & 1, abort);
                mbar_wait(bar(B_SFULL + h), (cnt + i) & 1, abort);
                tc::fence_after();
                const Scales &sc = ring[gi % kRing];
                const int key0 = s.kb0 + ch * kChunk;
                const int bad = sc.bad;
                const bool masked = key0 < lo_max || key0 + kChunk > hi_min || bad;
                const bool slow = masked || capped || a.slopes;
                // Scores to exponents of weights, in place.  (Rolled: this and the body below, both unrolled, are longer
                // than the instruction caches next to the schedulers, and waiting for instructions cost more than the
                // second reading: 372 against 339 us for capped, masked chunks of 3700 tokens.)
                if (slow) {
                    const float up = a.softcap * kLog2e;
                    const float away = (float)(pos - key0);
#pragma unroll 1
                    for (int p = 0; p < 4; ++p) {
                        float x[32];
                        tc::ld32(ts + 32u * p, x);
                        const int r0 = vis.lo - key0 - 32 * p, r1 = vis.hi - key0 - 32 * p;
                        const uint32_t below = r0 >= 32 ? ~0u : r0 <= 0 ? 0u : (1u << r0) - 1u;
                        const uint32_t till = r1 >= 32 ? ~0u : r1 <= 0 ? 0u : (1u << r1) - 1u;
                        uint32_t seen = till & ~below;
                        const float2 g0 = sc.k[2 * p], g1 = sc.k[2 * p + 1];
                        const float k0 = g0.x * f0, k1 = g1.x * f0;
                        if (bad >> (2 * p) & 1) seen &= 0xffff0000u;
                        if (bad >> (2 * p + 1) & 1) seen &= 0x0000ffffu;
                        const float away_p = away - 32.f * p;
                        tc::wait_ld_into(x);
                        float most = 0.f;
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float k = e < 16 ? k0 : k1;
                            const float2 y = tc::fmul2(make_float2(x[e], x[e + 1]), make_float2(k, k));
                            x[e] = y.x;
                            x[e + 1] = y.y;
                            most = fmaxf(most, fmaxf(fabsf(y.x), fabsf(y.y)));
                        }
                        if (capped) {
                            if (__all_sync(0xffffffffu, most <= kTanhNear)) {
#pragma unroll
                                for (int e = 0; e < 32; e += 2) {
                                    const float2 y = tc::fmul2(tanh_near(make_float2(x[e], x[e + 1])), make_float2(up, up));
                                    x[e] = y.x;
                                    x[e + 1] = y.y;
                                }
                            } else {
#pragma unroll
                                for (int e = 0; e < 32; ++e) x[e] = up * tanh_score(x[e]);
                            }
                        }
                        if (a.slopes) {
#pragma unroll
                            for (int e = 0; e < 32; ++e) x[e] -= slope * fabsf(away_p - (float)e);
                        }
#pragma unroll
                        for (int e = 0; e < 32; ++e) x[e] = seen >> e & 1 ? x[e] + (e < 16 ? g0.y : g1.y) : -INFINITY;
                        __syncwarp();
                        tc::st32(ts + 32u * p, reinterpret_cast<const uint32_t *>(x));
                    }
                    tc::wait_st();
                    if (sc.bad & kFar) far_sum(ts, sc, far, M, l);
                }
                float x[128];
#pragma unroll
                for (int p = 0; p < 4; ++p) tc::ld32(ts + 32u * p, x + 32 * p);
#pragma unroll
                for (int p = 0; p < 4; ++p) tc::wait_ld_into(x + 32 * p);
                // t = fo.x f1 x + fo.y is a weight's exponent (x itself after the slow way)
                const float2 *fo = slow ? unit : sc.k;
                const float f1 = slow ? 1.f : f0;
                // ---- the largest weight's exponent, the row's reference
                float top = -INFINITY;
#pragma unroll
                for (int g = 0; g < 8; ++g) {
                    float m = fmaxf(x[16 * g], x[16 * g + 1]);
#pragma unroll
                    for (int e = 2; e < 16; e += 2) m = tc::fmax3(m, x[16 * g + e], x[16 * g + e + 1]);
                    const float2 kv = fo[g];
                    top = fmaxf(top, fmaf(m, kv.x * f1, kv.y));
                }
                const bool raise = top > M + 8.f || (M == -INFINITY && top > -INFINITY);
                float alpha = 1.f;
                if (raise) {
                    alpha = exp2_fast(M - top);
                    M = top;
                    l *= alpha;
                }
                if (i > 0 && __any_sync(0xffffffffu, raise)) {   // O_h holds every product so far: S_h waited for them
#pragma unroll 1
                    for (int p = 0; p < D / 32; ++p) {
                        float o[32];
                        tc::ld32(to + 32u * p, o);
                        tc::wait_ld_into(o);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] *= alpha;
                        tc::st32(to + 32u * p, reinterpret_cast<const uint32_t *>(o));
                    }
                }
                // ---- the weights
                const float ref = (M == -INFINITY ? 0.f : M) - kTcBias;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    uint32_t w[32];
#pragma unroll
                    for (int g = 4 * q; g < 4 * q + 4; ++g) {
                        const float2 kv = fo[g];
                        const float fg = kv.x * f1, dg = kv.y - ref;
                        const float2 ff = make_float2(fg, fg), dd = make_float2(dg, dg);
                        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            const float2 t = tc::ffma2(make_float2(x[16 * g + e], x[16 * g + e + 1]), ff, dd);
                            const float2 p = make_float2(exp2_fast(t.x), exp2_fast(t.y));
                            sum = tc::fadd2(sum, p);
                            w[8 * (g & 3) + e / 2] = pack_f16(p.x, p.y);
                        }
                        const float s0 = sum.x + sum.y;
                        l += s0 == 0.f ? 0.f : s0 * sc.iv[g];
                    }
                    __syncwarp();
                    tc::st32(ts + 32u * q, w);
                }
                tc::wait_st();
                tc::fence_before();
                mbar_arrive(bar(B_PFULL + h));
            }
            // ---- the segment's result
            if (n > 0) mbar_wait(bar(B_PVDONE + h), (cnt + n - 1) & 1, abort);
            cnt += n;
            gc += s.chunks;
            if (far.P != INFINITY) far_mean<D>(to, far, M, l);   // (of whole warps)
            bool fold = false;   // a narrow segment's second half is folded in
            float a0 = 1.f, a1 = 0.f;
            if (s.narrow && s.chunks > 1) {
                if (h == 1) {
                    tc::fence_before();
                    xch[tr] = make_float2(M, l);
                    mbar_arrive(bar(B_XCH));
                    mbar_wait(bar(B_XDONE), nx & 1, abort);   // O_1 and xch are read
                } else {
                    mbar_wait(bar(B_XCH), nx & 1, abort);
                    const float2 y = xch[tr];
                    const float m = fmaxf(M, y.x), ref = m == -INFINITY ? 0.f : m;
                    a0 = exp2_fast(M - ref);
                    a1 = exp2_fast(y.x - ref);
                    l = l * a0 + y.y * a1;
                    M = m;
                    fold = true;
                }
                ++nx;
            }
            if (!went_well(abort)) break;
            if (!s.narrow || h == 0) {
                tc::fence_after();
                const bool all = cur.u == 0 && s.u1 == cur.units;
                const int64_t oi = (int64_t)(s.row.t0 + tok) * a.Hq + head;
                const int64_t pi = ((int64_t)blockIdx.x * 2 + (cur.u == 0 ? 1 : 0)) * R + tr + 128 * h;
                const float ref = M == -INFINITY ? 0.f : M;
                const float scale = !all ? 1.f : l == 0.f ? 0.f : 1.f / l;
                // rows go out through the warp's own rows of the Q tile (no product reads them any more; another warp
                // may be filling its own for the next segment already), 2 D bytes a row at a time, so that stores are
                // whole lines
                auto slot = [&](int row, int ch) {
                    return base + L::q + h * L::kTile + sw128<D>(32 * (warp & 3) + row, ch);
                };
                auto flush = [&](uint8_t *dst, int64_t row_bytes, int64_t my_row) {   // lane's row of the result (-1: none)
                    __syncwarp();
#pragma unroll 4
                    for (int i = 0; i < D / 8; ++i) {
                        const int rr = i * (256 / D) + lane / (D / 8), ch = lane % (D / 8);
                        const int64_t row = __shfl_sync(0xffffffffu, my_row, rr);
                        const uint4 y = *reinterpret_cast<const uint4 *>(slot(rr, ch));
                        if (row >= 0) reinterpret_cast<uint4 *>(dst + row * row_bytes)[ch] = y;
                    }
                    __syncwarp();
                };
#pragma unroll 1
                for (int p = 0; p < D / 32; ++p) {
                    float o[32];
                    if (n > 0) {
                        tc::ld32(to + 32u * p, o);
                        tc::wait_ld_into(o);
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0.f;
                    }
                    if (fold) {
                        float o1[32];
                        tc::ld32(to + 128u + 32u * p, o1);
                        tc::wait_ld_into(o1);
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = o[e] * a0 + o1[e] * a1;
                    }
                    if (all) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint4 pk;
                            __nv_bfloat162 *b = reinterpret_cast<__nv_bfloat162 *>(&pk);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                b[j] = __floats2bfloat162_rn(o[8 * e + 2 * j] * scale, o[8 * e + 2 * j + 1] * scale);
                            *reinterpret_cast<uint4 *>(slot(lane, 4 * p + e)) = pk;
                        }
                    } else {
                        constexpr int kHalves = D / 64;   // 32-dim pieces of a pass of fp32
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            *reinterpret_cast<float4 *>(slot(lane, 8 * (p % kHalves) + e)) =
                                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
                        if (p % kHalves == kHalves - 1)
                            flush(reinterpret_cast<uint8_t *>(po.o) + (p / kHalves) * (2 * D), 4 * D, valid ? pi : -1);
                    }
                }
                if (all) flush(reinterpret_cast<uint8_t *>(a.out), 2 * D, valid ? oi : -1);
                if (valid) {
                    if (all) a.lse[oi] = l == 0.f ? -INFINITY : (ref - kTcBias + log2f(l)) * kLn2;
                    else po.ml[pi] = make_float2(M, l);
                }
                tc::fence_before();
                if (fold) mbar_arrive(bar(B_XDONE));
            }
            left -= s.u1 - cur.u;
            if (left > 0) plan_next(a, units, R, cur);
        }
    } else if (warp > kIssueWarp) {
        // ------------------------------------------------------------ codes to operands
        const int cw = warp - kIssueWarp - 1;
        // A block is the 512 bytes (kKeys keys) that a warp copies or converts at a time; warp cw takes every kConvWarps-th.
        // lane -> (key, 16-byte chunk) so that eight lanes' 16-byte writes meet no bank twice
        constexpr int kKeys = 512 / D, kBlocks = kChunk / kKeys, kTurns = (kBlocks + kConvWarps - 1) / kConvWarps;
        const int ck = D == 128 ? (lane & 3) | (lane >> 1 & 4) : lane & 3;
        const int kr = D == 128 ? (lane >> 2 & 1) | (lane >> 3 & 2) : lane >> 2;
        int gc = 0;
        for (int left = share; left > 0 && cur.r < c.n_rows;) {
            const Seg s = segment(a, units, cur, left);
            const int32_t *line = c.table + (int64_t)cur.r * c.max_pages;
            // Lane g of every warp holds group g % 8 of a chunk: its page (-2: no keys, -1: no such page), and where its
            // 16 keys lie, in blocks of 16 keys (they are contiguous in a page and head).
            auto ids_of = [&](int ch) {
                const int key = s.kb0 + ch * kChunk + 16 * (lane & 7);
                int id = -2;
                if (ch < s.chunks && key < s.ke) {
                    id = line[key >> c.page_shift];
                    if (id < 0 || id >= c.n_pages) {
                        if (cw == 0) set_status(c.status, XGR_DEV_INDEX);
                        id = -1;
                    }
                }
                return id;
            };
            auto block_of = [&](int ch, int id) {
                const int key = s.kb0 + ch * kChunk + 16 * (lane & 7);
                return id < 0 ? -1 : (id * c.Hkv + cur.g) * (c.page / 16) + (key & (c.page - 1)) / 16;
            };
            int met = 0;   // kFar: a chunk of the segment had a scale past the limits
            // a thread's codes wait in shared memory of its own (16 bytes of each block)
            const uint32_t raw = L::raw + 16u * lane, raw_v = raw + kChunk * D;
            auto load = [&](const uint8_t *src, uint32_t to, int ch, int block) {
                if (ch < s.chunks) {
                    const int left = s.ke - s.kb0 - ch * kChunk;               // keys from the chunk's first one on
#pragma unroll
                    for (int i = 0; i < kTurns; ++i) {
                        const int blk = i * kConvWarps + cw, kl = blk * kKeys + kr;
                        const int b = __shfl_sync(0xffffffffu, block, kl / 16);
                        const bool in = b >= 0 && kl < left;
                        if (blk < kBlocks)
                            cp_async16_zfill(sb + to + blk * 512, src + (int64_t)(in ? b : 0) * (16 * D) + (kl % 16) * D + ck * 16, in);
                    }
                }
                cp_async_commit();
            };
            auto put = [&](uint32_t off, uint32_t from) {
#pragma unroll
                for (int i = 0; i < kTurns; ++i) {
                    const int blk = i * kConvWarps + cw, kl = blk * kKeys + kr;
                    if (blk < kBlocks) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(base + from + blk * 512);
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                        uint32_t o[8];
#pragma unroll
                        for (int e = 0; e < 4; ++e) codes_to_f16<FMT>(w[e], o[2 * e], o[2 * e + 1]);
                        *reinterpret_cast<uint4 *>(base + off + sw128<D>(kl, 2 * ck)) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4 *>(base + off + sw128<D>(kl, 2 * ck + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                }
                fence_async_smem();
            };
            int ids = ids_of(0), next = ids_of(1);
            int block = block_of(0, ids);
            load(c.k, raw, 0, block);
            load(c.v, raw_v, 0, block);
            for (int ch = 0; ch < s.chunks; ++ch) {
                const int gi = gc + ch, st = gi & 1;
                const int ids2 = next;
                next = ids_of(ch + 2);
                if (gi >= 2) mbar_wait(bar(B_KEMPTY + st), ((gi >> 1) - 1) & 1, abort);
                // (S of chunk gi - 2 is complete, so the softmax is done with the scales of chunk gi - 4)
                if (cw == 0) {   // the chunk's scales
                    float ks = 0.f, vs = 1.f;
                    if (ids >= 0) {
                        const int64_t at_s = (int64_t)ids * c.Hkv + cur.g;
                        ks = clean_scale(c.ks[at_s]);
                        vs = clean_scale(c.vs[at_s]);
                    }
                    if (__any_sync(0xffffffffu, !(vs >= kLowV && vs <= kHighV) || ks != ks)) met = kFar;
                    const float lv = vs != vs ? vs : fmaxf(log2f(vs), kZeroLogV);
                    Scales &sc = ring[gi % kRing];
                    const uint32_t gone = __ballot_sync(0xffffffffu, ids == -1) & 255u;
                    if (lane < 8) {
                        sc.k[lane] = make_float2(ks, met ? 0.f : lv);
                        sc.iv[lane] = met ? 0.f : exp2f(-lv);
                        sc.lv[lane] = lv;
                    }
                    if (lane == 0) sc.bad = (int)gone | met;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_SC + gi % kRing));
                }
                cp_async_wait_group<1>();
                put(L::k + st * L::kTile, raw);
                mbar_arrive(bar(B_KFULL + st));
                block = block_of(ch + 1, ids2);
                load(c.k, raw, ch + 1, block);
                if (gi >= 2) mbar_wait(bar(B_VEMPTY + st), ((gi >> 1) - 1) & 1, abort);
                cp_async_wait_group<1>();
                put(L::v + st * L::kTile, raw_v);
                mbar_arrive(bar(B_VFULL + st));
                load(c.v, raw_v, ch + 1, block);
                ids = ids2;
            }
            if (!went_well(abort)) break;
            gc += s.chunks;
            left -= s.u1 - cur.u;
            if (left > 0) plan_next(a, units, R, cur);
        }
        cp_async_wait_all();
    } else {
        // ------------------------------------------------------------ products
        {
            constexpr uint32_t idS = tc::idesc_f16(128, 128, false), idO = tc::idesc_f16(128, D, true);
            int gc = 0, cnt0 = 0, cnt1 = 0, nq0 = 0, nq1 = 0;
            // operands' descriptors: their low words are these, the high word is the same for all
            const uint32_t dq = tc::desc_lo(sb + L::q, 16), dk = tc::desc_lo(sb + L::k, 16), dv = tc::desc_lo(sb + L::v, L::kHalf);
            bool ok = true;
            for (int left = share; ok && left > 0 && cur.r < c.n_rows;) {
                const Seg s = segment(a, units, cur, left);
                if (lane == 0 && s.chunks > 0) {
                    const int n[2] = {s.tile_chunks(0), s.tile_chunks(1)};
                    const int cnt[2] = {cnt0, cnt1};
                    // the buffers of the segment before are free
                    if (cnt0 > 0) ok = mbar_wait(bar(B_PVDONE), (cnt0 - 1) & 1, abort);
                    if (ok && cnt1 > 0) ok = mbar_wait(bar(B_PVDONE + 1), (cnt1 - 1) & 1, abort);
                    if (ok) ok = mbar_wait(bar(B_QFULL), nq0 & 1, abort);
                    if (ok && n[1] > 0 && !s.narrow) ok = mbar_wait(bar(B_QFULL + 1), nq1 & 1, abort);
                    const bool alone = s.narrow || n[1] == 0;   // a chunk feeds one tile: it commits for both
                    int is[2] = {0, 0}, ip[2] = {0, 0};
                    uint32_t idle = 0;
                    while (ok && (ip[0] < n[0] || ip[1] < n[1])) {
                        bool progress = false;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            if (ip[h] < is[h]) {   // O_h += W_h V
                                const int gi = gc + s.chunk_of(h, ip[h]), st = gi & 1;
                                if (mbar_test(bar(B_PFULL + h), (cnt[h] + ip[h]) & 1) &&
                                    mbar_test(bar(B_VFULL + st), (gi >> 1) & 1)) {
                                    tc::fence_after();
                                    const uint32_t v = dv + st * (L::kTile >> 4);
#pragma unroll
                                    for (int k = 0; k < 8; ++k)
                                        tc::mma_ts(tmem + 256u + 128u * h, tmem + 128u * h + 8u * k, tc::desc_of(v + k * (2048 >> 4)),
                                                   idO, (k > 0 || ip[h] > 0) ? 1u : 0u);
                                    tc::commit(bar(B_PVDONE + h));
                                    tc::commit(bar(B_VEMPTY + st));
                                    if (alone) tc::commit(bar(B_VEMPTY + st));
                                    ++ip[h];
                                    progress = true;
                                }
                            }
                            if (is[h] < n[h] && is[h] == ip[h] &&
                                (is[h] == 0 || mbar_test(bar(B_PVDONE + h), (cnt[h] + is[h] - 1) & 1))) {   // S_h = Q_h K^T
                                const int gi = gc + s.chunk_of(h, is[h]), st = gi & 1;
                                if (mbar_test(bar(B_KFULL + st), (gi >> 1) & 1)) {
                                    tc::fence_after();
                                    const uint32_t q = dq + (s.narrow ? 0 : h) * (L::kTile >> 4);
                                    const uint32_t kk = dk + st * (L::kTile >> 4);
#pragma unroll
                                    for (int k = 0; k < D / 16; ++k) {
                                        const uint32_t off = ((uint32_t)(k >> 2) * L::kHalf + (uint32_t)(k & 3) * 32u) >> 4;
                                        tc::mma_ss(tmem + 128u * h, tc::desc_of(q + off), tc::desc_of(kk + off), idS, k > 0);
                                    }
                                    tc::commit(bar(B_SFULL + h));
                                    tc::commit(bar(B_KEMPTY + st));
                                    if (alone) tc::commit(bar(B_KEMPTY + st));
                                    ++is[h];
                                    progress = true;
                                }
                            }
                        }
                        if (progress) {
                            idle = 0;
                        } else if (++idle >= kSpinLimit) {
                            *abort = 1;
                            ok = false;
                        } else if ((idle & 255) == 0 && *abort) {
                            ok = false;
                        }
                    }
                    cnt0 += n[0];
                    cnt1 += n[1];
                    ++nq0;
                    if (!s.narrow && n[1] > 0) ++nq1;
                }
                ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
                gc += s.chunks;
                left -= s.u1 - cur.u;
                if (left > 0) plan_next(a, units, R, cur);
            }
            if (lane == 0) {   // every product issued has completed before tensor memory is given back
                tc::commit(bar(B_DONE));
                mbar_wait(bar(B_DONE), 0, nullptr);
            }
            __syncwarp();
        }
    }
    tc::fence_before();
    __syncthreads();
    if (tid == 0 && *abort) set_status(c.status, XGR_DEV_TIMEOUT);
    if (warp == kIssueWarp) {
        tc::fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

template <int D, int FMT>
cudaError_t launch_t(const AttendArgs &a, const PlanOut &po, int ctas, int min_units, cudaStream_t s) {
    static bool ready[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
        cudaFuncAttributes fa;
        e = cudaFuncGetAttributes(&fa, cache_attend_tc_kernel<D, FMT>);
        if (e != cudaSuccess) return e;
        if (fa.numRegs != 128) return cudaErrorInvalidConfiguration;   // the warpgroups share out 512 x 128
        e = cudaFuncSetAttribute(cache_attend_tc_kernel<D, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)Lay<D>::total);
        if (e != cudaSuccess) return e;
        ready[dev] = true;
    }
    return launch_pdl(cache_attend_tc_kernel<D, FMT>, dim3(ctas), dim3(kThreads), Lay<D>::total, s, a, po, min_units);
}

}  // namespace

cudaError_t launch_attend_tc(const AttendArgs &a, const PlanOut &po, int ctas, int min_units, cudaStream_t s) {
    if (a.c.D == 128)
        return a.c.fmt == XGR_CACHE_E4M3 ? launch_t<128, XGR_CACHE_E4M3>(a, po, ctas, min_units, s)
                                         : launch_t<128, XGR_CACHE_INT8>(a, po, ctas, min_units, s);
    return a.c.fmt == XGR_CACHE_E4M3 ? launch_t<64, XGR_CACHE_E4M3>(a, po, ctas, min_units, s)
                                     : launch_t<64, XGR_CACHE_INT8>(a, po, ctas, min_units, s);
}

}  // namespace xgr
