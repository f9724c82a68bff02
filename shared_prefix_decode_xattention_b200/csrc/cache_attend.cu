// cache_attend.cu -- attention over the paged 8-bit cache for rows with few
// query rows (a decode step's single tokens, a few speculated ones, small
// beams), and the join of partial results.
//
// Mathematics: with codes k_j, v_j, scales a_j, b_j (one for each page and kv
// head) the scores are x_j = (q . k_j) a_j scale (capped, biased), the output
// sum_j w_j v_j / l with w_j = 2^(x_j log2 e - m) b_j and l = sum_j 2^(x_j log2 e - m):
// the scales leave the products, so the tensor cores multiply the codes
// themselves.  Every 8-bit code is an fp16 number, and a bf16 query row is one
// but for a power of two (2^e of its largest element, put back on the scores;
// elements below 2^-17 of the row's largest lose bits, less than 2^-25 of it
// absolute), so no product is rounded; sums, maxima and l are fp32.  The weights
// are rounded to fp16 (2^-11 relative, finer than the bf16 of the output).  To
// keep them within its range b_j is taken relative to a reference of the warp's,
// 2^6 times the first scale it meets, as long as all its scales lie between 2^-11
// and 2 of that (a caller's usually do).  From the first that does not on (pages
// of zeros beside others, an outlier, another quantiser's) each row keeps the
// largest x_j log2 e + log2 b_j of the keys it sees as a reference of its own and
// w_j is an exponential of its own, so that a page nobody attends, however large
// its scale, takes no bits from the others.
//
// Layout: bound by streaming the codes from HBM.  A warp takes 32 keys at a
// time through a ring of its own in shared memory (cp.async, 16 bytes a lane,
// zero-filled behind the row's end), and multiplies with mma.sync m16n8k16: few
// query rows (16 or 32 a tile) would leave a 128-row tcgen05 tile empty.  The
// rows of a tile share one pass over the keys and one conversion of the codes.
// The contraction index of a product may be permuted freely, so a lane's
// fragment of K is 16 consecutive bytes of one key and of V 16 consecutive
// dims of four keys: conversion needs no shuffles, the weights' fragments are
// the scores' own registers, and all shared-memory reads are 16 bytes wide and
// free of bank conflicts (perm and swz below).
//
// Measured: 64 rows of one token over 8.4k-10.2k e4m3 keys (1.23 GB, 32 / 8 heads,
// D = 128): 220 us, 5.6 TB/s; capped 246 us (ten passes after a pause; 266 where
// hundreds run back to back).  Three rows of 9k-180k int8 keys with a distance bias
// (0.33 GB): 85 us.  Some 780 instructions a warp and tile keep half
// of the issue slots busy, so what is left is latency and issue, not bytes alone.
#include <type_traits>

#include "cache_codes.cuh"
#include "cache_plan.cuh"

namespace xgr {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = 4;
constexpr int kStages = 2;
constexpr int kTileKeys = 32;

// n index (0..7) of a fragment -> key within a group of 8
template <int D>
__device__ __forceinline__ constexpr int perm(int g) {
    return D == 128 ? ((g & 1) << 2) | (g >> 1) : g ^ ((g >> 1) & 1);
}
// 16-byte chunk c of key `key` is stored at chunk c ^ swz(key)
template <int D>
__device__ __forceinline__ constexpr int swz(int key) {
    return D == 128 ? key & 7 : ((key >> 2) & 1) << 1;
}

template <int D, int MT>
struct Smem {
    static constexpr int kStageBytes = kTileKeys * D * 2;      // K then V
    alignas(16) uint8_t ring[kWarps][kStages][kStageBytes];    // after the loop: O [kWarps][R][D] fp32
    alignas(16) float sc[kWarps][kStages][4];                  // K, K, V, V scales of the two 16-key halves
    int bad[kWarps][kStages];                                  // bit h: half h lies in a page that is not there
    float m[kWarps][16 * MT], l[kWarps][16 * MT];
    float vr[kWarps][16 * MT];                                 // what O is relative to, beside 2^m
    PlanSmem<kThreads> plan;
    alignas(16) uint32_t qf[MT > 1 ? MT * (D / 16) * 128 : 4];  // query fragments (MT > 1; else in registers)
    static_assert(16 * MT * D * 4 <= kStages * kStageBytes, "the O buffer fits the rings");
};

__device__ __forceinline__ void mma16816(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, int FMT, int MT>
__global__ void __launch_bounds__(kThreads, MT == 1 ? 3 : 2) cache_attend_kernel(AttendArgs a, PlanOut po,
                                                                              int min_units) {
    constexpr int R = 16 * MT;
    constexpr int KS = D / 16;                 // k steps of Q K^T
    constexpr int NT = D / 8;                  // n tiles of P V
    constexpr int kChunks = D / 16;            // 16-byte chunks of a key
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Smem<D, MT> &sm = *reinterpret_cast<Smem<D, MT> *>(smem_raw);
    const CacheArgs &c = a.c;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const int qr = lane / 4, qc = lane % 4;    // fragment row and column group

    griddep_wait();
    griddep_launch_dependents();
    Cursor cur;
    NoParts units;
    int64_t begin, end;
    if (!plan_begin<kThreads>(a, R, min_units, sm.plan, po, units, cur, begin, end)) return;

    const uint32_t ring0 = smem_u32(&sm.ring[warp][0][0]);
    const uint32_t sc0 = smem_u32(&sm.sc[warp][0][0]);

    for (int64_t at = begin; at < end;) {
        const RowSpan row = row_span(c, cur.r, a.max_q);
        const int u1 = (int)min((int64_t)cur.units, cur.u + (end - at));
        const KeyRange sk = segment_keys(a, units, row, cur, u1, R);
        int kb = sk.lo, ke = sk.hi;

        // ---- this lane's query rows: qr + 8 i of each 16-row tile
        int lo[2 * MT], hi[2 * MT], pos[2 * MT];
        float fac[2 * MT], slope[2 * MT];
        uint32_t qf[MT][KS][4];
        int lo_min = 0x7fffffff, hi_max = 0, lo_max = 0, hi_min = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            const int ia = cur.t * R + qr + 8 * i;
            const bool valid = ia < row.n * a.G;
            const int tok = valid ? ia / a.G : 0, h = cur.g * a.G + (valid ? ia % a.G : 0);
            KeyRange k = query_keys(a, row, cur.r, tok);
            if (!valid) k = KeyRange{0, 0};
            lo[i] = k.lo;
            hi[i] = k.hi;
            pos[i] = row.len - row.n + tok;
            slope[i] = a.slopes ? a.slopes[h] * kLog2e : 0.f;
            if (valid) {
                if (k.lo < k.hi) {
                    lo_min = min(lo_min, k.lo);
                    hi_max = max(hi_max, k.hi);
                }
                lo_max = max(lo_max, k.lo);
                hi_min = min(hi_min, k.hi);
            }
            // the row's elements d = (qc + 4 j) * 16 .. + 15
            float f[D / 4];
            float top = 0.f;
            const __nv_bfloat16 *src = a.q + (int64_t)(row.t0 + tok) * a.q_stride + (int64_t)h * D;
#pragma unroll
            for (int j = 0; j < D / 64; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint4 x = valid ? *reinterpret_cast<const uint4 *>(src + (qc + 4 * j) * 16 + 8 * e)
                                          : make_uint4(0, 0, 0, 0);
                    unpack8(x, f + 16 * j + 8 * e);
                }
#pragma unroll
            for (int e = 0; e < D / 4; ++e) top = fmaxf(top, fabsf(f[e]));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int ex = query_exp(top);
            const float down = pow2i(-ex);
            fac[i] = a.scale * pow2i(ex);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                qf[i / 2][s][i & 1] = pack_f16(f[4 * s] * down, f[4 * s + 1] * down);
                qf[i / 2][s][2 + (i & 1)] = pack_f16(f[4 * s + 2] * down, f[4 * s + 3] * down);
            }
        }
        if constexpr (MT > 1) {   // the fragments of two tiles do not fit the registers
            if (warp == 0)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int s = 0; s < KS; ++s)
                        *reinterpret_cast<uint4 *>(&sm.qf[((mt * KS + s) * 32 + lane) * 4]) =
                            make_uint4(qf[mt][s][0], qf[mt][s][1], qf[mt][s][2], qf[mt][s][3]);
            __syncthreads();
        }
        lo_min = __reduce_min_sync(0xffffffffu, lo_min);
        hi_max = __reduce_max_sync(0xffffffffu, hi_max);
        lo_max = __reduce_max_sync(0xffffffffu, lo_max);
        hi_min = __reduce_min_sync(0xffffffffu, hi_min);
        kb = max(kb, lo_min);
        ke = min(ke, hi_max);

        const int kb0 = kb & ~(kTileKeys - 1);
        const int tiles = ke > kb ? (ke - kb0 + kTileKeys - 1) / kTileKeys : 0;
        const int mine = (tiles - warp + kWarps - 1) / kWarps;   // of this warp (tiles >= 0, warp < kWarps)
        const int32_t *line = c.table + (int64_t)cur.r * c.max_pages;

        const int64_t page_bytes = (int64_t)c.Hkv * c.page * D, head_off = (int64_t)cur.g * c.page * D;
        // this lane's place in 512 copied bytes (32 / kChunks keys), swizzled
        const int kl0 = lane / kChunks;
        const uint32_t lane_dst = kl0 * D + ((lane % kChunks ^ swz<D>(kl0)) << 4);
        // pages of the two halves of the warp's i-th tile (-2: no keys there, -1: no such page)
        auto ids_of = [&](int i, int *id) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int key = kb0 + (warp + kWarps * i) * kTileKeys + 16 * h;
                id[h] = -2;
                if (i < mine && key < ke) {
                    id[h] = line[key >> c.page_shift];
                    if (id[h] < 0 || id[h] >= c.n_pages) {
                        if (lane == 0) set_status(c.status, XGR_DEV_INDEX);
                        id[h] = -1;
                    }
                }
            }
        };
        // Copies the warp's i-th tile: 16 keys of a page and head are contiguous, so a half is a base and offsets
        // that do not depend on the tile.
        auto issue = [&](int i, const int *id) {
            if (i < mine) {
                const int st = i % kStages;
                const int key0 = kb0 + (warp + kWarps * i) * kTileKeys;
                const uint32_t dst = ring0 + st * Smem<D, MT>::kStageBytes + lane_dst;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int left = id[h] >= 0 ? ke - key0 - 16 * h : 0;     // keys of the half that are there
                    const int64_t off = left > 0 ? id[h] * page_bytes + head_off + ((key0 + 16 * h) & (c.page - 1)) * D : 0;
                    const uint8_t *ks = c.k + off + lane * 16, *vs = c.v + off + lane * 16;
#pragma unroll
                    for (int n = 0; n < kChunks / 2; ++n) {
                        constexpr int kKeys = 32 / kChunks;                    // keys of one copy of the warp
                        const bool in = n * kKeys + lane / kChunks < left;
                        const uint32_t to = dst + (h * kChunks / 2 + n) * 512;
                        const uint32_t at_x = D == 128 && (n & 1) ? to ^ 64u : to;
                        cp_async16_zfill(at_x, ks + n * 512, in);
                        cp_async16_zfill(at_x + kTileKeys * D, vs + n * 512, in);
                    }
                }
                if (lane < 4) {
                    const int page = lane & 1 ? id[1] : id[0];
                    const int64_t off = page >= 0 ? (int64_t)page * c.Hkv + cur.g : 0;
                    cp_async4_zfill(sc0 + (st * 4 + lane) * 4, (lane < 2 ? c.ks : c.vs) + off, page >= 0);
                }
                if (lane == 0) sm.bad[warp][st] = (id[0] == -1 ? 1 : 0) | (id[1] == -1 ? 2 : 0);
            }
            cp_async_commit();
        };

        float o[MT][NT][4];
        float m[2 * MT], l[2 * MT];
        // O is relative to 2^m / inv_vref (a power of two; 0: no scale met yet) or, where inv_vref < 0, to 2^vr (of the
        // row, in shared memory)
        float inv_vref = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
            m[i] = -INFINITY;
            l[i] = 0.f;
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[mt][n][e] = 0.f;

        int id[2];
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            ids_of(i, id);
            issue(i, id);
        }
        ids_of(kStages - 1, id);

        for (int i = 0; i < mine; ++i) {
            __syncwarp();                       // the slot about to be filled is read out
            issue(i + kStages - 1, id);
            ids_of(i + kStages, id);
            cp_async_wait_group<kStages - 1>();
            __syncwarp();
            const int st = i % kStages;
            const int key0 = kb0 + (warp + kWarps * i) * kTileKeys;
            const uint8_t *kt = sm.ring[warp][st];
            const uint8_t *vt = kt + kTileKeys * D;
            const float4 sc = *reinterpret_cast<const float4 *>(sm.sc[warp][st]);
            const int bad = sm.bad[warp][st];

            // ---- S = Q K^T on the codes
            float s[MT][4][4];
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                const int kl = nt * 8 + perm<D>(qr);
                uint32_t kw[D / 16];
#pragma unroll
                for (int j = 0; j < D / 64; ++j) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(kt + kl * D + (((qc + 4 * j) ^ swz<D>(kl)) << 4));
                    kw[4 * j] = x.x;
                    kw[4 * j + 1] = x.y;
                    kw[4 * j + 2] = x.z;
                    kw[4 * j + 3] = x.w;
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[mt][nt][e] = 0.f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t b0, b1;
                    codes_to_f16<FMT>(kw[ks], b0, b1);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        if constexpr (MT > 1) {
                            const uint4 q = *reinterpret_cast<const uint4 *>(&sm.qf[((mt * KS + ks) * 32 + lane) * 4]);
                            const uint32_t qa[4] = {q.x, q.y, q.z, q.w};
                            mma16816(s[mt][nt], qa, b0, b1);
                        } else {
                            mma16816(s[mt][nt], qf[mt][ks], b0, b1);
                        }
                    }
                }
            }

            // ---- scores in log2 units: one factor a half, or capped, biased and masked one by one
            const bool masked = key0 < lo_max || key0 + kTileKeys > hi_min || bad;
            const bool slow = masked || a.softcap > 0.f || a.slopes;
            float ksc[2] = {sc.x, sc.y}, vsc[2] = {sc.z, sc.w};
#pragma unroll
            for (int hf = 0; hf < 2; ++hf)
                if (!(ksc[hf] + vsc[hf] < INFINITY)) {   // a scale that is no number: every score of the half is NaN,
                    ksc[hf] = __int_as_float(0x7fc00000);   // and a key that is not seen still weighs 0
                    vsc[hf] = 0.f;
                }
            if (slow) {
                const float up = a.softcap * kLog2e;
                const float to2 = a.softcap > 0.f ? 2.f * kLog2e / a.softcap : kLog2e;
#pragma unroll
                for (int r2 = 0; r2 < 2 * MT; ++r2) {
                    const int mt = r2 / 2, e0 = 2 * (r2 & 1);
                    float most = 0.f;
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt) {
                        const float y = fac[r2] * ksc[nt / 2] * to2;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            s[mt][nt][e0 + e] *= y;
                            most = fmaxf(most, fabsf(s[mt][nt][e0 + e]));
                        }
                    }
                    if (a.softcap > 0.f) {
                        if (__all_sync(0xffffffffu, most <= kTanhNear)) {
#pragma unroll
                            for (int nt = 0; nt < 4; ++nt) {
                                const float2 y = tc::fmul2(tanh_near(make_float2(s[mt][nt][e0], s[mt][nt][e0 + 1])), make_float2(up, up));
                                s[mt][nt][e0] = y.x;
                                s[mt][nt][e0 + 1] = y.y;
                            }
                        } else {
#pragma unroll
                            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                                for (int e = 0; e < 2; ++e) s[mt][nt][e0 + e] = up * tanh_score(s[mt][nt][e0 + e]);
                        }
                    }
                    if (a.slopes) {
#pragma unroll
                        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int key = key0 + nt * 8 + perm<D>(2 * qc + e);
                                s[mt][nt][e0 + e] -= slope[r2] * fabsf((float)(pos[r2] - key));
                            }
                    }
                    if (masked) {
#pragma unroll
                        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int key = key0 + nt * 8 + perm<D>(2 * qc + e);
                                if (key < lo[r2] || key >= hi[r2] || (bad >> (nt / 2) & 1)) s[mt][nt][e0 + e] = -INFINITY;
                            }
                    }
                }
            }

            // ---- running maximum, weights
            float vrel[2] = {vsc[0] * inv_vref, vsc[1] * inv_vref};
            const auto near = [](float x) { return __float_as_uint(x) - __float_as_uint(0x1p-11f) <= 12u << 23; };   // 2^-11 <= x <= 2
            bool odd = false;
            if (!(near(vrel[0]) && near(vrel[1]))) {
                if (inv_vref == 0.f && (vsc[0] > 0.f || vsc[1] > 0.f)) {   // (of no scale yet)
                    const float v = fminf(fmaxf(vsc[0] > 0.f ? vsc[0] : vsc[1], 0x1p-90f), 0x1p90f);
                    inv_vref = 1.f / (64.f * __uint_as_float(__float_as_uint(v) & 0x7f800000u));
                    vrel[0] = vsc[0] * inv_vref;
                    vrel[1] = vsc[1] * inv_vref;
                }
                odd = (vsc[0] > 0.f && !near(vrel[0])) || (vsc[1] > 0.f && !near(vrel[1])) || inv_vref < 0.f;
                if (odd && inv_vref > 0.f) {
                    if (qc == 0)
#pragma unroll
                        for (int r2 = 0; r2 < 2 * MT; ++r2) sm.vr[warp][qr + 8 * r2] = m[r2] - log2_fast(inv_vref);
                    __syncwarp();
                    inv_vref = -inv_vref;
                }
            }
            float alpha[2 * MT];
            bool grew = false;
            const auto weigh = [&](auto is_odd) {   // (two bodies: a branch for each row would hold their overlap back)
                constexpr bool kOdd = decltype(is_odd)::value;
                const float logv[2] = {kOdd ? log2_fast(vsc[0]) : 0.f, kOdd ? log2_fast(vsc[1]) : 0.f};
#pragma unroll
                for (int r2 = 0; r2 < 2 * MT; ++r2) {
                    const int mt = r2 / 2, e0 = 2 * (r2 & 1);
                    float f[2], mx = -INFINITY, tw = -INFINITY;
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        f[hf] = slow ? 1.f : fac[r2] * ksc[hf] * kLog2e;
                        const float top = fmaxf(fmaxf(s[mt][2 * hf][e0], s[mt][2 * hf][e0 + 1]),
                                                fmaxf(s[mt][2 * hf + 1][e0], s[mt][2 * hf + 1][e0 + 1]));
                        mx = fmaxf(mx, top * f[hf]);
                        if constexpr (kOdd) tw = fmaxf(tw, top * f[hf] + logv[hf]);
                    }
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    const float m_new = fmaxf(m[r2], mx);
                    const float ref = m_new == -INFINITY ? 0.f : m_new;
                    alpha[r2] = exp2_fast(m[r2] - ref);      // 0 while nothing was seen
                    grew |= m_new != m[r2];
                    m[r2] = m_new;
                    const float bias = ref - kBias;
                    float t_ref = 0.f, o_alpha = alpha[r2];
                    if constexpr (kOdd) {
                        tw = fmaxf(tw, __shfl_xor_sync(0xffffffffu, tw, 1));
                        tw = fmaxf(tw, __shfl_xor_sync(0xffffffffu, tw, 2));
                        const float t_old = sm.vr[warp][qr + 8 * r2], t_new = fmaxf(t_old, tw);
                        t_ref = t_new == -INFINITY ? 0.f : t_new;
                        o_alpha = exp2_fast(t_old - t_ref);
                        grew |= t_new != t_old;
                        __syncwarp();
                        if (qc == 0) sm.vr[warp][qr + 8 * r2] = t_new;
                        __syncwarp();
                    }
                    float sum = 0.f;
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float x = s[mt][nt][e0 + e];
                            const float p = exp2_fast(fmaf(x, f[nt / 2], -bias));
                            sum += p;
                            if constexpr (kOdd) s[mt][nt][e0 + e] = exp2_fast(fmaf(x, f[nt / 2], logv[nt / 2] - t_ref + kBias));
                            else s[mt][nt][e0 + e] = p * vrel[nt / 2];
                        }
                    l[r2] = l[r2] * alpha[r2] + sum;
                    alpha[r2] = o_alpha;                     // (from here on O's)
                }
            };
            if (!odd) weigh(std::false_type{});
            else weigh(std::true_type{});
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int r2 = 0; r2 < 2 * MT; ++r2)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        o[r2 / 2][n][2 * (r2 & 1)] *= alpha[r2];
                        o[r2 / 2][n][2 * (r2 & 1) + 1] *= alpha[r2];
                    }
            }

            // ---- O += W V on the codes
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                uint32_t pa[MT][4];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    pa[mt][0] = pack_f16(s[mt][2 * u][0], s[mt][2 * u][1]);
                    pa[mt][1] = pack_f16(s[mt][2 * u][2], s[mt][2 * u][3]);
                    pa[mt][2] = pack_f16(s[mt][2 * u + 1][0], s[mt][2 * u + 1][1]);
                    pa[mt][3] = pack_f16(s[mt][2 * u + 1][2], s[mt][2 * u + 1][3]);
                }
                uint32_t vw[4][D / 32];   // the lane's dims of its four keys
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int kl = 16 * u + (k / 2) * 8 + perm<D>(2 * qc + (k & 1));
                    if constexpr (D == 128) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(vt + kl * D + ((perm<D>(qr) ^ swz<D>(kl)) << 4));
                        vw[k][0] = x.x;
                        vw[k][1] = x.y;
                        vw[k][2] = x.z;
                        vw[k][3] = x.w;
                    } else {
                        const uint2 x = *reinterpret_cast<const uint2 *>(vt + kl * D + (((qr >> 1) ^ swz<D>(kl)) << 4) + (qr & 1) * 8);
                        vw[k][0] = x.x;
                        vw[k][1] = x.y;
                    }
                }
#pragma unroll
                for (int wd = 0; wd < D / 32; ++wd) {
                    uint32_t b0[4], b1[4];
                    codes_to_f16<FMT>(__byte_perm(vw[0][wd], vw[1][wd], 0x5140), b0[0], b0[1]);
                    codes_to_f16<FMT>(__byte_perm(vw[0][wd], vw[1][wd], 0x7362), b0[2], b0[3]);
                    codes_to_f16<FMT>(__byte_perm(vw[2][wd], vw[3][wd], 0x5140), b1[0], b1[1]);
                    codes_to_f16<FMT>(__byte_perm(vw[2][wd], vw[3][wd], 0x7362), b1[2], b1[3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) mma16816(o[mt][4 * wd + e], pa[mt], b0[e], b1[e]);
                }
            }
        }

        // ---- join the warps
        cp_async_wait_all();
        __syncthreads();
        float *ob = reinterpret_cast<float *>(smem_raw) + warp * R * D;   // over the rings
#pragma unroll
        for (int r2 = 0; r2 < 2 * MT; ++r2) {
            float t = l[r2];
            t += __shfl_xor_sync(0xffffffffu, t, 1);
            t += __shfl_xor_sync(0xffffffffu, t, 2);
            const int rr = qr + 8 * r2;
            if (qc == 0) {
                sm.m[warp][rr] = m[r2];
                sm.l[warp][rr] = t;
                // (no scale passes 2^128, so neither does this)
                sm.vr[warp][rr] = m[r2] == -INFINITY || inv_vref == 0.f ? 0.f
                                  : inv_vref > 0.f ? 1.f / inv_vref : exp2f(fminf(sm.vr[warp][rr] - m[r2], 0x1.fffffep6f));
            }
            // lane (qr, qc) holds, for each n tile, dims of n index 2 qc and 2 qc + 1
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int d0 = D == 128 ? perm<D>(2 * qc + e) * 16 : (2 * qc + e) * 8;
#pragma unroll
                for (int n = 0; n < NT; n += 4)
                    *reinterpret_cast<float4 *>(ob + rr * D + d0 + n) =
                        make_float4(o[r2 / 2][n][2 * (r2 & 1) + e], o[r2 / 2][n + 1][2 * (r2 & 1) + e],
                                    o[r2 / 2][n + 2][2 * (r2 & 1) + e], o[r2 / 2][n + 3][2 * (r2 & 1) + e]);
            }
        }
        __syncthreads();
        const bool all = cur.u == 0 && u1 == cur.units;   // the whole segment was this block's
        const int slot = cur.u == 0 ? 1 : 0;
        const float *obase = reinterpret_cast<const float *>(smem_raw);
        // a thread a row: the warps' factors, relative to the largest (in place of m), the factor that is left of all of
        // them and the row's sum (in place of l): in this order no product leaves fp32's range where the result does not
        const int64_t part = ((int64_t)blockIdx.x * 2 + slot) * R;
        auto out_row = [&](int ia) { return (int64_t)(row.t0 + ia / a.G) * a.Hq + cur.g * a.G + ia % a.G; };
        if (tid < R) {
            float mm = -INFINITY;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) mm = fmaxf(mm, sm.m[k][tid]);
            const float ref = mm == -INFINITY ? 0.f : mm;
            float f[kWarps], lsum = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                f[k] = exp2_fast(sm.m[k][tid] - ref);
                lsum += sm.l[k][tid] * f[k];
            }
            float most = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                f[k] *= sm.vr[k][tid];
                most = fmaxf(most, f[k]);
            }
#pragma unroll
            for (int k = 0; k < kWarps; ++k) sm.m[k][tid] = most > 0.f ? f[k] / most : 0.f;
            const bool huge = !all && most > 0x1p80f;   // (sums of such values would overflow: the part's mean instead)
            sm.l[0][tid] = !all && !huge ? 1.f : lsum == 0.f ? 0.f : 1.f / lsum;
            sm.l[1][tid] = most;
            if (huge) {
                mm += log2f(lsum);
                lsum = 1.f;
            }
            const int ia = cur.t * R + tid;
            if (ia < row.n * a.G) {
                if (all) a.lse[out_row(ia)] = lsum == 0.f ? -INFINITY : (ref - kBias + log2f(lsum)) * kLn2;
                else po.ml[part + tid] = make_float2(mm, lsum);
            }
        }
        __syncthreads();
        for (int idx = tid; idx < R * D / 8; idx += kThreads) {
            const int rr = idx / (D / 8), d = (idx % (D / 8)) * 8;
            const int ia = cur.t * R + rr;
            if (ia >= row.n * a.G) break;                          // (rows ascend)
            float x[8] = {};
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float fv = sm.m[k][rr];
                const float4 y0 = *reinterpret_cast<const float4 *>(obase + (k * R + rr) * D + d);
                const float4 y1 = *reinterpret_cast<const float4 *>(obase + (k * R + rr) * D + d + 4);
                x[0] += y0.x * fv; x[1] += y0.y * fv; x[2] += y0.z * fv; x[3] += y0.w * fv;
                x[4] += y1.x * fv; x[5] += y1.y * fv; x[6] += y1.z * fv; x[7] += y1.w * fv;
            }
            const float scale = sm.l[0][rr], most = sm.l[1][rr];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = x[e] * scale * most;
            if (all) {
                uint4 pk;
                __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&pk);
#pragma unroll
                for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(x[2 * e], x[2 * e + 1]);
                *reinterpret_cast<uint4 *>(a.out + out_row(ia) * D + d) = pk;
            } else {
                float4 *dst = reinterpret_cast<float4 *>(po.o + (part + rr) * D + d);
                dst[0] = make_float4(x[0], x[1], x[2], x[3]);
                dst[1] = make_float4(x[4], x[5], x[6], x[7]);
            }
        }
        __syncthreads();   // the rings and (m, l) are free for the next segment
        at += u1 - cur.u;
        if (at < end) plan_next(a, units, R, cur);
        if (cur.r >= c.n_rows) break;
    }
}

// Folds the parts of the segments that were cut.  Column c of the grid looks at
// the segment that CTA c begins in the middle of, and takes it if c is the first
// such CTA; a row of the tile is folded by WPR warps (one where parts are few,
// four, each every fourth part, where a long row may have many).  O and l of
// part k count 2^(m_k - max m).
template <int D, int WPR>
__global__ void __launch_bounds__(128) cache_join_kernel(AttendArgs a, int R, PlanOut po, float bias) {
    constexpr int N = D / 32;                       // dims of a lane
    __shared__ float acc[4][D];
    __shared__ float red[4];
    griddep_wait();
    griddep_launch_dependents();
    const Cursor cur = po.first[blockIdx.x];
    if (cur.u == 0) return;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    auto inside = [&](int c) {                      // CTA c begins in the middle of the same segment
        if (c >= (int)gridDim.x) return false;
        const Cursor f = po.first[c];
        return f.u > 0 && f.r == cur.r && f.t == cur.t && f.g == cur.g;
    };
    const int c0 = blockIdx.x - 1;                  // (CTA 0 begins at a segment's start)
    if (inside(c0)) return;
    int n = 2;                                      // parts: CTA c0's, this one's, those of the CTAs after it
    for (;; n += 32) {
        const uint32_t more = __ballot_sync(0xffffffffu, inside(c0 + n + lane));
        if (more != 0xffffffffu) {
            n += __ffs(~more) - 1;
            break;
        }
    }
    const int rr = blockIdx.y * (4 / WPR) + warp / WPR, sub = warp % WPR;
    const RowSpan row = row_span(a.c, cur.r, a.max_q);
    const int ia = cur.t * R + rr;
    if (ia >= row.n * a.G) return;                  // (of all warps of a row)
    auto part = [&](int k) { return ((int64_t)(c0 + k) * 2 + (k == 0 ? 1 : 0)) * R + rr; };
    float m = -INFINITY;
    for (int k = lane; k < n; k += 32) m = fmaxf(m, po.ml[part(k)].x);
    m = warp_max(m);
    const float ref = m == -INFINITY ? 0.f : m;
    float l = 0.f, x[N];
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = 0.f;
#pragma unroll 4
    for (int k = sub; k < n; k += WPR) {
        const int64_t pi = part(k);
        const float2 ml = po.ml[pi];
        const float f = exp2_fast(ml.x - ref);
        l += f * ml.y;
        if constexpr (N == 4) {
            const float4 y = reinterpret_cast<const float4 *>(po.o + pi * D)[lane];
            x[0] += f * y.x; x[1] += f * y.y; x[2] += f * y.z; x[3] += f * y.w;
        } else {
            const float2 y = reinterpret_cast<const float2 *>(po.o + pi * D)[lane];
            x[0] += f * y.x; x[1] += f * y.y;
        }
    }
    if constexpr (WPR > 1) {
#pragma unroll
        for (int e = 0; e < N; ++e) acc[warp][lane * N + e] = x[e];
        if (lane == 0) red[warp] = l;
        __syncthreads();
        if (warp > 0) return;
        l = red[0] + red[1] + red[2] + red[3];
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int d = lane * N + e;
            x[e] = acc[0][d] + acc[1][d] + acc[2][d] + acc[3][d];
        }
    }
    const int64_t oi = (int64_t)(row.t0 + ia / a.G) * a.Hq + cur.g * a.G + ia % a.G;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    __nv_bfloat162 *dst = reinterpret_cast<__nv_bfloat162 *>(a.out + oi * D + lane * N);
#pragma unroll
    for (int e = 0; e < N / 2; ++e) dst[e] = __floats2bfloat162_rn(x[2 * e] * inv, x[2 * e + 1] * inv);
    if (lane == 0) a.lse[oi] = l == 0.f ? -INFINITY : (ref - bias + log2f(l)) * kLn2;
}

// The lowest key that the queries of each tile see (the row's length where they
// see none), a warp a tile: with documents in a row it may lie far above 0, and
// the work has to be shared out without the keys below it.
__global__ void __launch_bounds__(128) cache_tile_lo_kernel(AttendArgs a, int R, int64_t slots) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t slot = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
    if (slot >= slots) return;
    int r;
    int64_t t;
    const RowSpan row = slot_tile(a, R, slot, r, t);
    if (t < 0 || t >= row_tiles(a, row, R)) return;
    const int i0 = (int)(t * R / a.G), i1 = (int)((min((t + 1) * R, (int64_t)row.n * a.G) - 1) / a.G);
    int low = row.len;
    for (int i = i0 + (int)(threadIdx.x % 32); i <= i1; i += 32) {
        const KeyRange q = query_keys(a, row, r, i);
        if (q.lo < q.hi) low = min(low, q.lo);
    }
    low = __reduce_min_sync(0xffffffffu, low);
    if (threadIdx.x % 32 == 0) a.tile_lo[slot] = low;
}

constexpr int kSmallCtas = 3 * kSms;         // 16-row tiles: three CTAs an SM
constexpr int kWideCtas = 2 * kSms;          // 32-row tiles: two
constexpr int kTcRows256 = 256;              // tcgen05 tiles: one
// Fewest units a CTA takes: one row of 9300 keys takes 24.1 us with 4, 24.9 with 2, 26.4 with 8; four rows of 1000 to
// 2000 keys 20.7, 22.1, 25.7.
constexpr int kMinUnits = 4;
// A 256-row segment's rows and result cost about as much as three units of its keys, and as two where a cap makes keys
// dearer.  7 and 12 packed chunks of 61 to 1000 tokens: without a cap 188 and 318 us with 3, 201 and 333 with 2 (7: 224
// with 1); with a cap 218 and 367 with 2, 224 and 378 with 3 (7: 241 with 1).  Equal chunks differ by less than 2%.
constexpr int kTcLead = 3;
constexpr int kTcLeadCapped = 2;
// Rows of at most this many units are not cut and need no join: 200 rows of 300 to 800 keys 86 us, cut and joined 93.
constexpr int kWholeUnits = 8;

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

struct WsLayout {
    size_t first, o, ml, lo, total;
};
WsLayout ws_layout(int D, int G, int n_rows, int n_tokens) {
    WsLayout w{};
    w.first = 0;
    w.o = up256((size_t)kSmallCtas * sizeof(Cursor));
    const size_t parts = 2 * std::max<size_t>({(size_t)kSmallCtas * 16, (size_t)kWideCtas * 32, (size_t)kSms * kTcRows256});
    w.ml = w.o + up256(parts * D * 4);
    w.lo = w.ml + up256(parts * 8);
    w.total = w.lo + up256((size_t)((int64_t)n_tokens * G / 16 + n_rows) * 4);   // (16: the lowest tile)
    return w;
}

template <int D, int FMT, int MT>
cudaError_t launch_small(const AttendArgs &a, const PlanOut &po, int ctas, int min_units, cudaStream_t s) {
    const size_t smem = sizeof(Smem<D, MT>);
    static bool ready[kMaxDevices] = {};   // the attribute is set on the first (uncaptured) launch of a device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!ready[dev]) {
        e = cudaFuncSetAttribute(cache_attend_kernel<D, FMT, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        ready[dev] = true;
    }
    return launch_pdl(cache_attend_kernel<D, FMT, MT>, dim3(ctas), dim3(kThreads), smem, s, a, po, min_units);
}

template <int D, int FMT>
cudaError_t launch_kind(const AttendArgs &a, int R, const PlanOut &po, int ctas, int min_units, cudaStream_t s) {
    if (R == 16) return launch_small<D, FMT, 1>(a, po, ctas, min_units, s);
    if (R == 32) return launch_small<D, FMT, 2>(a, po, ctas, min_units, s);
    return launch_attend_tc(a, po, ctas, min_units, s);
}

}  // namespace

size_t attend_ws_bytes(int D, int G, int n_rows, int n_tokens) { return ws_layout(D, G, n_rows, n_tokens).total; }

cudaError_t launch_cache_attend(const AttendArgs &in, cudaStream_t s) {
    AttendArgs a = in;
    const CacheArgs &c = a.c;
    a.whole = (int64_t)c.max_pages * c.page <= kWholeUnits * kUnitKeys;
    // 16 or 32 query rows a tile on mma.sync while no row has more; else 256 a tile on tcgen05.  Measured on 64 rows
    // over 8.4k-10.2k keys, no cap: 16 query rows 230 us in 16-row tiles, 327 in 32-row ones; 32 query rows 337 us in
    // 32-row tiles, 588 on tcgen05; 64 query rows 639 us in two 32-row tiles, 593 on tcgen05.  (All rows of a call go one
    // way: a chunk among single tokens takes them along to the 256-row tiles.)
    const int64_t most = (int64_t)a.max_q * a.G;
    const int R = most <= 16 ? 16 : most <= 32 ? 32 : kTcRows256;
    const int cap = R == 16 ? kSmallCtas : R == 32 ? kWideCtas : kSms;
    a.lead = R != kTcRows256 || a.whole ? 0 : a.softcap > 0.f ? kTcLeadCapped : kTcLead;
    const int min_units = a.whole ? 1 : kMinUnits + a.lead;
    // no more CTAs than there can be shares of the line
    const int64_t segs = (((int64_t)c.n_tokens * a.G + R - 1) / R + c.n_rows) * c.Hkv;
    const int64_t row_units = a.whole ? 1 : (int64_t)c.max_pages * c.page / kUnitKeys + 2 + a.lead;
    const int ctas = (int)std::min<int64_t>(cap, (segs * row_units + min_units - 1) / min_units);
    const WsLayout l = ws_layout(c.D, a.G, c.n_rows, c.n_tokens);
    a.tile_lo = reinterpret_cast<int32_t *>(a.ws + l.lo);
    PlanOut po{};
    if (!a.whole) {
        po.first = reinterpret_cast<Cursor *>(a.ws + l.first);
        po.o = reinterpret_cast<float *>(a.ws + l.o);
        po.ml = reinterpret_cast<float2 *>(a.ws + l.ml);
    }
    cudaError_t e;
    if (a.first) {
        const int64_t slots = (int64_t)c.n_tokens * a.G / R + c.n_rows;
        e = launch_pdl(cache_tile_lo_kernel, dim3((unsigned)((slots + 3) / 4)), dim3(128), 0, s, a, R, slots);
        if (e != cudaSuccess) return e;
    }
    if (c.D == 128)
        e = c.fmt == XGR_CACHE_E4M3 ? launch_kind<128, XGR_CACHE_E4M3>(a, R, po, ctas, min_units, s)
                                    : launch_kind<128, XGR_CACHE_INT8>(a, R, po, ctas, min_units, s);
    else
        e = c.fmt == XGR_CACHE_E4M3 ? launch_kind<64, XGR_CACHE_E4M3>(a, R, po, ctas, min_units, s)
                                    : launch_kind<64, XGR_CACHE_INT8>(a, R, po, ctas, min_units, s);
    if (e != cudaSuccess || a.whole) return e;
    const float bias = R == kTcRows256 ? kTcBias : kBias;
    if (R == kTcRows256) {
        const dim3 grid(ctas, R / 4);
        return c.D == 128 ? launch_pdl(cache_join_kernel<128, 1>, grid, dim3(128), 0, s, a, R, po, bias)
                          : launch_pdl(cache_join_kernel<64, 1>, grid, dim3(128), 0, s, a, R, po, bias);
    }
    const dim3 grid(ctas, R);
    return c.D == 128 ? launch_pdl(cache_join_kernel<128, 4>, grid, dim3(128), 0, s, a, R, po, bias)
                      : launch_pdl(cache_join_kernel<64, 4>, grid, dim3(128), 0, s, a, R, po, bias);
}

}  // namespace xgr
