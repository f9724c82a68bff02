// cache_store.cu -- xgr_cache_store: new tokens into the paged 8-bit cache.
//
// For each page, kv head and side (K or V) that gets new tokens: the largest
// magnitude of the new values picks the page's scale, the smallest power of
// two s with max |x| <= s * qmax; codes are x / s rounded to nearest.  With
// powers of two the division is exact, so the one rounding is the code's, and
// when a later token makes the scale grow, the older codes move by a power of
// two (exact but for what falls below the code's last place).
//
// A group of W warps takes one (page, kv head, side): the page's tokens sit in
// its registers between the maximum and the rounding, so the values are read
// once.  W is set by the page's size, 64 values a thread: wide loads (two
// 16-byte reads, one 16-byte write a thread and step) and enough of them in
// flight.  Bound by HBM: 2 bytes in, 1 byte out a value; 590k tokens of 4 heads (1.83
// GB) in 308 us, 5.9 TB/s, ten passes after a pause; 328 where hundreds run back to back.
#include <cuda_fp8.h>

#include "cache.cuh"

namespace xgr {

namespace {

constexpr int kThreads = 256;

// slot base of row r: no row's touched pages exceed the gap to the next base
// (n tokens touch at most ceil((n - 1) / page) + 1 pages, the gap is at least
// floor(n / page) + 2)
__device__ __forceinline__ int slot_base(const CacheArgs &c, int r) { return (c.cu[r] >> c.page_shift) + 2 * r; }

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

// |x| <= 127, by the choice of the scale: adding 1.5 * 2^23 rounds to the nearest
// whole number, ties to even, and leaves it in the low byte (the conversion
// instruction runs at an eighth of the rate: 355 against 306 us for 590k tokens in short runs)
__device__ __forceinline__ uint32_t int8x4(float a, float b, float c, float d) {
    auto q = [](float x) { return __float_as_uint(x + 12582912.f); };
    return __byte_perm(__byte_perm(q(a), q(b), 0x0040), __byte_perm(q(c), q(d), 0x0040), 0x5410);
}

template <int FMT>
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
    if constexpr (FMT == XGR_CACHE_E4M3) return e4m3x4(a, b, c, d);
    else return int8x4(a, b, c, d);
}

template <int FMT>
__device__ __forceinline__ float code_value(uint32_t byte) {
    if constexpr (FMT == XGR_CACHE_E4M3) {
        const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3);
        return __half2float(__half(h));
    } else {
        return (float)(int8_t)byte;
    }
}

// Exponent of the smallest power of two s >= 2^-126 with x <= s * qmax, x given
// as its bf16 bits (finite, >= 0).  qmax = 448 = 1.75 * 2^8 or 127 = 1.984375 * 2^6.
template <int FMT>
__device__ __forceinline__ int scale_exp(uint32_t bits) {
    constexpr uint32_t kFrac = FMT == XGR_CACHE_E4M3 ? 0x60u : 0x7eu;
    constexpr int kExp = FMT == XGR_CACHE_E4M3 ? 8 : 6;
    const int e = (int)(bits >> 7) - 127 - kExp + ((bits & 0x7fu) > kFrac);
    return max(e, -126);
}

template <int D, int W, int NI, int FMT>
__global__ void __launch_bounds__(kThreads) cache_store_kernel(StoreArgs a, int n_slots) {
    constexpr int kGroups = 8 / W;           // (page, head) pairs of a block
    constexpr int kLanes = 32 * W;
    constexpr int kChunks = D / 16;          // 16-value chunks of a token
    __shared__ uint32_t part[8];
    griddep_wait();
    griddep_launch_dependents();
    const CacheArgs &c = a.c;
    const int group = threadIdx.x / kLanes, tid = threadIdx.x % kLanes;
    const int64_t unit = (int64_t)blockIdx.x * kGroups + group;
    const int slot = (int)(unit / c.Hkv), g = (int)(unit % c.Hkv);
    const bool v_side = blockIdx.y != 0;
    if (!v_side && blockIdx.x <= c.n_rows / kThreads) {   // (there are more threads than rows)
        const int i = blockIdx.x * kThreads + threadIdx.x;
        if (i < c.n_rows && out_of_order(c, cu_pair(c, i))) set_status(c.status, XGR_DEV_INDEX);
    }
    if (slot >= n_slots) return;

    // the row of this slot: slots are the rows themselves when no row has two
    // tokens, else found among the rows' slot bases
    int r = slot, j = 0, below = 0, above = 0x7fffffff;   // (the largest base passed on the way that is below, the least above)
    if (a.max_n > 1) {
        int lo = 0, hi = c.n_rows - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2, base = slot_base(c, mid);
            if (base <= slot) {
                lo = mid;
                below = max(below, base);
            } else {
                hi = mid - 1;
                above = min(above, base);
            }
        }
        r = lo;
        j = slot - slot_base(c, r);
        if (j < 0) return;
    }
    const RowSpan row = row_span(c, r, a.max_n);
    if (row.n == 0) return;
    // where d_cu is out of order: the search for the row's other slots takes the same way, or the row is left out whole
    if (below > slot - j || above < ((row.t0 + row.n) >> c.page_shift) + 2 * (r + 1)) return;
    const int start = row.len - row.n;
    const int p = (start >> c.page_shift) + j;
    if (p > (row.len - 1) >> c.page_shift) return;
    const int id = c.table[(int64_t)r * c.max_pages + p];
    if (id < 0 || id >= c.n_pages) {
        if (tid == 0) set_status(c.status, XGR_DEV_INDEX);
        return;
    }
    const int pos0 = p << c.page_shift;
    const int t_lo = max(start - pos0, 0), t_hi = min(row.len - pos0, c.page);   // the page's new tokens

    const __nv_bfloat16 *src = (v_side ? a.v : a.k) + (int64_t)g * D;
    const int64_t tok0 = (int64_t)row.t0 + pos0 - start;                          // packed token of slot 0
    uint4 x[NI][2];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int ch = i * kLanes + tid, t = ch / kChunks;
        if (t >= t_lo && t < t_hi) {
            const uint4 *s = reinterpret_cast<const uint4 *>(src + (tok0 + t) * a.stride + (ch % kChunks) * 16);
            x[i][0] = __ldcs(s);
            x[i][1] = __ldcs(s + 1);
        } else {
            x[i][0] = x[i][1] = make_uint4(0, 0, 0, 0);
        }
    }
    float *scale_at = (v_side ? c.vs : c.ks) + (int64_t)id * c.Hkv + g;
    const float was = t_lo > 0 ? *scale_at : 0.f;   // older tokens in the page hold its scale up
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {   // magnitudes of bf16 pairs compare as whole numbers, NaN and infinity above all
            const uint32_t w[4] = {x[i][h].x, x[i][h].y, x[i][h].z, x[i][h].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) top = __vmaxu2(top, w[e] & 0x7fff7fffu);
        }
    top = max(top & 0xffffu, top >> 16);
    top = __reduce_max_sync(0xffffffffu, top);
    if constexpr (W > 1) {
        if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = top;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + group), "n"(kLanes) : "memory");
#pragma unroll
        for (int w = 0; w < W; ++w) top = max(top, part[group * W + w]);
    }
    const bool poison = top >= 0x7f80u;
    const float want = __int_as_float((scale_exp<FMT>(poison ? 0u : top) + 127) << 23);
    const bool sick = poison || was != was;   // a NaN scale stays until the page is begun anew
    const float scale = sick ? __int_as_float(0x7fc00000) : fmaxf(want, was);
    const bool grown = t_lo > 0 && scale != was && !(was != was);
    // a power of two (all this kernel writes) divides exactly by multiplying with its inverse
    const bool pow2 = sick || (__float_as_uint(scale) & 0x7fffffu) == 0;
    const float inv = 1.f / scale;
    auto quot = [&](float v) { return sick ? 0.f : pow2 ? v * inv : __fdiv_rn(v, scale); };
    if (tid == 0) *scale_at = scale;

    uint8_t *dst = (v_side ? c.v : c.k) + ((int64_t)id * c.Hkv + g) * ((int64_t)c.page * D);
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int ch = i * kLanes + tid, t = ch / kChunks;
        uint4 *d = reinterpret_cast<uint4 *>(dst + ch * 16);
        if (t >= t_lo && t < t_hi) {
            uint32_t o[4];
            if (pow2) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float f[8];
                    unpack8(x[i][h], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] *= inv;
                    o[2 * h] = pack4<FMT>(f[0], f[1], f[2], f[3]);
                    o[2 * h + 1] = pack4<FMT>(f[4], f[5], f[6], f[7]);
                }
                if (sick) o[0] = o[1] = o[2] = o[3] = 0;
            } else {   // a larger scale of older tokens, from another quantiser
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float f[8];
                    unpack8(x[i][h], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = __fdiv_rn(f[e], scale);
                    o[2 * h] = pack4<FMT>(f[0], f[1], f[2], f[3]);
                    o[2 * h + 1] = pack4<FMT>(f[4], f[5], f[6], f[7]);
                }
            }
            *d = make_uint4(o[0], o[1], o[2], o[3]);
        } else if (t < t_lo && grown) {
            const uint4 old = *d;
            const uint32_t w[4] = {old.x, old.y, old.z, old.w};
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                o[e] = pack4<FMT>(quot(code_value<FMT>(w[e] & 255u) * was), quot(code_value<FMT>((w[e] >> 8) & 255u) * was),
                                  quot(code_value<FMT>((w[e] >> 16) & 255u) * was), quot(code_value<FMT>(w[e] >> 24) * was));
            *d = make_uint4(o[0], o[1], o[2], o[3]);
        }
    }
}

template <int D, int W, int NI>
cudaError_t launch_w(const StoreArgs &a, cudaStream_t s) {
    const int64_t slots = a.max_n > 1 ? a.c.n_tokens / a.c.page + 2ll * a.c.n_rows : a.c.n_rows;
    const int64_t blocks = (slots * a.c.Hkv * W + 7) / 8;
    if (blocks > 0x7fffffffll || slots > 0x7fffffffll) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks, 2);
    return a.c.fmt == XGR_CACHE_E4M3
               ? launch_pdl(cache_store_kernel<D, W, NI, XGR_CACHE_E4M3>, grid, dim3(kThreads), 0, s, a, (int)slots)
               : launch_pdl(cache_store_kernel<D, W, NI, XGR_CACHE_INT8>, grid, dim3(kThreads), 0, s, a, (int)slots);
}

}  // namespace

cudaError_t launch_cache_store(const StoreArgs &a, cudaStream_t s) {
    if (a.c.D == 128) switch (a.c.page) {
        case 16: return launch_w<128, 1, 4>(a, s);
        case 32: return launch_w<128, 2, 4>(a, s);
        case 64: return launch_w<128, 4, 4>(a, s);
        case 128: return launch_w<128, 8, 4>(a, s);
    }
    if (a.c.D == 64) switch (a.c.page) {
        case 16: return launch_w<64, 1, 2>(a, s);
        case 32: return launch_w<64, 1, 4>(a, s);
        case 64: return launch_w<64, 2, 4>(a, s);
        case 128: return launch_w<64, 4, 4>(a, s);
    }
    return cudaErrorInvalidValue;
}

}  // namespace xgr
