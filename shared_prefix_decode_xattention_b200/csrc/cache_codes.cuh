// cache_codes.cuh -- the cache's 8-bit codes as fp16 (internal): every code of
// either format is an fp16 number, so the conversion does not round.
#pragma once

#include "cache.cuh"

namespace xgr {

// cp.async of 16 or 4 bytes, zeros where `in` is false (src is not read then)
__device__ __forceinline__ void cp_async16_zfill(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async4_zfill(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0)
                 : "memory");
}

// the four codes of a word -> two fp16 pairs (elements 0, 1 and 2, 3)
template <int FMT>
__device__ __forceinline__ void codes_to_f16(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if constexpr (FMT == XGR_CACHE_E4M3) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {   // 1024 + (code + 128) is an fp16 number with the byte as its low bits
        const uint32_t u = w ^ 0x80808080u;
        const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));   // 1152
        const uint32_t l = __byte_perm(u, 0x64646464u, 0x4140), h = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 a = __hsub2(*reinterpret_cast<const __half2 *>(&l), off);
        const __half2 b = __hsub2(*reinterpret_cast<const __half2 *>(&h), off);
        lo = *reinterpret_cast<const uint32_t *>(&a);
        hi = *reinterpret_cast<const uint32_t *>(&b);
    }
}

__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Exponent e of the power of two that brings a query row whose largest
// magnitude is `top` near 1 (0 for a row of zeros, or one that is not finite).
__device__ __forceinline__ int query_exp(float top) {
    const int ex = (int)(__float_as_uint(top) >> 23) - 127;
    return top > 0.f && top < INFINITY ? min(max(ex, -126), 126) : 0;
}
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((127 + e) << 23); }   // -126 <= e <= 127

}  // namespace xgr
