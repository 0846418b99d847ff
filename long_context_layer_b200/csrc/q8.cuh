// The 8-bit cache: formats, block scales, and conversions (included by the q8 translation units).
//
// A block is the 16 tokens of one (page, KV head) of K or of V.  Its scale is 2^e, e the smallest integer
// >= -100 with max|x| <= QMAX * 2^e.  A power of two instead of max|x| / QMAX costs int8 up to one bit of
// its step (half a bit on average) and e4m3 nothing, and buys: scaling is exact (no rounding but the one
// to 8 bits), the stored values are exact in bf16, fp16 and fp32, and a block whose scale grows as tokens
// are appended re-rounds its older values to steps that at least double, so all their roundings together
// stay below half a step * (1 + 1/2 + 1/4 + ...) = one step (e4m3 values move exactly, subnormals aside).
#pragma once

#include "common.cuh"

#include <cuda_fp16.h>
#include <cuda_fp8.h>

namespace delta {

enum : int { kE4M3 = 0, kInt8 = 1 };

// Bits of the block scale for a largest magnitude of `amax` (its float bits); NaN when it is not finite.
template <int FMT>
__device__ __forceinline__ uint32_t block_scale_bits(uint32_t amax) {
    if (amax >= 0x7f800000u) return 0x7fc00000u;
    const int x = int(amax >> 23) - 127;             // amax in [2^x, 2^(x+1)); -127: zero or subnormal
    const uint32_t mant = amax & 0x7fffffu;
    // 448 = 1.75 * 2^8, 127 = 1.984375 * 2^6: one exponent more when amax's mantissa is above QMAX's
    int e = FMT == kE4M3 ? x - 8 + (mant > 0x600000u ? 1 : 0) : x - 6 + (mant > 0x7e0000u ? 1 : 0);
    e = max(e, -100);
    return uint32_t(e + 127) << 23;
}
// 1 / scale of a finite scale > 0.  Exact for the powers of two that block_scale_bits makes; a block written elsewhere
// may hold any other scale, and then the quotient x / scale is rounded twice in fp32 before its rounding to 8 bits.
__device__ __forceinline__ float scale_inverse(uint32_t bits) {
    const uint32_t e = bits >> 23;
    if ((bits & 0x7fffffu) == 0u && e >= 1u && e <= 252u) return __uint_as_float((254u << 23) - bits);
    return 1.0f / __uint_as_float(bits);
}
__device__ __forceinline__ bool scale_finite(uint32_t bits) { return bits < 0x7f800000u; }

// Two scaled values to two payload bytes (low byte first), rounded to nearest even.
template <int FMT>
__device__ __forceinline__ uint32_t pack8x2(float a, float b) {
    if constexpr (FMT == kE4M3) {
        return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    } else {
        return (uint32_t(__float2int_rn(a)) & 0xffu) | ((uint32_t(__float2int_rn(b)) & 0xffu) << 8);
    }
}
// Two payload bytes to the numbers they hold (unscaled).
template <int FMT>
__device__ __forceinline__ float2 unpack8x2(uint32_t w) {
    if constexpr (FMT == kE4M3) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w & 0xffffu), __NV_E4M3);
        return __half22float2(__half2(h));
    } else {
        return make_float2(float(int8_t(w & 0xffu)), float(int8_t((w >> 8) & 0xffu)));
    }
}
template <int FMT>
__device__ __forceinline__ uint32_t pack8x4(float a, float b, float c, float d) {
    return pack8x2<FMT>(a, b) | (pack8x2<FMT>(c, d) << 16);
}

// 16 bytes of T.
template <typename T>
struct Raw16;
template <>
struct Raw16<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void get(uint4 w, float (&x)[8]) {
        unpack_bf16x2(w.x, x[0], x[1]);
        unpack_bf16x2(w.y, x[2], x[3]);
        unpack_bf16x2(w.z, x[4], x[5]);
        unpack_bf16x2(w.w, x[6], x[7]);
    }
    // Running largest magnitude as bits (NaN > infinity > finite), two halfwords at once; top() is one float's.
    static __device__ __forceinline__ uint32_t more(uint32_t m, uint4 w) {
        m = __vimax3_u16x2(m, w.x & 0x7fff7fffu, w.y & 0x7fff7fffu);
        return __vimax3_u16x2(m, w.z & 0x7fff7fffu, w.w & 0x7fff7fffu);
    }
    static __device__ __forceinline__ uint32_t top(uint32_t m) { return max(m << 16, m & 0xffff0000u); }
};
template <>
struct Raw16<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ uint32_t more(uint32_t m, uint4 w) {
        m = __vimax3_u32(m, w.x & 0x7fffffffu, w.y & 0x7fffffffu);
        return __vimax3_u32(m, w.z & 0x7fffffffu, w.w & 0x7fffffffu);
    }
    static __device__ __forceinline__ uint32_t top(uint32_t m) { return m; }
    static __device__ __forceinline__ void get(uint4 w, float (&x)[4]) {
        x[0] = __uint_as_float(w.x);
        x[1] = __uint_as_float(w.y);
        x[2] = __uint_as_float(w.z);
        x[3] = __uint_as_float(w.w);
    }
};

}  // namespace delta
