// checkpoint.cuh -- the 8-bit checkpoint of an activation: e4m3 codes under a power
// of two for each block of 32 columns of a row.
//
//   a = max|x| of the block (an infinity counts as the largest finite bf16),
//   scale 2^e with the least e >= -127 for which a <= 448 2^e,  code = e4m3(x / 2^e)
//
// The power of two makes the quotient exact, so a value is rounded once, by half a
// step of e4m3 (2^-4 of it, or 2^-10 2^e where that is more).  The scale's byte is
// e + 127; 255, NaN, where the block holds a NaN.  An infinity comes back as one
// (448 2^120 is beyond binary32), and so does a finite value from 248 2^120 on, whose
// code is 256's.
//
// Codes are [rows, cols] bytes, scales [rows, ceil(cols / 32)] bytes, both row-major.

#pragma once

#include "fp4.cuh"

namespace {

// A block's scale byte from its max|x| as bf16 bits (NaN above 0x7F80).
__device__ __forceinline__ uint32_t ckpt_scale(uint32_t a) {
    if (a > 0x7F80u) return 255u;
    a = min(a, 0x7F7Fu);
    // 1.m 2^(E - 127) <= 1.75 2^8 2^e: e = E - 135, one more where m is above 0.75
    const uint32_t e = (a + 0x1Fu) >> 7;  // E, or E + 1 where the seven bits of m exceed 0x60
    return e > 8u ? e - 8u : 0u;
}

// What its elements are multiplied by: 2^-e.
__device__ __forceinline__ float ckpt_factor(uint32_t code) { return __uint_as_float((254u - min(code, 253u)) << 23); }

// Four bf16 (two words) -> four codes.
__device__ __forceinline__ uint32_t ckpt_codes4(uint32_t w0, uint32_t w1, float f) {
    const uint32_t lo = cvt_fp8x2<FP8Q_E4M3FN>(__uint_as_float(w0 << 16) * f, __uint_as_float(w0 & 0xFFFF0000u) * f);
    const uint32_t hi = cvt_fp8x2<FP8Q_E4M3FN>(__uint_as_float(w1 << 16) * f, __uint_as_float(w1 & 0xFFFF0000u) * f);
    return lo | hi << 16;
}

// 2^e of a scale byte (subnormal for 0), NaN for 255.
__device__ __forceinline__ float ckpt_value(uint32_t code) { return sf_value<FP8Q_MXFP4>(code); }

// Four codes -> four values.
__device__ __forceinline__ void ckpt_decode4(uint32_t four, float s, float (&v)[4]) {
    const uint32_t a = fp8x2_to_f16x2<FP8Q_E4M3FN>(four & 0xFFFFu), b = fp8x2_to_f16x2<FP8Q_E4M3FN>(four >> 16);
    v[0] = f16_lo(a) * s, v[1] = f16_hi(a) * s, v[2] = f16_lo(b) * s, v[3] = f16_hi(b) * s;
}

// A whole sector in one store.
__device__ __forceinline__ void st_v8(void* p, const uint4& a, const uint4& b) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w), "r"(b.x),
                 "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
}

__device__ __forceinline__ Two add_two(Two a, Two b) {
    Two d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// quant_quad() at a scale that takes the exact quotient without a divide, two lanes at a time: the negative of -x's.
template <int FMT>
__device__ __forceinline__ uint32_t codes4_fast(uint32_t w0, uint32_t w1, Two s, Two mr, uint32_t t2) {
    const Two a = minus_quotient(widen2(bf16x2_clamp(w0, t2) ^ 0x80008000u), s, mr), b = minus_quotient(widen2(bf16x2_clamp(w1, t2) ^ 0x80008000u), s, mr);
    const uint32_t lo = cvt_fp8x2<FMT>(__uint_as_float((uint32_t)a), __uint_as_float((uint32_t)(a >> 32)));
    const uint32_t hi = cvt_fp8x2<FMT>(__uint_as_float((uint32_t)b), __uint_as_float((uint32_t)(b >> 32)));
    return lo | hi << 16;
}

}  // namespace
