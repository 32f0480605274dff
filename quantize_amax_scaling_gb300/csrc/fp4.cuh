// fp4.cuh -- the microscaled 4-bit formats: geometry of a packed operand, the
// block scale and the codes of one block, and the values they stand for.
//
// A packed operand of an [rows, cols] matrix is two arrays:
//   codes   rows x fp4_row_bytes(cols) bytes, two e2m1 codes a byte (the even
//           column in the low four bits), each row filled up with zero codes
//           to a multiple of 32 columns, so that every row starts on the
//           16-byte boundary that a tensor-map copy needs;
//   scales  one byte a block, in tiles of 128 rows x 4 blocks, the order in
//           which the tensor cores' scale memory takes them: the scale of
//           (row, block) lies in tile (row / 128) * ceil(blocks / 4) + block / 4,
//           at byte (row % 32) * 16 + (row % 128) / 32 * 4 + block % 4 of its
//           512.  Each row's blocks are filled up to a multiple of 4 with zero
//           scales; the rows that fill up the last tile are never written.

#pragma once

#include "fp8q_common.cuh"

#include <atomic>

namespace {

// A kernel's shared-memory limit, set on its first call on each device.
template <typename K>
cudaError_t allow_smem(K kern, int bytes, std::atomic<uint64_t>& devices) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (devices.load(std::memory_order_acquire) >> dev & 1)) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev < 64) devices.fetch_or(1ull << dev, std::memory_order_release);
    return e;
}

inline bool valid_fp4(int fmt) { return fmt == FP8Q_MXFP4 || fmt == FP8Q_NVFP4; }

constexpr int64_t kFp4MaxDim = 0x7FFFFF80;  // rows and columns of an operand: tile coordinates are 32-bit

template <int FMT>
struct Fp4 {
    static constexpr int kBlock = FMT == FP8Q_MXFP4 ? 32 : 16;  // columns a scale
    static constexpr int kSfCols = 4 * kBlock;                  // columns a scale tile
};

__host__ __device__ inline int64_t fp4_row_bytes(int64_t cols) { return (cols + 31) / 32 * 16; }
template <int FMT>
__host__ __device__ inline int64_t fp4_sf_tiles(int64_t cols) {  // scale tiles a row of tiles
    return (cols + Fp4<FMT>::kSfCols - 1) / Fp4<FMT>::kSfCols;
}

__device__ __forceinline__ void st_v2(void* p, uint2 v) {
    asm volatile("st.global.cs.v2.u32 [%0], {%1,%2};" ::"l"(p), "r"(v.x), "r"(v.y) : "memory");
}

// Four pairs of binary32 values -> eight e2m1 codes (nearest, ties to even,
// held at +-6; the first value in the lowest four bits).
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&f)[8]) {
    uint32_t d;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(d)
        : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
    return d;
}

// Eight e2m1 codes -> four f16x2 words of their values, exact.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// The value of a scale byte: 2^(code - 127) (subnormal for 0, NaN for 255), or e4m3.
template <int FMT>
__device__ __forceinline__ float sf_value(uint32_t code) {
    if (FMT == FP8Q_MXFP4) {
        if (code == 255u) return __uint_as_float(0x7FC00000u);
        return code ? __uint_as_float(code << 23) : 0x1p-127f;
    }
    return f16_lo(fp8x2_to_f16x2<FP8Q_E4M3FN>(code));
}

// What a CTA derives from the tensor scale of the 16-block format.
struct Fp4Scale {
    float s;     // the tensor scale
    float s6;    // RN(6 s)
    float r6;    // RN(1 / s6) where `fast`
    bool good;   // s6 positive and finite
    bool fast;   // s6 in [2^-60, 2^60]: the exact quotient without a divide
};

__device__ __forceinline__ Fp4Scale make_fp4_scale(const float* scale) {
    Fp4Scale c;
    c.s = scale ? __ldg(scale) : 1.0f;
    c.s6 = __fmul_rn(c.s, 6.0f);
    c.good = c.s6 > 0.0f && c.s6 <= 3.402823466e38f;
    c.fast = c.s6 >= 0x1p-60f && c.s6 <= 0x1p60f;
    c.r6 = c.fast ? __frcp_rn(c.s6) : 1.0f;
    return c;
}

// RN(x / s) with r = RN(1 / s): Markstein's correction step (fp8q_common.cuh),
// exact for bf16 x while nothing leaves the normal range.
__device__ __forceinline__ float quotient(float x, float s, float r) {
    const float y0 = __fmul_rn(x, r);
    return __fmaf_rn(-__fmaf_rn(y0, s, -x), r, y0);
}

// A block's scale byte, and what its elements are divided by.
struct BlockScale {
    uint32_t code;
    float d;     // MX: the factor 2^-e; NV: RN(block scale * tensor scale)
    float r;     // NV: RN(1 / d)
    int mode;    // NV: 0 all codes zero, 1 exact quotient by r, 2 divide
};

// a: the block's max|x| as bf16 bits (NaN above 0x7F80).
template <int FMT>
__device__ __forceinline__ BlockScale block_scale(uint32_t a, const Fp4Scale& c) {
    BlockScale b;
    if (FMT == FP8Q_MXFP4) {
        // e = max(-127, floor(log2 a) - 2): the exponent field less two.  An
        // infinity takes the largest finite number's exponent.
        const uint32_t e = min(a >> 7, 254u);
        const uint32_t code = e > 2u ? e - 2u : 0u;
        b.code = a > 0x7F80u ? 255u : code;
        b.d = __uint_as_float((254u - code) << 23);  // 2^(127 - code), normal for code <= 252
        b.r = 1.0f;
        b.mode = 1;
        return b;
    }
    const float af = __uint_as_float(a << 16);
    float v;
    if (c.fast)  // beyond 2^17 s6 the scale is held at 448 anyway
        v = quotient(fminf(af, c.s6 * 131072.0f), c.s6, c.r6);
    else
        v = __fdiv_rn(af, c.s6);
    b.code = cvt_fp8x2<FP8Q_E4M3FN>(v, 0.0f) & 0xFFu;
    if (!c.good && a != 0u) b.code = 0x7Fu;
    if (a > 0x7F80u) b.code = 0x7Fu;
    if (a == 0u) b.code = 0u;
    b.d = __fmul_rn(sf_value<FMT>(b.code), c.s);
    b.mode = 0;
    b.r = 1.0f;
    if (b.d > 0.0f) {
        const bool q = b.d >= 0x1p-60f && b.d <= 0x1p60f && af <= b.d * 131072.0f;
        b.mode = q ? 1 : 2;
        if (q) b.r = __frcp_rn(b.d);
    }
    return b;
}

// Sixteen bf16 (eight words, the even column low) -> sixteen codes (two words).
template <int FMT>
__device__ __forceinline__ uint2 block_codes(const uint32_t (&w)[8], const BlockScale& b) {
    uint32_t o[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[4 * h + i] << 16);
            f[2 * i + 1] = __uint_as_float(w[4 * h + i] & 0xFFFF0000u);
        }
        if (FMT == FP8Q_MXFP4) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(f[i], b.d);  // exact, or below half the smallest code
        } else if (b.mode == 1) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = quotient(f[i], b.d, b.r);
        } else if (b.mode == 2) {
#pragma unroll
            for (int i = 0; i < 8; ++i)  // d may be infinite: an infinity is +-6 all the same
                f[i] = fabsf(f[i]) > 3.402823466e38f ? f[i] : __fdiv_rn(f[i], b.d);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = copysignf(0.0f, f[i]);
        }
        o[h] = cvt_e2m1x8(f);
    }
    return make_uint2(o[0], o[1]);
}

__device__ __forceinline__ uint32_t absmax16(const uint32_t (&w)[8]) {  // both halves, sign undefined
    return bf16x2_absmax(bf16x2_absmax(bf16x2_absmax(w[0], w[1]), bf16x2_absmax(w[2], w[3])),
                         bf16x2_absmax(bf16x2_absmax(w[4], w[5]), bf16x2_absmax(w[6], w[7])));
}

}  // namespace
