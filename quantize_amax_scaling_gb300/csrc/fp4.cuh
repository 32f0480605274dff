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
#include "packed_f32.cuh"

#include <atomic>
#include <cstdlib>

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

// The SMs of the current device, or of the part of it that this process has.
inline int sm_count() {
#ifdef FP8Q_TEST_HOOKS
    if (const char* n = getenv("FP8Q_TEST_SM_COUNT")) return atoi(n);
#endif
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return 152;
    int n = known[dev].load(std::memory_order_relaxed);
    if (!n) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 2) n = 152;
        known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

inline bool valid_fp4(int fmt) { return fmt == FP8Q_MXFP4 || fmt == FP8Q_NVFP4; }

constexpr int64_t kFp4MaxDim = 0x7FFFFC00;  // rows and columns of an operand: coordinates within a tile beyond the last stay in 32 bits

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

// 32 and 8 bytes that are read once; not by the read-only path, whose data may not
// change while a kernel lives: see wait_behind().
__device__ __forceinline__ void ld_once_v8(const void* p, uint4& a, uint4& b) {
    asm volatile("ld.global.L1::no_allocate.L2::256B.v8.u32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(a.x), "=r"(a.y), "=r"(a.z), "=r"(a.w), "=r"(b.x), "=r"(b.y), "=r"(b.z), "=r"(b.w)
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ uint2 ld_once_v2(const void* p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.L2::256B.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p) : "memory");
    return v;
}

// The kernels of launch_behind() may start while the kernel before them in their
// stream still runs, and touch no global memory before wait_behind(), which
// returns when that kernel has ended and what it wrote can be read.  Every thread
// calls it, so that a kernel never ends before the one ahead of it.
__device__ __forceinline__ void wait_behind() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The same, and the next kernel may start as soon as all CTAs have come here: it
// waits in its turn, so two kernels of a stream are under way at most.
// (Quantize and multiply, NVFP4, 1 x 16384 x 4096: 12.5 us, 16.6 with launches in
// order; residual norm and product, 1555 x 11264 x 4096: 49 and 55 us.)
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void start_behind() {
    wait_behind();
    let_next_start();
}

// launch_kernel() for them; clusters of `cluster` CTAs.
template <typename... KArgs, typename... Args>
fp8q_status launch_behind(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, unsigned cluster, cudaStream_t s,
                          const char* where, Args&&... args) {
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<Args&&>(args)...);
    return e == cudaSuccess ? FP8Q_OK : cuda_fail(e, where);
}

// Four pairs of binary32 values -> eight e2m1 codes (nearest, ties to even,
// held at +-6; the first value in the lowest four bits).
__device__ __forceinline__ uint32_t cvt_e2m1x8(const unsigned long long (&f)[4]) {
    uint32_t d;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t.reg .f32 x, y;\n\t"
        "mov.b64 {x, y}, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 a, y, x;\n\t"
        "mov.b64 {x, y}, %2;\n\tcvt.rn.satfinite.e2m1x2.f32 b, y, x;\n\t"
        "mov.b64 {x, y}, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 c, y, x;\n\t"
        "mov.b64 {x, y}, %4;\n\tcvt.rn.satfinite.e2m1x2.f32 d, y, x;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(d)
        : "l"(f[0]), "l"(f[1]), "l"(f[2]), "l"(f[3]));
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
    float s;      // the tensor scale
    float s6;     // RN(6 s)
    float r6;     // RN(1 / s6) where `fast`
    float s64;    // s 2^64
    float cap;    // s6 2^17
    float limit;  // the largest block maximum whose elements take the exact quotient without a divide
    bool good;    // s6 positive and finite
    bool fast;    // s in [2^-50, 2^50]: with block scales from 2^-9 to 448 everything stays in [2^-60, 2^60]
};

__device__ __forceinline__ Fp4Scale make_fp4_scale(const float* scale) {
    Fp4Scale c;
    c.s = scale ? *scale : 1.0f;
    c.s6 = __fmul_rn(c.s, 6.0f);
    c.good = c.s6 > 0.0f && c.s6 <= 3.402823466e38f;
    c.fast = c.s >= 0x1p-50f && c.s <= 0x1p50f;
    c.r6 = c.fast ? __frcp_rn(c.s6) : 1.0f;
    c.s64 = c.fast ? c.s * 0x1p64f : 1.0f;
    c.cap = c.s6 * 131072.0f;
    c.limit = c.fast ? c.s * (448.0f * 131072.0f) : -1.0f;
    return c;
}

// RN(x / s) with r = RN(1 / s): Markstein's correction step (fp8q_common.cuh),
// exact for bf16 x while nothing leaves the normal range.
__device__ __forceinline__ float quotient(float x, float s, float r) {
    const float y0 = __fmul_rn(x, r);
    return __fmaf_rn(-__fmaf_rn(y0, s, -x), r, y0);
}

// Two binary32 values in one 64-bit register, as the two-lane instructions take
// them.  Kept whole between operations: as two floats they cost moves.
using Two = unsigned long long;
__device__ __forceinline__ Two two(uint32_t lo, uint32_t hi) {
    Two d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
    return d;
}
__device__ __forceinline__ Two two(float v) { return two(__float_as_uint(v), __float_as_uint(v)); }
__device__ __forceinline__ Two widen2(uint32_t w) { return two(w << 16, w & 0xFFFF0000u); }  // two bf16
__device__ __forceinline__ Two mul_two(Two a, Two b) {
    Two d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Two fma_two(Two a, Two b, Two c) {
    Two d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// -quotient() for two, with mr = -RN(1 / s): without a minus the step takes three
// instructions, and a zero still comes out with the sign opposite to x's (each
// sum of two zeros below is of unlike ones for x = -0, of negative ones for +0).
__device__ __forceinline__ Two minus_quotient(Two x, Two s, Two mr) {
    const Two z0 = mul_two(x, mr);
    return fma_two(fma_two(z0, s, x), mr, z0);
}

// The same on pairs of floats.
__device__ __forceinline__ float2 quotient2(float2 x, float2 s, float2 r, float2 mr) {
    const float2 y0 = mul2_rn(x, r);
    return fma2_rn(fma2_rn(y0, s, mul2_rn(x, splat2(-1.0f))), mr, y0);
}

// A block's scale byte, and what its elements are divided by.
struct BlockScale {
    uint32_t code;
    float d;    // MX: the factor 2^-e; NV: RN(block scale * tensor scale), 1 where that is 0
    float r;    // NV: RN(1 / d), 0 where all codes are zero
    bool slow;  // NV: beyond the exact quotient's range
};

// a: the block's max|x| as bf16 bits (NaN above 0x7F80).  FAST: c.fast.
template <int FMT, bool FAST>
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
        b.slow = false;
        return b;
    }
    const float af = __uint_as_float(a << 16);
    if (FAST) {
        // beyond 2^17 s6 the scale is held at 448 anyway; a NaN stays one
        float v;
        asm("min.NaN.f32 %0, %1, %2;" : "=f"(v) : "f"(af), "f"(c.cap));
        b.code = cvt_fp8x2<FP8Q_E4M3FN>(quotient(v, c.s6, c.r6), 0.0f);
        const float f = f16_lo(fp8x2_to_f16x2<FP8Q_E4M3FN>(b.code));
        b.d = __fmul_rn(f, c.s);
        // RN(1 / d): the approximation and one correction (packed_f32.cuh) for d 2^64, which
        // lies where that is checked for every significand
        const float e = __fmul_rn(f, c.s64), y = rcp_approx_ftz(e);
        b.r = fmaf(y, fmaf(-e, y, 1.0f), y) * 0x1p64f;
        b.slow = af > c.limit;
    } else {
        b.code = cvt_fp8x2<FP8Q_E4M3FN>(__fdiv_rn(af, c.s6), 0.0f) & 0xFFu;
        if (a > 0x7F80u || !c.good) b.code = 0x7Fu;
        if (a == 0u) b.code = 0u;
        b.d = __fmul_rn(sf_value<FMT>(b.code), c.s);
        b.r = 1.0f;
        b.slow = b.d > 0.0f;
    }
    if (!(b.d > 0.0f)) b.r = 0.0f, b.d = 1.0f;  // quotient() of it: zero, with x's sign
    return b;
}

// Off the fast path: d may be infinite, and an infinity is +-6 all the same.
__device__ __noinline__ float slow_quotient(float x, float d) {
    return fabsf(x) > 3.402823466e38f ? x : __fdiv_rn(x, d);
}

// Eight values of a block -> eight codes.
template <int FMT>
__device__ __forceinline__ uint32_t codes8(Two (&f)[4], const BlockScale& b) {
    if (FMT == FP8Q_MXFP4) {
        const Two d = two(b.d);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = mul_two(f[i], d);  // exact, or below half the smallest code
    } else if (!b.slow) {
        const Two mr = two(-b.r), d = two(b.d);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = minus_quotient(f[i], d, mr);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = two(__float_as_uint(-slow_quotient(__uint_as_float((uint32_t)f[i]), b.d)),
                       __float_as_uint(-slow_quotient(__uint_as_float((uint32_t)(f[i] >> 32)), b.d)));
    }
    return FMT == FP8Q_MXFP4 ? cvt_e2m1x8(f) : cvt_e2m1x8(f) ^ 0x88888888u;  // the signs of x
}

// Eight bf16 of a block (four words, the even column low).
template <int FMT>
__device__ __forceinline__ uint32_t codes8(const uint32_t (&w)[4], const BlockScale& b) {
    Two f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = widen2(w[i]);
    return codes8<FMT>(f, b);
}

// Sixteen bf16 (eight words) -> sixteen codes (two words).
template <int FMT>
__device__ __forceinline__ uint2 block_codes(const uint32_t (&w)[8], const BlockScale& b) {
    const uint32_t lo[4] = {w[0], w[1], w[2], w[3]}, hi[4] = {w[4], w[5], w[6], w[7]};
    return make_uint2(codes8<FMT>(lo, b), codes8<FMT>(hi, b));
}

__device__ __forceinline__ uint32_t absmax16(const uint32_t (&w)[8]) {  // both halves, sign undefined
    return bf16x2_absmax(bf16x2_absmax(bf16x2_absmax(w[0], w[1]), bf16x2_absmax(w[2], w[3])),
                         bf16x2_absmax(bf16x2_absmax(w[4], w[5]), bf16x2_absmax(w[6], w[7])));
}

}  // namespace
