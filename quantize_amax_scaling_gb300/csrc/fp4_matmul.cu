// fp4_matmul.cu -- the product of two microscaled 4-bit operands.
//
//   D[m][n] = RN_out( (sum_k A[m][k] B[n][k]) * RN(sa * sb) )
//
// with both operands packed along k (fp4.cuh).  First form: 64x64 tiles of D,
// operands widened to binary32 in shared memory, one fused multiply-add a
// product in order of k.

#include "fp4.cuh"

namespace {

constexpr int kMT = 64, kKT = 64;

struct Fp4MatmulArgs {
    const uint8_t *a, *a_sf, *b, *b_sf;
    const float *a_scale, *b_scale;
    void* d;
    int64_t m, n, k;
};

template <int FMT>
__device__ __forceinline__ void widen_tile(float (*t)[kMT + 1], const uint8_t* q, const uint8_t* sf, int64_t r0,
                                           int64_t rows, int64_t k0, int64_t k) {
    const int64_t ld = fp4_row_bytes(k), across = fp4_sf_tiles<FMT>(k);
    // 64 rows x 8 words of eight codes
    for (int id = threadIdx.x; id < kMT * kKT / 8; id += kThreads) {
        const int row = id >> 3, wd = id & 7;
        const int64_t r = r0 + row, c = k0 + wd * 8;
        float v[8] = {};
        if (r < rows && c < 2 * ld) {
            const int64_t blk = c / Fp4<FMT>::kBlock;
            const float s = sf_value<FMT>(
                sf[((r / 128) * across + blk / 4) * 512 + (r % 32) * 16 + (r % 128) / 32 * 4 + blk % 4]);
            uint32_t h[4];
            e2m1x8_to_f16(*reinterpret_cast<const uint32_t*>(q + r * ld + c / 2), h);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = f16_lo(h[i]) * s;
                v[2 * i + 1] = f16_hi(h[i]) * s;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) t[wd * 8 + i][row] = v[i];
    }
}

template <int FMT, bool F32>
__global__ void __launch_bounds__(kThreads) fp4_matmul_kernel(const Fp4MatmulArgs p) {
    __shared__ float ta[kKT][kMT + 1], tb[kKT][kMT + 1];
    const int64_t tiles_n = (p.n + kMT - 1) / kMT;
    const int64_t m0 = (int64_t)blockIdx.x / tiles_n * kMT, n0 = (int64_t)blockIdx.x % tiles_n * kMT;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < p.k; k0 += kKT) {
        widen_tile<FMT>(ta, p.a, p.a_sf, m0, p.m, k0, p.k);
        widen_tile<FMT>(tb, p.b, p.b_sf, n0, p.n, k0, p.k);
        __syncthreads();
        for (int kk = 0; kk < kKT; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(ta[kk][ty + 16 * i], tb[kk][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
    const float alpha = __fmul_rn(p.a_scale ? __ldg(p.a_scale) : 1.0f, p.b_scale ? __ldg(p.b_scale) : 1.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m >= p.m || n >= p.n) continue;
            const float v = __fmul_rn(acc[i][j], alpha);
            if (F32)
                static_cast<float*>(p.d)[m * p.n + n] = v;
            else
                static_cast<uint16_t*>(p.d)[m * p.n + n] = (uint16_t)cvt_bf16x2(v, 0.0f);
        }
}

}  // namespace

extern "C" {

fp8q_status fp8q_fp4_matmul(const uint8_t* a, const uint8_t* a_sf, const uint8_t* b, const uint8_t* b_sf, void* d,
                            int64_t m, int64_t n, int64_t k, fp8q_format fmt, fp8q_out_type out, const float* a_scale,
                            const float* b_scale, void* stream) {
    if (!valid_fp4(fmt) || m < 0 || n < 0 || k < 0) return FP8Q_ERR_INVALID_ARG;
    if (out != FP8Q_OUT_BF16 && out != FP8Q_OUT_F32) return FP8Q_ERR_INVALID_ARG;
    if (m == 0 || n == 0) return FP8Q_OK;
    if (k == 0) return FP8Q_ERR_INVALID_ARG;
    if (m > kFp4MaxDim || n > kFp4MaxDim || k > kFp4MaxDim) return FP8Q_ERR_UNSUPPORTED;
    if (!a || !a_sf || !b || !b_sf || !d) return FP8Q_ERR_INVALID_ARG;
    if (fmt == FP8Q_MXFP4 && (a_scale || b_scale)) return FP8Q_ERR_INVALID_ARG;
    if (((uintptr_t)d & (out == FP8Q_OUT_F32 ? 3u : 1u)) || ((uintptr_t)a_scale & 3u) || ((uintptr_t)b_scale & 3u))
        return FP8Q_ERR_INVALID_ARG;
    if (((uintptr_t)a | (uintptr_t)a_sf | (uintptr_t)b | (uintptr_t)b_sf) & 15u) return FP8Q_ERR_UNSUPPORTED;
    Fp4MatmulArgs p = {a, a_sf, b, b_sf, a_scale, b_scale, d, m, n, k};
    const int64_t tm = (m + kMT - 1) / kMT, tn = (n + kMT - 1) / kMT;
    if (tm > 0x7FFFFFFF / tn) return FP8Q_ERR_UNSUPPORTED;
    auto kern = fmt == FP8Q_MXFP4 ? (out == FP8Q_OUT_F32 ? fp4_matmul_kernel<FP8Q_MXFP4, true> : fp4_matmul_kernel<FP8Q_MXFP4, false>)
                                  : (out == FP8Q_OUT_F32 ? fp4_matmul_kernel<FP8Q_NVFP4, true> : fp4_matmul_kernel<FP8Q_NVFP4, false>);
    return launch_kernel(kern, dim3((unsigned)(tm * tn)), dim3(kThreads), 0, static_cast<cudaStream_t>(stream),
                         "fp4_matmul_kernel", p);
}

}  // extern "C"
