// checkpoint_calls.cuh -- activations kept in 8 bits (checkpoint.cuh) and read back, and
// the backward pass of the GELU from such a checkpoint, with the quantization and
// the bias's gradient that follow it.
//
// All three stream HBM: 3 and 1/32 bytes an element to and from a checkpoint, 4 and
// 1/32 through the backward pass with FP8 codes out.  (Part of fp8_matmul.cu's
// translation unit.)

#pragma once

#include "checkpoint.cuh"

namespace {

// ----------------------------------------------------------------------------
// To a checkpoint and back

struct CkptArgs {
    const uint16_t* x;
    uint16_t* y;
    uint8_t *q, *sf;
    int64_t rows, cols, blocks;  // blocks of 32, a row
    int64_t items;               // of sixteen elements (whole blocks), or of a block
};

constexpr int kCkptPer = 2;  // items a thread of the kernels of whole blocks, at a time

// Rows of whole blocks, which lie one behind another: sixteen elements a lane, two lanes a block.
__global__ void __launch_bounds__(kThreads) checkpoint_quantize_kernel(const CkptArgs a) {
    start_behind();
    const int64_t first = (int64_t)blockIdx.x * (kThreads * kCkptPer) + threadIdx.x;
    uint4 w[kCkptPer][2];
#pragma unroll
    for (int u = 0; u < kCkptPer; ++u)
        if (first + u * kThreads < a.items) ld_once_v8(a.x + (first + u * kThreads) * 16, w[u][0], w[u][1]);
#pragma unroll
    for (int u = 0; u < kCkptPer; ++u) {
        const int64_t i = first + u * kThreads;
        const uint32_t v[8] = {w[u][0].x, w[u][0].y, w[u][0].z, w[u][0].w, w[u][1].x, w[u][1].y, w[u][1].z, w[u][1].w};
        uint32_t m = absmax16(v);
        m = max(m & 0x7FFFu, m >> 16 & 0x7FFFu);
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        const uint32_t code = ckpt_scale(m);
        const float f = ckpt_factor(code);
        const uint32_t four = code | __shfl_down_sync(0xFFFFFFFFu, code, 2) << 8 | __shfl_down_sync(0xFFFFFFFFu, code, 4) << 16 |
                              __shfl_down_sync(0xFFFFFFFFu, code, 6) << 24;
        if (i < a.items) {
            st_v4(a.q + i * 16, make_uint4(ckpt_codes4(v[0], v[1], f), ckpt_codes4(v[2], v[3], f), ckpt_codes4(v[4], v[5], f), ckpt_codes4(v[6], v[7], f)));
            const int64_t blocks = a.items >> 1, b = i >> 1;
            if ((threadIdx.x & 7) == 0 && b + 4 <= blocks)
                *reinterpret_cast<uint32_t*>(a.sf + b) = four;
            else if ((threadIdx.x & 1) == 0 && (b & ~(int64_t)3) + 4 > blocks)
                a.sf[b] = (uint8_t)code;
        }
    }
}

// Rows of any length, from anywhere: a block a warp, a column a lane.
__global__ void __launch_bounds__(kThreads) checkpoint_quantize_rows_kernel(const CkptArgs a) {
    start_behind();
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t b = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; b < a.items; b += step) {
        const int64_t row = b / a.blocks, col = (b - row * a.blocks) * 32 + lane;
        const uint32_t w = col < a.cols ? a.x[row * a.cols + col] : 0u;
        const uint32_t code = ckpt_scale(__reduce_max_sync(0xFFFFFFFFu, w & 0x7FFFu));
        if (col < a.cols) a.q[row * a.cols + col] = (uint8_t)ckpt_codes4(w, 0u, ckpt_factor(code));
        if (lane == 0) a.sf[b] = (uint8_t)code;
    }
}

__global__ void __launch_bounds__(kThreads) checkpoint_dequantize_kernel(const CkptArgs a) {
    start_behind();
    const int64_t first = (int64_t)blockIdx.x * (kThreads * kCkptPer) + threadIdx.x;
    uint4 w[kCkptPer];
    uint32_t code[kCkptPer];
#pragma unroll
    for (int u = 0; u < kCkptPer; ++u) {
        const int64_t i = first + u * kThreads;
        if (i < a.items) w[u] = *reinterpret_cast<const uint4*>(a.q + i * 16), code[u] = a.sf[i >> 1];
    }
#pragma unroll
    for (int u = 0; u < kCkptPer; ++u) {
        const int64_t i = first + u * kThreads;
        if (i >= a.items) break;
        const float s = ckpt_value(code[u]);
        const uint32_t in[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float v[4];
            ckpt_decode4(in[j], s, v);
            o[2 * j] = cvt_bf16x2(v[0], v[1]), o[2 * j + 1] = cvt_bf16x2(v[2], v[3]);
        }
        st_v4(a.y + i * 16, make_uint4(o[0], o[1], o[2], o[3]));
        st_v4(a.y + i * 16 + 8, make_uint4(o[4], o[5], o[6], o[7]));
    }
}

__global__ void __launch_bounds__(kThreads) checkpoint_dequantize_rows_kernel(const CkptArgs a) {
    start_behind();
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t b = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; b < a.items; b += step) {
        const int64_t row = b / a.blocks, col = (b - row * a.blocks) * 32 + lane;
        if (col >= a.cols) continue;
        float v[4];
        ckpt_decode4(a.q[row * a.cols + col], ckpt_value(a.sf[b]), v);
        a.y[row * a.cols + col] = (uint16_t)(cvt_bf16x2(v[0], 0.0f) & 0xFFFFu);
    }
}

// ----------------------------------------------------------------------------
// Back through the GELU

constexpr int kNoCodes = -1;  // in place of the codes' format

struct GeluBackArgs {
    const uint16_t* dy;
    const uint8_t *h, *h_sf;  // NULL: no GELU
    uint16_t* dx;
    uint8_t* q;
    const float* scale;
    float *amax, *d_bias, *space;
    int64_t rows, cols, blocks;
    int64_t per_strip;
    int32_t strips;
};

// d/dx of x s(x), s(x) = 1 / (1 + t), t = exp(-2 sqrt(2 / pi) (x + 0.044715 x^3)):
//   s + x s (t s) 2 sqrt(2 / pi) (1 + 3 0.044715 x^2)
// Beyond +-10 it is 1 and 0 to 35 places, and given as such.
__device__ __forceinline__ float gelu_slope(float x) {
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(x), "f"(10.0f));
    const float x2 = x * x;
    float t, s;
    asm("ex2.approx.f32 %0, %1;" : "=f"(t) : "f"(x * fmaf(x2, -0.102943239f, -2.302208198f)));
    asm("rcp.approx.f32 %0, %1;" : "=f"(s) : "f"(1.0f + t));
    const float d = fmaf(x * fmaf(x2, 0.214064417f, 1.595769122f), s * (t * s), s);
    return x < -10.0f ? 0.0f : d;
}

constexpr int kGbCols = 256;  // columns a CTA: eight a lane, every eighth row a warp

// VEC: eight columns side by side a lane, in one load each; otherwise every 32nd.
template <int FMT, bool VEC>
__global__ void __launch_bounds__(kThreads) gelu_backward_kernel(const GeluBackArgs a) {
    __shared__ float part[kThreads / 32][kGbCols];
    __shared__ uint32_t red[kThreads / 32];
    start_behind();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t col0 = (int64_t)blockIdx.x * kGbCols, strip = blockIdx.y;
    const int64_t col = col0 + (VEC ? lane * 8 : lane);
    const int64_t r1 = min((strip + 1) * a.per_strip, a.rows);
    const QScale c = make_qscale_value(a.q ? *a.scale : 1.0f);
    float sum[8] = {};
    uint32_t m2 = 0;
    if (col < a.cols) {
#pragma unroll 2
        for (int64_t r = strip * a.per_strip + warp; r < r1; r += kThreads / 32) {
            const int64_t at = r * a.cols + col;
            uint32_t y[4] = {}, h[2] = {};
            float s[VEC ? 1 : 8];
            if (VEC) {
                const uint4 v = *reinterpret_cast<const uint4*>(a.dy + at);
                y[0] = v.x, y[1] = v.y, y[2] = v.z, y[3] = v.w;
                if (a.h) {
                    const uint2 u = *reinterpret_cast<const uint2*>(a.h + at);
                    h[0] = u.x, h[1] = u.y;
                    s[0] = ckpt_value(a.h_sf[r * a.blocks + (col >> 5)]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col + j * 32 < a.cols) {
                        y[j >> 1] |= (uint32_t)a.dy[at + j * 32] << (j & 1) * 16;
                        if (a.h) {
                            h[j >> 2] |= (uint32_t)a.h[at + j * 32] << (j & 3) * 8;
                            s[j] = ckpt_value(a.h_sf[r * a.blocks + (col >> 5) + j]);
                        }
                    } else if (!VEC) {
                        s[j] = 0.0f;
                    }
            }
            float d[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) d[2 * j] = __uint_as_float(y[j] << 16), d[2 * j + 1] = __uint_as_float(y[j] & 0xFFFF0000u);
            if (a.h) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float v[4];
                    ckpt_decode4(h[j], VEC ? s[0] : 1.0f, v);
#pragma unroll
                    for (int i = 0; i < 4; ++i) d[4 * j + i] *= gelu_slope(VEC ? v[i] : v[i] * s[VEC ? 0 : 4 * j + i]);
                }
            }
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 8; ++j) sum[j] += d[j];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = cvt_bf16x2(d[2 * j], d[2 * j + 1]);
            m2 = bf16x2_absmax(m2, bf16x2_absmax(bf16x2_absmax(w[0], w[1]), bf16x2_absmax(w[2], w[3])));
            uint2 o = make_uint2(0, 0);
            if (FMT != kNoCodes)
                o = c.fast ? make_uint2(quant_quad<FMT & 1, true>(w[0], w[1], c), quant_quad<FMT & 1, true>(w[2], w[3], c))
                           : make_uint2(quant_quad<FMT & 1, false>(w[0], w[1], c), quant_quad<FMT & 1, false>(w[2], w[3], c));
            if (VEC) {
                if (a.dx) st_v4(a.dx + at, make_uint4(w[0], w[1], w[2], w[3]));
                if (FMT != kNoCodes) st_v2(a.q + at, o);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (col + j * 32 < a.cols) {
                        if (a.dx) a.dx[at + j * 32] = (uint16_t)(w[j >> 1] >> (j & 1) * 16);
                        if (FMT != kNoCodes) a.q[at + j * 32] = (uint8_t)((j < 4 ? o.x : o.y) >> (j & 3) * 8);
                    }
            }
        }
    }
    if (a.amax) flush_amax(m2, 0, a.amax, red);
    if (!a.d_bias) return;
    // the eight warps' sums in their order
#pragma unroll
    for (int j = 0; j < 8; ++j) part[warp][VEC ? lane * 8 + j : lane + j * 32] = sum[j];
    __syncthreads();
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) v += part[w][threadIdx.x];
    if (col0 + threadIdx.x < a.cols) (a.strips > 1 ? a.space + strip * a.cols : a.d_bias)[col0 + threadIdx.x] = v;
}

// The strips' sums, 32 columns a CTA, every 32nd strip a warp, all in a fixed order.
__global__ void __launch_bounds__(1024) gelu_backward_sum_kernel(const GeluBackArgs a) {
    __shared__ float part[32][33];
    start_behind();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t col = (int64_t)blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (col < a.cols)
        for (int s = w; s < a.strips; s += 32) v += a.space[s * a.cols + col];
    part[w][lane] = v;
    __syncthreads();
    if (w > 0 || col >= a.cols) return;
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += part[i][lane];
    a.d_bias[col] = v;
}

// ----------------------------------------------------------------------------
// Host

struct GbStrips {
    int64_t strips, per_strip;
};
// As many CTAs as four an SM, of 32 rows or more; by the sizes alone, so that the sums' order is.
GbStrips gb_strips(int64_t rows, int64_t cols) {
    const int64_t across = (cols + kGbCols - 1) / kGbCols;
    int64_t strips = (4 * 152 + across - 1) / across;
    if (strips > (rows + 31) / 32) strips = (rows + 31) / 32;
    const int64_t per = (rows + strips - 1) / strips;
    return {(rows + per - 1) / per, per};
}

template <int FMT>
fp8q_status launch_gelu_backward(const GeluBackArgs& a, bool vec, cudaStream_t s) {
    const dim3 grid((unsigned)((a.cols + kGbCols - 1) / kGbCols), (unsigned)a.strips);
    return launch_behind(vec ? gelu_backward_kernel<FMT, true> : gelu_backward_kernel<FMT, false>, grid, dim3(kThreads), 0, 1, s,
                         "gelu_backward_kernel", a);
}

fp8q_status check_ckpt(const void* x, const uint8_t* q, const uint8_t* sf, int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0) return FP8Q_ERR_INVALID_ARG;
    if (rows > kFp4MaxDim || cols > kFp4MaxDim) return FP8Q_ERR_UNSUPPORTED;
    if (rows == 0 || cols == 0) return FP8Q_OK;
    if (!x || !q || !sf || ((uintptr_t)x & 1u)) return FP8Q_ERR_INVALID_ARG;
    return FP8Q_OK;
}

fp8q_status launch_ckpt(CkptArgs a, bool back, cudaStream_t s) {
    a.blocks = (a.cols + 31) / 32;
    const uintptr_t x = back ? (uintptr_t)a.y : (uintptr_t)a.x;
    const bool whole = a.cols % 32 == 0 && (x & (back ? 15u : 31u)) == 0 && ((uintptr_t)a.q & 15u) == 0 && ((uintptr_t)a.sf & 3u) == 0;
    if (whole) {
        a.items = a.rows * a.cols / 16;
        const int64_t grid = (a.items + kThreads * kCkptPer - 1) / (kThreads * kCkptPer);
        if (grid > 0x7FFFFFFF) return FP8Q_ERR_UNSUPPORTED;
        return launch_behind(back ? checkpoint_dequantize_kernel : checkpoint_quantize_kernel, dim3((unsigned)grid), dim3(kThreads), 0, 1, s,
                             back ? "checkpoint_dequantize_kernel" : "checkpoint_quantize_kernel", a);
    }
    a.items = a.rows * a.blocks;
    const int64_t want = (a.items + kThreads / 32 - 1) / (kThreads / 32), most = 64 * (int64_t)sm_count();
    return launch_behind(back ? checkpoint_dequantize_rows_kernel : checkpoint_quantize_rows_kernel, dim3((unsigned)(want < most ? want : most)),
                         dim3(kThreads), 0, 1, s, back ? "checkpoint_dequantize_rows_kernel" : "checkpoint_quantize_rows_kernel", a);
}

}  // namespace

extern "C" {

int64_t fp8q_checkpoint_scale_bytes(int64_t rows, int64_t cols) {
    if (rows < 0 || cols < 0 || rows > kFp4MaxDim || cols > kFp4MaxDim) return 0;
    return rows * ((cols + 31) / 32);
}

fp8q_status fp8q_checkpoint_quantize(const void* x_bf16, uint8_t* q, uint8_t* sf, int64_t rows, int64_t cols, void* stream) {
    const fp8q_status bad = check_ckpt(x_bf16, q, sf, rows, cols);
    if (bad != FP8Q_OK || rows == 0 || cols == 0) return bad;
    CkptArgs a = {};
    a.x = static_cast<const uint16_t*>(x_bf16);
    a.q = q;
    a.sf = sf;
    a.rows = rows;
    a.cols = cols;
    return launch_ckpt(a, false, static_cast<cudaStream_t>(stream));
}

fp8q_status fp8q_checkpoint_dequantize(const uint8_t* q, const uint8_t* sf, void* y_bf16, int64_t rows, int64_t cols, void* stream) {
    const fp8q_status bad = check_ckpt(y_bf16, q, sf, rows, cols);
    if (bad != FP8Q_OK || rows == 0 || cols == 0) return bad;
    CkptArgs a = {};
    a.y = static_cast<uint16_t*>(y_bf16);
    a.q = const_cast<uint8_t*>(q);
    a.sf = const_cast<uint8_t*>(sf);
    a.rows = rows;
    a.cols = cols;
    return launch_ckpt(a, true, static_cast<cudaStream_t>(stream));
}

int64_t fp8q_gelu_backward_workspace(int64_t rows, int64_t cols) {
    if (rows <= 0 || cols <= 0 || rows > kFp4MaxDim || cols > kFp4MaxDim) return 0;
    const GbStrips st = gb_strips(rows, cols);
    return st.strips > 1 ? st.strips * cols * (int64_t)sizeof(float) : 0;
}

fp8q_status fp8q_gelu_backward_quantize_amax(const fp8q_gelu_grad* g, void* stream) {
    if (!g || g->rows < 0 || g->cols < 0 || !valid_fmt(g->fmt)) return FP8Q_ERR_INVALID_ARG;
    if (g->rows > kFp4MaxDim || g->cols > kFp4MaxDim) return FP8Q_ERR_UNSUPPORTED;
    if (g->cols == 0) return FP8Q_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if ((uintptr_t)g->d_bias & 3u) return FP8Q_ERR_INVALID_ARG;
    if (g->rows == 0) {  // the sums over no rows
        if (!g->d_bias) return FP8Q_OK;
        const cudaError_t e = cudaMemsetAsync(g->d_bias, 0, (size_t)g->cols * sizeof(float), s);
        return e == cudaSuccess ? FP8Q_OK : cuda_fail(e, "fp8q_gelu_backward_quantize_amax");
    }
    if (!g->d_y || (g->h != nullptr) != (g->h_sf != nullptr) || (g->q != nullptr) != (g->scale != nullptr)) return FP8Q_ERR_INVALID_ARG;
    if (!g->q && !g->d_x && !g->d_bias && !g->amax) return FP8Q_ERR_INVALID_ARG;
    if ((((uintptr_t)g->d_y | (uintptr_t)g->d_x) & 1u) || (((uintptr_t)g->scale | (uintptr_t)g->amax | (uintptr_t)g->workspace) & 3u))
        return FP8Q_ERR_INVALID_ARG;
    const GbStrips st = gb_strips(g->rows, g->cols);
    if (g->d_bias && st.strips > 1 && (!g->workspace || g->workspace_bytes < fp8q_gelu_backward_workspace(g->rows, g->cols)))
        return FP8Q_ERR_INVALID_ARG;
    GeluBackArgs a;
    a.dy = static_cast<const uint16_t*>(g->d_y);
    a.h = g->h;
    a.h_sf = g->h_sf;
    a.dx = static_cast<uint16_t*>(g->d_x);
    a.q = g->q;
    a.scale = g->scale;
    a.amax = g->amax;
    a.d_bias = g->d_bias;
    a.space = static_cast<float*>(g->workspace);
    a.rows = g->rows;
    a.cols = g->cols;
    a.blocks = (g->cols + 31) / 32;
    a.per_strip = st.per_strip;
    a.strips = (int32_t)st.strips;
    const bool vec = g->cols % 8 == 0 && (((uintptr_t)g->d_y | (uintptr_t)g->d_x) & 15u) == 0 && (((uintptr_t)g->h | (uintptr_t)g->q) & 7u) == 0;
    const fp8q_status rc = !g->q               ? launch_gelu_backward<kNoCodes>(a, vec, s)
                           : g->fmt == FP8Q_E4M3FN ? launch_gelu_backward<FP8Q_E4M3FN>(a, vec, s)
                                                   : launch_gelu_backward<FP8Q_E5M2>(a, vec, s);
    if (rc != FP8Q_OK || !a.d_bias || a.strips == 1) return rc;
    return launch_behind(gelu_backward_sum_kernel, dim3((unsigned)((a.cols + 31) / 32)), dim3(1024), 0, 1, s, "gelu_backward_sum_kernel", a);
}

}  // extern "C"
