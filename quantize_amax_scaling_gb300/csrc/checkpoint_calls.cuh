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
    int64_t items;               // of sixteen elements, or stretches of rows
    int64_t across;              // of them, a row
    int32_t stretch;             // blocks, a multiple of four
};

// Rows of whole sixteens: sixteen elements a lane, two lanes a block (two or four of them a thread are 1% and 2% slower).
// HALF: the last block of a row is one of sixteen columns, its second lane's item empty (8192x2064 9.5 us and 9.2 back; a column
// a lane, as below, 31 and 21).
template <bool HALF>
__device__ __forceinline__ int64_t ckpt_at(const CkptArgs& a, int64_t item) {  // its first element; rows * cols for an empty one
    if (!HALF) return item * 16;
    const int64_t row = a.items <= INT32_MAX ? (int64_t)((uint32_t)item / (uint32_t)a.across) : item / a.across, col = (item - row * a.across) * 16;
    return col < a.cols ? row * a.cols + col : a.rows * a.cols;
}

template <bool HALF>
__global__ void __launch_bounds__(kThreads) checkpoint_quantize_kernel(const CkptArgs a) {
    start_behind();
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t at = i < a.items ? ckpt_at<HALF>(a, i) : a.rows * a.cols;
    const bool on = at < a.rows * a.cols;
    uint4 w[2] = {};
    if (on) ld_once_v8(a.x + at, w[0], w[1]);
    const uint32_t v[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
    uint32_t m = absmax16(v);
    m = max(m & 0x7FFFu, m >> 16 & 0x7FFFu);
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    const uint32_t code = ckpt_scale(m);
    const float f = ckpt_factor(code);
    const uint32_t four = code | __shfl_down_sync(0xFFFFFFFFu, code, 2) << 8 | __shfl_down_sync(0xFFFFFFFFu, code, 4) << 16 |
                          __shfl_down_sync(0xFFFFFFFFu, code, 6) << 24;
    if (i >= a.items) return;
    if (on) st_v4(a.q + at, make_uint4(ckpt_codes4(v[0], v[1], f), ckpt_codes4(v[2], v[3], f), ckpt_codes4(v[4], v[5], f), ckpt_codes4(v[6], v[7], f)));
    const int64_t blocks = a.items >> 1, b = i >> 1;
    if ((threadIdx.x & 7) == 0 && b + 4 <= blocks)
        *reinterpret_cast<uint32_t*>(a.sf + b) = four;
    else if ((threadIdx.x & 1) == 0 && (b & ~(int64_t)3) + 4 > blocks)
        a.sf[b] = (uint8_t)code;
}

// Rows of any length, from anywhere: a stretch of a row a warp, four blocks side by side at a time, a column of each a lane.
// The place of a stretch takes a division, more than the codes of a block.
struct CkptRow {
    int64_t at;     // of the lane's first element
    int64_t block;  // the first block
    int blocks;     // there
    int left;       // elements of the row from the lane's first on, held at 2^20
};
__device__ __forceinline__ CkptRow ckpt_row(const CkptArgs& a, int64_t item) {
    const int64_t row = a.items <= INT32_MAX ? (int64_t)((uint32_t)item / (uint32_t)a.across) : item / a.across, b = (item - row * a.across) * a.stretch;
    const int64_t col = b * 32 + (threadIdx.x & 31);
    return {row * a.cols + col, row * a.blocks + b, (int)min(a.blocks - b, (int64_t)a.stretch), (int)min(a.cols - col, (int64_t)1 << 20)};
}

__global__ void __launch_bounds__(kThreads) checkpoint_quantize_rows_kernel(const CkptArgs a) {
    start_behind();
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; i < a.items; i += step) {
        CkptRow r = ckpt_row(a, i);
        const uint16_t* x = a.x + r.at;
        uint8_t *q = a.q + r.at, *sf = a.sf + r.block + lane;
#pragma unroll 2
        for (int b = 0; b < r.blocks; b += 4, x += 128, q += 128, sf += 4, r.left -= 128) {
            uint32_t w[4], mine = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = 32 * j < r.left ? x[32 * j] : 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t code = ckpt_scale(__reduce_max_sync(0xFFFFFFFFu, w[j] & 0x7FFFu));
                if (32 * j < r.left) q[32 * j] = (uint8_t)cvt_fp8x2<FP8Q_E4M3FN>(__uint_as_float(w[j] << 16) * ckpt_factor(code), 0.0f);
                if (lane == j) mine = code;
            }
            if (lane < min(4, r.blocks - b)) *sf = (uint8_t)mine;
        }
    }
}

template <bool HALF>
__global__ void __launch_bounds__(kThreads) checkpoint_dequantize_kernel(const CkptArgs a) {
    start_behind();
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (i >= a.items) return;
    const int64_t at = ckpt_at<HALF>(a, i);
    if (HALF && at >= a.rows * a.cols) return;
    const uint4 w = *reinterpret_cast<const uint4*>(a.q + at);
    const float s = ckpt_value(a.sf[i >> 1]);
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float v[4];
        ckpt_decode4(in[j], s, v);
        o[2 * j] = cvt_bf16x2(v[0], v[1]), o[2 * j + 1] = cvt_bf16x2(v[2], v[3]);
    }
    st_v8(a.y + at, make_uint4(o[0], o[1], o[2], o[3]), make_uint4(o[4], o[5], o[6], o[7]));
}

__global__ void __launch_bounds__(kThreads) checkpoint_dequantize_rows_kernel(const CkptArgs a) {
    start_behind();
    const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5; i < a.items; i += step) {
        CkptRow r = ckpt_row(a, i);
        const uint8_t *q = a.q + r.at, *sf = a.sf + r.block;
        uint16_t* y = a.y + r.at;
#pragma unroll 2
        for (int b = 0; b < r.blocks; b += 4, q += 128, sf += 4, y += 128, r.left -= 128) {
            uint32_t c[4], s[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (32 * j < r.left) c[j] = q[32 * j], s[j] = sf[j];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (32 * j < r.left) y[32 * j] = (uint16_t)(cvt_bf16x2(f16_lo(fp8x2_to_f16x2<FP8Q_E4M3FN>(c[j])) * ckpt_value(s[j]), 0.0f) & 0xFFFFu);
        }
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

// d/dx of x s(x), s(x) = 1 / (1 + t), t = exp(-2 sqrt(2 / pi) (x + 0.044715 x^3)), for two:
//   s + x s (1 - s) 2 sqrt(2 / pi) (1 + 3 0.044715 x^2)
// 1 - s is off by 2^-24, which counts up to x = 4.2 and makes 2^-20 there; beyond, s is 1 in binary32.  For |x| up to 2^50
// nothing but t and its exponent overflows, and these into 0 and 1.
__device__ __forceinline__ Two gelu_slope2(Two x) {
    const Two x2 = mul_two(x, x);
    const Two u = mul_two(x, fma_two(x2, two(-0.102943239f), two(-2.302208198f)));
    float t0, t1, s0, s1;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t0) : "f"(__uint_as_float((uint32_t)u)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t1) : "f"(__uint_as_float((uint32_t)(u >> 32))));
    const Two t = add_two(two(__float_as_uint(t0), __float_as_uint(t1)), two(1.0f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s0) : "f"(__uint_as_float((uint32_t)t)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s1) : "f"(__uint_as_float((uint32_t)(t >> 32))));
    const Two s = two(__float_as_uint(s0), __float_as_uint(s1));
    const Two rest = fma_two(s, two(-1.0f), two(1.0f));
    return fma_two(mul_two(mul_two(s, x), rest), fma_two(x2, two(0.214064417f), two(1.595769122f)), s);
}
constexpr int kGbCtas = 2;  // of an SM

// x held where gelu_slope2() is 1 and 0; NaN stays.
__device__ __forceinline__ uint32_t near_zero(uint32_t x) {
    float v;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(v) : "f"(__uint_as_float(x)), "f"(64.0f));
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(v) : "f"(v), "f"(-64.0f));
    return __float_as_uint(v);
}

// VEC: sixteen columns side by side a lane; otherwise eight of every 32nd.  Every eighth row a warp.
template <bool VEC>
struct GbGeom {
    static constexpr int kPer = VEC ? 16 : 8;      // columns a lane
    static constexpr int kCols = kPer * 32;        // a CTA
};

// A lane's columns of one row, and where it finds those of its next.
template <bool VEC, bool GELU>
struct GbRow {
    static constexpr int N = GbGeom<VEC>::kPer, S = VEC ? 1 : 8;
    uint32_t y[N / 2], h[N / 4], sf[S];
    __device__ __forceinline__ void load(const uint16_t* dy, const uint8_t* ph, const uint8_t* psf, int64_t left) {
        if constexpr (VEC) {
            uint4 u, v;
            ld_once_v8(dy, u, v);
            y[0] = u.x, y[1] = u.y, y[2] = u.z, y[3] = u.w, y[4] = v.x, y[5] = v.y, y[6] = v.z, y[7] = v.w;
            if (GELU) {
                const uint4 w = *reinterpret_cast<const uint4*>(ph);
                h[0] = w.x, h[1] = w.y, h[2] = w.z, h[3] = w.w;
                sf[0] = *psf;
            }
        } else {
#pragma unroll
            for (int j = 0; j < N / 2; ++j) y[j] = 0;
#pragma unroll
            for (int j = 0; j < N / 4; ++j) h[j] = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j * 32 < left) {
                    y[j >> 1] |= (uint32_t)dy[j * 32] << (j & 1) * 16;
                    if (GELU) {
                        h[j >> 2] |= (uint32_t)ph[j * 32] << (j & 3) * 8;
                        sf[j] = psf[j];
                    }
                } else if (GELU) {
                    sf[j] = 127u;
                }
        }
    }
};

template <int FMT, bool VEC, bool GELU, bool FAST>
__device__ __forceinline__ void gb_rows(const GeluBackArgs& a, const QScale& c, int64_t r0, int64_t r1, int64_t col,
                                        Two (&sum)[GbGeom<VEC>::kPer / 2], uint32_t& m2) {
    constexpr int kWarps = kThreads / 32, N = GbGeom<VEC>::kPer;
    const int64_t left = a.cols - col, step = a.cols * kWarps, sf_step = a.blocks * kWarps;
    const uint16_t* dy = a.dy + r0 * a.cols + col;
    const uint8_t *ph = GELU ? a.h + r0 * a.cols + col : nullptr, *psf = GELU ? a.h_sf + r0 * a.blocks + (col >> 5) : nullptr;
    int64_t at = r0 * a.cols + col;
    GbRow<VEC, GELU> now, ahead;
    int n = (int)((r1 - r0 + kWarps - 1) / kWarps);  // this warp's rows
    if (r0 >= r1) return;
    now.load(dy, ph, psf, left);
#pragma unroll 2
    for (; n > 0; --n, at += step) {
        dy += step;
        if (GELU) ph += step, psf += sf_step;
        if (n > 1) ahead.load(dy, ph, psf, left);
        Two d[N / 2];
#pragma unroll
        for (int j = 0; j < N / 2; ++j) d[j] = widen2(now.y[j]);
        if (GELU) {
            Two x[N / 2];
            bool odd = false;  // a scale of 0 or NaN, or one whose values could leave gelu_slope2()'s range
#pragma unroll
            for (int j = 0; j < (VEC ? 1 : 8); ++j) odd |= now.sf[j] - 1u > 127u + 39u;
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                const uint32_t f = fp8x2_to_f16x2<FP8Q_E4M3FN>(j & 1 ? now.h[j >> 1] >> 16 : now.h[j >> 1]);
                const Two s = VEC ? two(now.sf[0] << 23, now.sf[0] << 23) : two(now.sf[VEC ? 0 : 2 * j] << 23, now.sf[VEC ? 0 : 2 * j + 1] << 23);
                x[j] = mul_two(two(__float_as_uint(f16_lo(f)), __float_as_uint(f16_hi(f))), s);
            }
            if (odd) {
#pragma unroll
                for (int j = 0; j < N / 2; ++j) {
                    float v[4];
                    ckpt_decode4(j & 1 ? now.h[j >> 1] >> 16 : now.h[j >> 1], 1.0f, v);
                    x[j] = two(near_zero(__float_as_uint(v[0] * ckpt_value(now.sf[VEC ? 0 : 2 * j]))), near_zero(__float_as_uint(v[1] * ckpt_value(now.sf[VEC ? 0 : 2 * j + 1]))));
                }
            }
#pragma unroll
            for (int j = 0; j < N / 2; ++j) d[j] = mul_two(d[j], gelu_slope2(x[j]));
        }
        uint32_t w[N / 2], o[N / 4];
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
            sum[j] = add_two(sum[j], d[j]);
            w[j] = cvt_bf16x2(__uint_as_float((uint32_t)d[j]), __uint_as_float((uint32_t)(d[j] >> 32)));
        }
        if (FMT != kNoCodes) {
            const Two s = two(c.s), mr = two(-c.r);
#pragma unroll
            for (int j = 0; j < N / 4; ++j)
                o[j] = FAST ? codes4_fast<FMT & 1>(w[2 * j], w[2 * j + 1], s, mr, c.t2) : quant_quad<FMT & 1, false>(w[2 * j], w[2 * j + 1], c);
        }
        if constexpr (VEC) {
            if (a.dx) {
                st_v4(a.dx + at, make_uint4(w[0], w[1], w[2], w[3]));
                st_v4(a.dx + at + 8, make_uint4(w[4], w[5], w[6], w[7]));
            }
            if (FMT != kNoCodes) st_v4(a.q + at, make_uint4(o[0], o[1], o[2], o[3]));
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j * 32 < left) {
                    if (a.dx) a.dx[at + j * 32] = (uint16_t)(w[j >> 1] >> (j & 1) * 16);
                    if (FMT != kNoCodes) a.q[at + j * 32] = (uint8_t)(o[j >> 2] >> (j & 3) * 8);
                }
        }
#pragma unroll
        for (int j = 0; j < N / 2; ++j) m2 = bf16x2_absmax(m2, w[j]);
        now = ahead;
    }
}

template <int FMT, bool VEC, bool GELU>
__global__ void __launch_bounds__(kThreads, kGbCtas) gelu_backward_kernel(const GeluBackArgs a) {
    constexpr int N = GbGeom<VEC>::kPer, kCols = GbGeom<VEC>::kCols;
    __shared__ float part[kThreads / 32][kCols];
    __shared__ uint32_t red[kThreads / 32];
    start_behind();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t col0 = (int64_t)blockIdx.x * kCols, strip = blockIdx.y;
    const int64_t col = col0 + (VEC ? lane * N : lane);
    const int64_t r0 = strip * a.per_strip + warp, r1 = min((strip + 1) * a.per_strip, a.rows);
    const QScale c = make_qscale_value(a.q ? *a.scale : 1.0f);
    Two sum[N / 2] = {};
    uint32_t m2 = 0;
    if (col < a.cols) {
        if (FMT == kNoCodes || c.fast)
            gb_rows<FMT, VEC, GELU, true>(a, c, r0, r1, col, sum, m2);
        else
            gb_rows<FMT, VEC, GELU, false>(a, c, r0, r1, col, sum, m2);
    }
    if (a.amax) flush_amax(m2, 0, a.amax, red);
    if (!a.d_bias) return;
    // the eight warps' sums in their order
#pragma unroll
    for (int j = 0; j < N; ++j) part[warp][VEC ? lane * N + j : lane + j * 32] = __uint_as_float((uint32_t)(sum[j >> 1] >> (j & 1) * 32));
    __syncthreads();
    for (int i = threadIdx.x; i < kCols; i += kThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) v += part[w][i];
        if (col0 + i < a.cols) (a.strips > 1 ? a.space + strip * a.cols : a.d_bias)[col0 + i] = v;
    }
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
// As many CTAs as are resident, of 32 rows or more; by the sizes alone, so that the sums' order is (and the workspace).
GbStrips gb_strips(int64_t rows, int64_t cols) {
    const int64_t wide = cols % 16 == 0 ? GbGeom<true>::kCols : GbGeom<false>::kCols, across = (cols + wide - 1) / wide;
    int64_t strips = kGbCtas * 152 / across;  // one CTA more than are resident would wait for all of them
    if (strips < 1) strips = 1;
    if (strips > (rows + 31) / 32) strips = (rows + 31) / 32;
    const int64_t per = (rows + strips - 1) / strips;
    return {(rows + per - 1) / per, per};
}

template <int FMT>
fp8q_status launch_gelu_backward(const GeluBackArgs& a, bool vec, cudaStream_t s) {
    const int64_t wide = vec ? GbGeom<true>::kCols : GbGeom<false>::kCols;
    const dim3 grid((unsigned)((a.cols + wide - 1) / wide), (unsigned)a.strips);
    return launch_behind(a.h ? (vec ? gelu_backward_kernel<FMT, true, true> : gelu_backward_kernel<FMT, false, true>)
                             : (vec ? gelu_backward_kernel<FMT, true, false> : gelu_backward_kernel<FMT, false, false>),
                         grid, dim3(kThreads), 0, 1, s, "gelu_backward_kernel", a);
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
    if (a.cols % 16 == 0 && (x & 31u) == 0 && ((uintptr_t)a.q & 15u) == 0 && ((uintptr_t)a.sf & 3u) == 0) {
        const bool half = a.cols % 32 != 0;
        a.across = 2 * a.blocks;
        a.items = a.rows * a.across;
        const int64_t grid = (a.items + kThreads - 1) / kThreads;
        if (grid > 0x7FFFFFFF) return FP8Q_ERR_UNSUPPORTED;
        return launch_behind(back ? (half ? checkpoint_dequantize_kernel<true> : checkpoint_dequantize_kernel<false>)
                                  : (half ? checkpoint_quantize_kernel<true> : checkpoint_quantize_kernel<false>),
                             dim3((unsigned)grid), dim3(kThreads), 0, 1, s, back ? "checkpoint_dequantize_kernel" : "checkpoint_quantize_kernel", a);
    }
    // as many stretches as warps are resident, of four to 32 blocks (1187x2731 with 32: 11.4 us; 8192x4095 with four: 49.9)
    const int64_t fill = a.rows * a.blocks / (64 * (int64_t)sm_count()) / 4 * 4;
    a.stretch = (int32_t)(fill < 4 ? 4 : fill > 32 ? 32 : fill);
    a.across = (a.blocks + a.stretch - 1) / a.stretch;
    a.items = a.rows * a.across;
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
    const bool vec = g->cols % 16 == 0 && ((uintptr_t)g->d_y & 31u) == 0 && (((uintptr_t)g->d_x | (uintptr_t)g->h | (uintptr_t)g->q) & 15u) == 0;
    const fp8q_status rc = !g->q               ? launch_gelu_backward<kNoCodes>(a, vec, s)
                           : g->fmt == FP8Q_E4M3FN ? launch_gelu_backward<FP8Q_E4M3FN>(a, vec, s)
                                                   : launch_gelu_backward<FP8Q_E5M2>(a, vec, s);
    if (rc != FP8Q_OK || !a.d_bias || a.strips == 1) return rc;
    return launch_behind(gelu_backward_sum_kernel, dim3((unsigned)((a.cols + 31) / 32)), dim3(1024), 0, 1, s, "gelu_backward_sum_kernel", a);
}

}  // extern "C"
