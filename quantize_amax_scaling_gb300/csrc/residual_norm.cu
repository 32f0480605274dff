// residual_norm.cu -- the RMS norms after and before a transformer block, fused
// with the block's gate, the residual scale and the quantization of the next
// block's input; forward and backward.
//
// Forward, row by row (H = hidden), binary32:
//   rstd1 = 1 / sqrt(mean(b^2) + eps);  y = b rstd1 g1          (y = b without g1)
//   r'    = bf16(r + (alpha gate) y)
//   rstd2 = 1 / sqrt(mean(r'^2) + eps); h = bf16(r' rstd2 g2)   (of the rounded r')
// Backward, with n1 = b rstd1, n2 = r' rstd2, dn = dh g2, w = alpha gate g1 n1:
//   D    = dr' + rstd2 (dn - n2 c2),     c2 = mean(dn n2)
//   db   = rstd1 (alpha gate g1 D - n1 c1), c1 = mean(w D)
//        = ... with sum w D = sum w (dr' + rstd2 dn) - rstd2 c2 sum w n2,
// so one reduction of three sums gives both means.
//   dg2 = sum dh n2, dg1 = sum alpha gate D n1, dgate = sum alpha D n1 g1.
//
// Both kernels stream HBM; a thread holds 16 columns of a row in registers as
// four groups of four (8-byte loads of the bf16 tensors, 16-byte loads of the
// binary32 weights, both contiguous across a warp; the weights come from L1).

#include "fp4.cuh"

#include <cooperative_groups.h>

#include <initializer_list>

namespace {

constexpr int kRnMaxH = 32768;
constexpr int kOutNone = -1;  // no codes wanted

struct RnArgs {
    const uint16_t *b, *r;
    uint16_t *ro, *h;
    uint8_t *q, *sf;
    const float *post, *pre, *scale;
    const void* gate;
    float *amax, *rstd_post, *rstd_pre;
    int64_t rows, per;
    int32_t H, T, gate_bf16;
    float alpha, eps;
};

__device__ __forceinline__ void widen4(uint2 v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x << 16);
    f[1] = __uint_as_float(v.x & 0xFFFF0000u);
    f[2] = __uint_as_float(v.y << 16);
    f[3] = __uint_as_float(v.y & 0xFFFF0000u);
}

__device__ __forceinline__ void load4(const float* p, float (&f)[4]) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
}

__device__ __forceinline__ void load_gate4(const void* g, int is_bf16, int64_t at, float (&f)[4]) {
    if (is_bf16)
        widen4(__ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(g) + at)), f);
    else
        load4(static_cast<const float*>(g) + at, f);
}

__device__ __forceinline__ void st_v2(void* p, uint2 v) {
    asm volatile("st.global.cs.v2.u32 [%0], {%1,%2};" ::"l"(p), "r"(v.x), "r"(v.y) : "memory");
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sum over the T threads of a row (T a multiple of 32; every thread of the CTA
// calls it).  `part` holds one float a warp and is not used again before the
// next barrier.
__device__ __forceinline__ float row_sum(float v, int T, float* part) {
    v = warp_sum(v);
    if (T == 32) return v;
    const int warp = threadIdx.x >> 5, first = (threadIdx.x / T) * (T >> 5);
    if ((threadIdx.x & 31) == 0) part[warp] = v;
    __syncthreads();
    v = part[first];
    for (int i = 1; i < (T >> 5); ++i) v += part[first + i];
    return v;
}

// Codes of four columns of h (bf16 pairs in w), a warp together, as
// fp8q_quantize_amax or fp8q_fp4_quantize_amax give them.
template <int FMT>
__device__ __forceinline__ void store_codes(const RnArgs& a, const QScale& c8, const Fp4Scale& c4, int64_t row, int64_t col,
                                            bool live, uint2 w) {
    if constexpr (FMT == FP8Q_E4M3FN || FMT == FP8Q_E5M2) {
        const uint32_t o = c8.fast ? quant_quad<FMT, true>(w.x, w.y, c8) : quant_quad<FMT, false>(w.x, w.y, c8);
        if (live && col < a.H) *reinterpret_cast<uint32_t*>(a.q + row * a.H + col) = o;
    } else if constexpr (FMT == FP8Q_MXFP4 || FMT == FP8Q_NVFP4) {
        constexpr int kLanes = Fp4<FMT>::kBlock / 4;  // lanes a block
        const uint32_t m = bf16x2_absmax(w.x, w.y);
        uint32_t am = max(m & 0x7FFFu, (m >> 16) & 0x7FFFu);
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, o));
        const BlockScale b = block_scale<FMT>(am, c4);
        const uint32_t full[8] = {w.x, w.y, 0, 0, 0, 0, 0, 0};
        const uint32_t mine = block_codes<FMT>(full, b).x & 0xFFFFu;
        const uint32_t both = mine | (__shfl_down_sync(0xFFFFFFFFu, mine, 1) << 16);
        const int64_t ld = fp4_row_bytes(a.H);
        if (live && (threadIdx.x & 1) == 0 && col < 2 * ld)
            *reinterpret_cast<uint32_t*>(a.q + row * ld + col / 2) = both;
        uint32_t s = b.code;
        s |= __shfl_down_sync(0xFFFFFFFFu, b.code, kLanes) << 8;
        s |= __shfl_down_sync(0xFFFFFFFFu, b.code, 2 * kLanes) << 16;
        s |= __shfl_down_sync(0xFFFFFFFFu, b.code, 3 * kLanes) << 24;
        const int64_t across = fp4_sf_tiles<FMT>(a.H), tile = col / Fp4<FMT>::kSfCols;
        if (live && (threadIdx.x & 31) % (4 * kLanes) == 0 && tile < across)
            *reinterpret_cast<uint32_t*>(a.sf + ((row / 128) * across + tile) * 512 + (row % 32) * 16 +
                                         (row % 128) / 32 * 4) = s;
    }
}

// U groups of four columns a thread; a row takes T threads, a CTA blockDim / T rows.
template <int FMT, int U>
__global__ void __launch_bounds__(1024) residual_norm_kernel(const RnArgs a) {
    __shared__ float part[2][32];
    __shared__ uint32_t red[32];
    const int T = a.T, t = threadIdx.x % T;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / T) + threadIdx.x / T;
    const bool live = row < a.rows;
    uint2 b[U], r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int col = (u * T + t) * 4;
        b[u] = r[u] = make_uint2(0, 0);
        if (live && col < a.H) {
            r[u] = ld_stream_v2(a.r + row * a.H + col);
            if (a.b) b[u] = ld_stream_v2(a.b + row * a.H + col);
        }
    }
    if (a.b) {
        float rstd = 1.0f;
        if (a.post) {
            float s = 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float f[4];
                widen4(b[u], f);
#pragma unroll
                for (int i = 0; i < 4; ++i) s = fmaf(f[i], f[i], s);
            }
            s = row_sum(s, T, part[0]);
            rstd = __frcp_rn(__fsqrt_rn(s / (float)a.H + a.eps));
            if (a.rstd_post && live && t == 0) a.rstd_post[row] = rstd;
        }
        const int64_t g0 = a.gate && live ? row / a.per * a.H : 0;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int col = (u * T + t) * 4;
            if (!live || col >= a.H) continue;
            float f[4], x[4], p[4] = {1, 1, 1, 1}, g[4] = {1, 1, 1, 1};
            widen4(b[u], f);
            widen4(r[u], x);
            if (a.post) load4(a.post + col, p);
            if (a.gate) load_gate4(a.gate, a.gate_bf16, g0 + col, g);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = fmaf(a.alpha * g[i], f[i] * rstd * p[i], x[i]);
            r[u] = make_uint2(cvt_bf16x2(x[0], x[1]), cvt_bf16x2(x[2], x[3]));
        }
    }
    if (a.ro) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int col = (u * T + t) * 4;
            if (live && col < a.H) st_v2(a.ro + row * a.H + col, r[u]);
        }
    }
    if (!a.pre) return;
    float s = 0.0f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float f[4];
        widen4(r[u], f);
#pragma unroll
        for (int i = 0; i < 4; ++i) s = fmaf(f[i], f[i], s);
    }
    s = row_sum(s, T, part[1]);
    const float rstd = __frcp_rn(__fsqrt_rn(s / (float)a.H + a.eps));
    if (a.rstd_pre && live && t == 0) a.rstd_pre[row] = rstd;
    QScale c8;
    Fp4Scale c4;
    if constexpr (FMT == FP8Q_E4M3FN || FMT == FP8Q_E5M2) c8 = make_qscale(a.scale);
    if constexpr (FMT == FP8Q_MXFP4 || FMT == FP8Q_NVFP4) c4 = make_fp4_scale(a.scale);
    uint32_t m2 = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int col = (u * T + t) * 4;
        uint2 o = make_uint2(0, 0);
        if (live && col < a.H) {
            float f[4], g[4];
            widen4(r[u], f);
            load4(a.pre + col, g);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = f[i] * rstd * g[i];
            o = make_uint2(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]));
            m2 = bf16x2_absmax(m2, bf16x2_absmax(o.x, o.y));
            if (a.h) st_v2(a.h + row * a.H + col, o);
        }
        if constexpr (FMT != kOutNone) store_codes<FMT>(a, c8, c4, row, col, live, o);
    }
    if (a.amax) {
        uint32_t m = max(abs_bits_lo(m2), m2 & 0x7FFF0000u);
        m = __reduce_max_sync(0xFFFFFFFFu, m);
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < (int)(blockDim.x >> 5); ++i) m = max(m, red[i]);
            atomicMax(reinterpret_cast<int*>(a.amax), (int)m);  // ordered like the values (flush_amax)
        }
    }
}

// ----------------------------------------------------------------------------
// Backward

// Rows are dealt out in strips, one strip to each T threads of a CTA (or of a
// cluster of `slices` CTAs, each with up to 4096 columns, for longer rows).  A
// strip keeps its columns' sums of dg1, dg2 and dgate in registers and writes
// them once; residual_norm_sum_kernel adds the strips in order, so a call gives
// the same bits every time.
constexpr int kRnCtas = 304;       // two CTAs on each of 152 SMs
constexpr int kRnSlice = 4096;     // columns a CTA

struct RnStrips {
    int32_t T, slices;
    int64_t per_strip, strips;
};

RnStrips rn_strips(int64_t rows, int32_t H) {
    RnStrips s;
    s.slices = (H + kRnSlice - 1) / kRnSlice;
    s.T = 256;
    while (s.T > 32 && H <= s.T * 8) s.T /= 2;
    const int64_t most = (int64_t)(kRnCtas / s.slices) * (256 / s.T);
    s.per_strip = (rows + most - 1) / most;
    s.strips = s.per_strip ? (rows + s.per_strip - 1) / s.per_strip : 0;
    return s;
}

struct RnBwdArgs {
    const uint16_t *dro, *dh, *ro, *b;
    const float *rstd_pre, *rstd_post, *pre, *post;
    const void* gate;
    uint16_t *dr, *db;
    float *dpre, *dpost;
    void* dgate;
    float* space;  // [strips][H] of dpre, of dpost, then [strips][2][H] of dgate: the group the strip
                   // began in and the one it ended in, where that one began before or goes on after
    int64_t rows, per, per_strip, strips;
    int32_t H, T, gate_bf16, width;  // width: columns a CTA
    float alpha;
};

__device__ __forceinline__ void store_gate4(void* p, int is_bf16, int64_t at, const float (&f)[4]) {
    if (is_bf16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + at) = make_uint2(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]));
    else
        *reinterpret_cast<float4*>(static_cast<float*>(p) + at) = make_float4(f[0], f[1], f[2], f[3]);
}

template <bool CLUSTER>
__global__ void __launch_bounds__(256) residual_norm_backward_kernel(const RnBwdArgs a) {
    namespace cg = cooperative_groups;
    __shared__ float part[2][8][3];
    __shared__ float sums[2][8][3];  // of each CTA of the cluster
    const int T = a.T, t = threadIdx.x % T, warp = threadIdx.x >> 5;
    int slices = 1, slice = 0;
    if (CLUSTER) {
        slices = (int)cg::this_cluster().num_blocks();
        slice = (int)cg::this_cluster().block_rank();
    }
    const int64_t strip = (int64_t)(blockIdx.x / slices) * (256 / T) + threadIdx.x / T;
    const int64_t row0 = strip * a.per_strip, row1 = min(row0 + a.per_strip, a.rows);
    const int c0 = slice * a.width, c1 = min(c0 + a.width, a.H);  // this CTA's columns
    const float inv_h = 1.0f / (float)a.H;

    float apre[4][4] = {}, apost[4][4] = {}, agate[4][4] = {};
    int64_t group = a.gate ? row0 / a.per : 0;
    int64_t gend = a.gate ? (group + 1) * a.per : 0;  // first row behind the group
    bool whole = a.gate && group * a.per >= row0;     // the group began in this strip

    for (int64_t it = 0; it < a.per_strip; ++it) {
        const int64_t row = row0 + it;
        const bool live = row < row1;
        uint2 vb[4], vo[4], vd[4], vh[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int col = c0 + (u * T + t) * 4;
            const int64_t at = row * a.H + col;
            vb[u] = vo[u] = vd[u] = vh[u] = make_uint2(0, 0);
            if (live && col < c1) {
                if (a.dro) vd[u] = ld_stream_v2(a.dro + at);
                if (a.dh) {
                    vh[u] = ld_stream_v2(a.dh + at);
                    vo[u] = ld_stream_v2(a.ro + at);
                }
                if (a.b) vb[u] = ld_stream_v2(a.b + at);
            }
        }
        const float rstd2 = a.dh && live ? a.rstd_pre[row] : 0.0f;
        const float rstd1 = a.post && live ? a.rstd_post[row] : 1.0f;
        const int64_t g0 = group * a.H;
        float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int col = c0 + (u * T + t) * 4;
            if (!live || col >= c1) continue;
            float fo[4], fh[4], fd[4], fb[4], p[4] = {1, 1, 1, 1}, q[4] = {1, 1, 1, 1}, g[4] = {1, 1, 1, 1};
            widen4(vo[u], fo);
            widen4(vh[u], fh);
            widen4(vd[u], fd);
            widen4(vb[u], fb);
            if (a.dh) load4(a.pre + col, q);
            if (a.post) load4(a.post + col, p);
            if (a.gate) load_gate4(a.gate, a.gate_bf16, g0 + col, g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float n2 = fo[i] * rstd2, dn = fh[i] * q[i];
                const float w = a.alpha * g[i] * p[i] * (fb[i] * rstd1);
                s0 = fmaf(dn, n2, s0);
                s1 = fmaf(w, fmaf(rstd2, dn, fd[i]), s1);
                s2 = fmaf(w, n2, s2);
            }
        }
        s0 = warp_sum(s0);
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if (T > 32) {
            float(*pt)[3] = part[it & 1];
            if ((threadIdx.x & 31) == 0) {
                pt[warp][0] = s0;
                pt[warp][1] = s1;
                pt[warp][2] = s2;
            }
            __syncthreads();
            const int first = (threadIdx.x / T) * (T >> 5);
            s0 = pt[first][0];
            s1 = pt[first][1];
            s2 = pt[first][2];
            for (int i = 1; i < (T >> 5); ++i) {
                s0 += pt[first + i][0];
                s1 += pt[first + i][1];
                s2 += pt[first + i][2];
            }
        }
        if (CLUSTER) {
            cg::cluster_group cl = cg::this_cluster();
            if ((int)threadIdx.x < slices) {
                float* d = cl.map_shared_rank(&sums[it & 1][slice][0], threadIdx.x);
                d[0] = s0;
                d[1] = s1;
                d[2] = s2;
            }
            cl.sync();
            s0 = s1 = s2 = 0.0f;
            for (int i = 0; i < slices; ++i) {
                s0 += sums[it & 1][i][0];
                s1 += sums[it & 1][i][1];
                s2 += sums[it & 1][i][2];
            }
        }
        const float c2 = s0 * inv_h;
        const float m1 = a.post ? (s1 - rstd2 * c2 * s2) * inv_h : 0.0f;  // mean(w D); no term without g1
        const bool flush = a.gate && live && (row + 1 == gend || row + 1 == row1);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int col = c0 + (u * T + t) * 4;
            if (!live || col >= c1) continue;
            const int64_t at = row * a.H + col;
            float fo[4], fh[4], D[4], fb[4], p[4] = {1, 1, 1, 1}, q[4] = {1, 1, 1, 1}, g[4] = {1, 1, 1, 1}, e[4];
            widen4(vo[u], fo);
            widen4(vh[u], fh);
            widen4(vd[u], D);
            widen4(vb[u], fb);
            if (a.dh) load4(a.pre + col, q);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float n2 = fo[i] * rstd2;
                D[i] = fmaf(rstd2, fmaf(-n2, c2, fh[i] * q[i]), D[i]);
                apre[u][i] = fmaf(fh[i], n2, apre[u][i]);
            }
            if (a.dr) st_v2(a.dr + at, make_uint2(cvt_bf16x2(D[0], D[1]), cvt_bf16x2(D[2], D[3])));
            if (!a.b) continue;
            if (a.post) load4(a.post + col, p);
            if (a.gate) load_gate4(a.gate, a.gate_bf16, g0 + col, g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float n1 = fb[i] * rstd1, aD = a.alpha * D[i];
                const float dy = aD * g[i];
                apost[u][i] = fmaf(dy, n1, apost[u][i]);
                agate[u][i] = fmaf(aD, n1 * p[i], agate[u][i]);
                e[i] = rstd1 * fmaf(-n1, m1, dy * p[i]);
            }
            if (a.db) st_v2(a.db + at, make_uint2(cvt_bf16x2(e[0], e[1]), cvt_bf16x2(e[2], e[3])));
            if (flush) {
                if (a.dgate) {
                    // a group that lies in this strip whole goes straight out
                    if (whole && (row + 1 == gend || row + 1 == a.rows)) {
                        store_gate4(a.dgate, a.gate_bf16, g0 + col, agate[u]);
                    } else {
                        float* sp = a.space + (2 * a.strips + 2 * strip + (whole ? 1 : 0)) * a.H + col;
                        *reinterpret_cast<float4*>(sp) = make_float4(agate[u][0], agate[u][1], agate[u][2], agate[u][3]);
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) agate[u][i] = 0.0f;
            }
        }
        if (a.gate && row + 1 == gend) {
            ++group;
            gend += a.per;
            whole = true;
        }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int col = c0 + (u * T + t) * 4;
        if (strip >= a.strips || col >= c1) continue;
        if (a.dpre)
            *reinterpret_cast<float4*>(a.space + strip * a.H + col) = make_float4(apre[u][0], apre[u][1], apre[u][2], apre[u][3]);
        if (a.dpost)
            *reinterpret_cast<float4*>(a.space + (a.strips + strip) * a.H + col) =
                make_float4(apost[u][0], apost[u][1], apost[u][2], apost[u][3]);
    }
    if (CLUSTER) cg::this_cluster().sync();  // nobody's `sums` goes away while another CTA may write it
}

// 32 columns a CTA, 32 strips at a time: blockIdx.y 0 adds dpre, 1 dpost, and
// 2 + s the group of dgate that lies across the border behind strip s, if it
// began in that strip.
__global__ void __launch_bounds__(1024) residual_norm_sum_kernel(const RnBwdArgs a) {
    __shared__ float t[32][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    const int what = blockIdx.y;
    float v = 0.0f;
    int64_t group = 0;
    if (what < 2) {
        if (what == 0 ? !a.dpre : !a.dpost) return;
        if (col < a.H)
            for (int64_t s = w; s < a.strips; s += 32) v += a.space[(what * a.strips + s) * a.H + col];
    } else {
        const int64_t s0 = what - 2, border = (s0 + 1) * a.per_strip;
        group = border / a.per;
        const int64_t begin = group * a.per, end = min(begin + a.per, a.rows);
        if (begin == border || begin < s0 * a.per_strip) return;
        const int64_t s1 = (end - 1) / a.per_strip;
        const float* sp = a.space + 2 * a.strips * a.H;
        if (col < a.H) {
            // its first rows are the tail of strip s0, the rest the heads of those that follow
            for (int64_t s = s0 + w; s <= s1; s += 32) v += sp[(2 * s + (s == s0 ? 1 : 0)) * a.H + col];
        }
    }
    t[w][lane] = v;
    __syncthreads();
    if (w == 0 && col < a.H) {
#pragma unroll
        for (int i = 1; i < 32; ++i) v += t[i][lane];
        if (what == 0)
            a.dpre[col] = v;
        else if (what == 1)
            a.dpost[col] = v;
        else if (a.gate_bf16)
            static_cast<uint16_t*>(a.dgate)[group * a.H + col] = (uint16_t)(cvt_bf16x2(v, 0.0f) & 0xFFFFu);
        else
            static_cast<float*>(a.dgate)[group * a.H + col] = v;
    }
}

template <int FMT>
fp8q_status launch_forward(const RnArgs& a, dim3 grid, dim3 block, cudaStream_t s) {
    auto kern = a.H > 16384 ? residual_norm_kernel<FMT, 8> : residual_norm_kernel<FMT, 4>;
    return launch_kernel(kern, grid, block, 0, s, "residual_norm_kernel", a);
}

bool misaligned(std::initializer_list<const void*> ps, uintptr_t mask) {
    uintptr_t v = 0;
    for (const void* p : ps) v |= (uintptr_t)p;
    return (v & mask) != 0;
}

}  // namespace

extern "C" {

fp8q_status fp8q_residual_norm_quantize_amax(const fp8q_residual_norm* n, void* stream) {
    if (!n) return FP8Q_ERR_INVALID_ARG;
    const bool fp4 = valid_fp4(n->fmt);
    if ((!fp4 && !valid_fmt(n->fmt)) || n->rows < 0 || n->hidden < 16 || n->hidden % 16 != 0) return FP8Q_ERR_INVALID_ARG;
    if (n->hidden > kRnMaxH || n->rows > kFp4MaxDim) return FP8Q_ERR_UNSUPPORTED;
    if (n->rows == 0) return FP8Q_OK;
    if (!n->residual || (n->block && !n->residual_out) || (!n->residual_out && !n->pre_weight)) return FP8Q_ERR_INVALID_ARG;
    if (!n->block && (n->post_weight || n->gate)) return FP8Q_ERR_INVALID_ARG;
    if (n->gate && n->rows_per_gate < 1) return FP8Q_ERR_INVALID_ARG;
    if ((n->pre_weight != nullptr) != (n->h || n->q)) return FP8Q_ERR_INVALID_ARG;
    if (n->q && ((fp4 && !n->sf) || (!fp4 && (n->sf || !n->scale)) || (n->fmt == FP8Q_MXFP4 && n->scale)))
        return FP8Q_ERR_INVALID_ARG;
    if (!n->q && n->sf) return FP8Q_ERR_INVALID_ARG;
    if (!n->pre_weight && n->amax) return FP8Q_ERR_INVALID_ARG;
    if (misaligned({n->scale, n->amax, n->rstd_post, n->rstd_pre}, 3)) return FP8Q_ERR_INVALID_ARG;
    if (misaligned({n->residual, n->residual_out, n->block, n->post_weight, n->pre_weight, n->gate, n->h, n->q, n->sf}, 15))
        return FP8Q_ERR_UNSUPPORTED;
    RnArgs a;
    a.b = static_cast<const uint16_t*>(n->block);
    a.r = static_cast<const uint16_t*>(n->residual);
    a.ro = static_cast<uint16_t*>(n->residual_out);
    a.h = static_cast<uint16_t*>(n->h);
    a.q = n->q;
    a.sf = n->sf;
    a.post = n->post_weight;
    a.pre = n->pre_weight;
    a.scale = n->scale;
    a.gate = n->gate;
    a.amax = n->amax;
    a.rstd_post = n->rstd_post;
    a.rstd_pre = n->rstd_pre;
    a.rows = n->rows;
    a.per = n->rows_per_gate;
    a.H = n->hidden;
    a.gate_bf16 = n->gate_is_bf16 != 0;
    a.alpha = n->alpha;
    a.eps = n->eps;
    a.T = 1024;
    while (a.T > 32 && a.H <= a.T * 8) a.T /= 2;
    const int block = a.T < 256 ? 256 : a.T, per_cta = block / a.T;
    const dim3 grid((unsigned)((a.rows + per_cta - 1) / per_cta));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!a.q) return launch_forward<kOutNone>(a, grid, dim3(block), s);
    switch (n->fmt) {
        case FP8Q_E4M3FN: return launch_forward<FP8Q_E4M3FN>(a, grid, dim3(block), s);
        case FP8Q_E5M2: return launch_forward<FP8Q_E5M2>(a, grid, dim3(block), s);
        case FP8Q_MXFP4: return launch_forward<FP8Q_MXFP4>(a, grid, dim3(block), s);
        default: return launch_forward<FP8Q_NVFP4>(a, grid, dim3(block), s);
    }
}

int64_t fp8q_residual_norm_backward_workspace(int64_t rows, int32_t hidden, int64_t rows_per_gate) {
    if (rows <= 0 || hidden <= 0) return 0;
    const RnStrips st = rn_strips(rows, hidden);
    return (rows_per_gate > 1 ? 4 : 2) * st.strips * hidden * (int64_t)sizeof(float);
}

fp8q_status fp8q_residual_norm_backward(const fp8q_residual_norm_grad* n, void* stream) {
    if (!n || n->rows < 0 || n->hidden < 16 || n->hidden % 16 != 0) return FP8Q_ERR_INVALID_ARG;
    if (n->hidden > kRnMaxH || n->rows > kFp4MaxDim) return FP8Q_ERR_UNSUPPORTED;
    if (n->rows == 0) return FP8Q_OK;
    if (!n->d_residual_out && !n->d_h) return FP8Q_ERR_INVALID_ARG;
    if (n->d_h ? (!n->residual_out || !n->rstd_pre || !n->pre_weight) : (n->pre_weight || n->d_pre_weight != nullptr))
        return FP8Q_ERR_INVALID_ARG;
    if (!n->block && (n->post_weight || n->gate || n->d_block)) return FP8Q_ERR_INVALID_ARG;
    if (n->post_weight ? !n->rstd_post : n->d_post_weight != nullptr) return FP8Q_ERR_INVALID_ARG;
    if (n->gate ? n->rows_per_gate < 1 : n->d_gate != nullptr) return FP8Q_ERR_INVALID_ARG;
    const RnStrips st = rn_strips(n->rows, n->hidden);
    const int64_t need = fp8q_residual_norm_backward_workspace(n->rows, n->hidden, n->gate ? n->rows_per_gate : 0);
    const bool spread = n->d_gate && n->rows_per_gate > 1;  // groups that may lie across strips
    if ((n->d_pre_weight || n->d_post_weight || spread) && (!n->workspace || n->workspace_bytes < need)) return FP8Q_ERR_INVALID_ARG;
    if (misaligned({n->rstd_pre, n->rstd_post}, 3)) return FP8Q_ERR_INVALID_ARG;
    if (misaligned({n->d_residual_out, n->d_h, n->residual_out, n->block, n->pre_weight, n->post_weight, n->gate, n->d_residual,
                    n->d_block, n->d_pre_weight, n->d_post_weight, n->d_gate, n->workspace}, 15))
        return FP8Q_ERR_UNSUPPORTED;
    RnBwdArgs a;
    a.dro = static_cast<const uint16_t*>(n->d_residual_out);
    a.dh = static_cast<const uint16_t*>(n->d_h);
    a.ro = static_cast<const uint16_t*>(n->residual_out);
    a.b = static_cast<const uint16_t*>(n->block);
    a.rstd_pre = n->rstd_pre;
    a.rstd_post = n->rstd_post;
    a.pre = n->pre_weight;
    a.post = n->post_weight;
    a.gate = n->gate;
    a.dr = static_cast<uint16_t*>(n->d_residual);
    a.db = static_cast<uint16_t*>(n->d_block);
    a.dpre = n->d_pre_weight;
    a.dpost = n->d_post_weight;
    a.dgate = n->d_gate;
    a.space = static_cast<float*>(n->workspace);
    a.rows = n->rows;
    a.per = n->rows_per_gate;
    a.per_strip = st.per_strip;
    a.strips = st.strips;
    a.H = n->hidden;
    a.T = st.T;
    a.gate_bf16 = n->gate_is_bf16 != 0;
    a.alpha = n->alpha;
    // slices of equal width, whole groups of four columns a thread
    a.width = ((n->hidden + st.slices - 1) / st.slices + 15) / 16 * 16;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int64_t per_cta = 256 / st.T;
    const unsigned ctas = (unsigned)((st.strips + per_cta - 1) / per_cta) * (unsigned)st.slices;
    fp8q_status rc;
    if (st.slices == 1) {
        rc = launch_kernel(residual_norm_backward_kernel<false>, dim3(ctas), dim3(256), 0, s, "residual_norm_backward_kernel", a);
    } else {
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)st.slices;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(ctas);
        cfg.blockDim = dim3(256);
        cfg.stream = s;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaLaunchKernelEx(&cfg, residual_norm_backward_kernel<true>, a);
        rc = e == cudaSuccess ? FP8Q_OK : cuda_fail(e, "residual_norm_backward_kernel");
    }
    if (rc != FP8Q_OK || (!a.dpre && !a.dpost && !spread)) return rc;
    // borders that a group lies across there are only where strips are not whole groups
    const bool borders = spread && st.strips > 1 && st.per_strip % n->rows_per_gate != 0;
    const dim3 grid((unsigned)((n->hidden + 31) / 32), 2u + (borders ? (unsigned)(st.strips - 1) : 0u));
    return launch_kernel(residual_norm_sum_kernel, grid, dim3(1024), 0, s, "residual_norm_sum_kernel", a);
}

}  // extern "C"
