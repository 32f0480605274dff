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
// Both kernels stream HBM.  Rows are dealt out in strips of consecutive rows, a
// strip to each T threads; a thread has 16 (or 32) columns of a row, in groups of
// eight, and brings the next rows of its strip into shared memory by asynchronous
// copies of its own (it alone reads them, so they need no barrier), while the
// weights of its columns stay in registers.

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
    int64_t rows, per, per_strip;
    int32_t H, T, gate_bf16;
    float alpha, eps;
};

__device__ __forceinline__ void widen8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
    return make_uint4(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]), cvt_bf16x2(f[4], f[5]), cvt_bf16x2(f[6], f[7]));
}

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p)), w = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    f[4] = w.x; f[5] = w.y; f[6] = w.z; f[7] = w.w;
}

__device__ __forceinline__ void load_gate8(const void* g, int is_bf16, int64_t at, float (&f)[8]) {
    if (is_bf16)
        widen8(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g) + at)), f);
    else
        load8(static_cast<const float*>(g) + at, f);
}

// Sixteen bytes from global to shared memory, or zeros (then nothing is read).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 ld_shared(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
// Eight gate values that lie in the ring: one 16-byte slot of bf16, or two of binary32.
__device__ __forceinline__ void ring_gate8(uint32_t at, uint32_t step, int is_bf16, float (&f)[8]) {
    const uint4 v = ld_shared(at);
    if (is_bf16) {
        widen8(v, f);
    } else {
        const uint4 w = ld_shared(at + step);
        f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y); f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
        f[4] = __uint_as_float(w.x); f[5] = __uint_as_float(w.y); f[6] = __uint_as_float(w.z); f[7] = __uint_as_float(w.w);
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// Sum over the T threads of a row (T a multiple of 32; every thread of the CTA
// calls it).  `part` holds one float a warp and is not written again before the
// next barrier but one.
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

// Codes of eight columns of h, a warp together, as fp8q_quantize_amax or
// fp8q_fp4_quantize_amax give them.
template <int FMT>
__device__ __forceinline__ void store_codes(const RnArgs& a, const QScale& c8, const Fp4Scale& c4, int64_t row, int col, bool live,
                                            const uint4& w) {
    if constexpr (FMT == FP8Q_E4M3FN || FMT == FP8Q_E5M2) {
        uint2 o;
        if (c8.fast)
            o = make_uint2(quant_quad<FMT, true>(w.x, w.y, c8), quant_quad<FMT, true>(w.z, w.w, c8));
        else
            o = make_uint2(quant_quad<FMT, false>(w.x, w.y, c8), quant_quad<FMT, false>(w.z, w.w, c8));
        if (live && col < a.H) st_v2(a.q + row * a.H + col, o);
    } else if constexpr (FMT == FP8Q_MXFP4 || FMT == FP8Q_NVFP4) {
        constexpr int kLanes = Fp4<FMT>::kBlock / 8;  // lanes a block
        const uint32_t m = bf16x2_absmax(bf16x2_absmax(w.x, w.y), bf16x2_absmax(w.z, w.w));
        uint32_t am = max(m & 0x7FFFu, (m >> 16) & 0x7FFFu);
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, o));
        const BlockScale b = block_scale<FMT>(am, c4);
        const uint32_t full[8] = {w.x, w.y, w.z, w.w, 0, 0, 0, 0};
        const uint32_t mine = block_codes<FMT>(full, b).x;
        const int64_t ld = fp4_row_bytes(a.H);
        if (live && col < 2 * ld) *reinterpret_cast<uint32_t*>(a.q + row * ld + col / 2) = mine;
        uint32_t s = b.code;
        s |= __shfl_down_sync(0xFFFFFFFFu, b.code, kLanes) << 8;
        s |= __shfl_down_sync(0xFFFFFFFFu, b.code, 2 * kLanes) << 16;
        s |= __shfl_down_sync(0xFFFFFFFFu, b.code, 3 * kLanes) << 24;
        const int64_t across = fp4_sf_tiles<FMT>(a.H), tile = col / Fp4<FMT>::kSfCols;
        if (live && (threadIdx.x & 31) % (4 * kLanes) == 0 && tile < across)
            *reinterpret_cast<uint32_t*>(a.sf + ((row / 128) * across + tile) * 512 + (row % 32) * 16 + (row % 128) / 32 * 4) = s;
    }
}

// U groups of eight columns a thread.  WREG: the weights stay in registers (rows
// of up to 512 threads); longer rows, with 64 registers a thread, read them from
// L1 for each row, and the longest have room for one row ahead in shared memory.
template <int FMT, int U, bool WREG>
__global__ void __launch_bounds__(WREG ? 512 : 1024) residual_norm_kernel(const RnArgs a) {
    extern __shared__ __align__(16) uint8_t ring_raw[];
    __shared__ float part[4][32];
    __shared__ uint32_t red[32];
    const int T = a.T, t = threadIdx.x % T;
    const int64_t strip = (int64_t)blockIdx.x * (blockDim.x / T) + threadIdx.x / T;
    const int64_t row0 = strip * a.per_strip, row1 = min(row0 + a.per_strip, a.rows);
    constexpr int kStages = U == 2 ? 3 : 1;  // rows under way
    const bool ring_gate = WREG && a.gate && a.per == 1;
    const uint32_t step = blockDim.x * 16;  // from one slot to the next
    const uint32_t slots = 1 + (a.b != nullptr) + (ring_gate ? (a.gate_bf16 ? 1 : 2) : 0);
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(ring_raw)) + threadIdx.x * 16;

    auto fetch = [&](int64_t row, uint32_t stage) {
        const bool live = row < row1;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int col = (u * T + t) * 8;
            const bool on = live && col < a.H;
            const int64_t at = on ? row * a.H + col : 0;
            uint32_t dst = ring + (stage * U + u) * slots * step;
            copy16(dst, a.r + at, on);
            if (a.b) copy16(dst += step, a.b + at, on);
            if (ring_gate) {
                if (a.gate_bf16) {
                    copy16(dst += step, static_cast<const uint16_t*>(a.gate) + at, on);
                } else {
                    copy16(dst += step, static_cast<const float*>(a.gate) + at, on);
                    copy16(dst += step, static_cast<const float*>(a.gate) + at + (on ? 4 : 0), on);
                }
            }
        }
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) fetch(i < a.per_strip ? row0 + i : row1, i);

    QScale c8;
    Fp4Scale c4;
    if constexpr (FMT == FP8Q_E4M3FN || FMT == FP8Q_E5M2) c8 = make_qscale(a.scale);
    if constexpr (FMT == FP8Q_MXFP4 || FMT == FP8Q_NVFP4) c4 = make_fp4_scale(a.scale);
    // alpha * gate * post of a column, without the gate where it comes with the row
    auto weight = [&](int u, int64_t group, float (&w)[8]) {
        const int col = (u * T + t) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = a.alpha;
        if (col >= a.H) return;
        float f[8];
        if (a.gate && !ring_gate) {
            load_gate8(a.gate, a.gate_bf16, group * a.H + col, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] *= f[i];
        }
        if (a.post) {
            load8(a.post + col, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] *= f[i];
        }
    };
    float W[WREG ? U : 1][8], P[WREG ? U : 1][8];
    int64_t group = a.gate && !ring_gate ? row0 / a.per : 0, gend = a.gate && !ring_gate ? (group + 1) * a.per : a.rows;
    if constexpr (WREG) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (a.b && row0 < a.rows) weight(u, group, W[u]);
            if (a.pre && (u * T + t) * 8 < a.H) load8(a.pre + (u * T + t) * 8, P[u]);
        }
    }
    const float inv_h = 1.0f / (float)a.H;
    uint32_t m2 = 0, stage = 0;
    for (int64_t it = 0; it < a.per_strip; ++it) {
        const int64_t row = row0 + it;
        const bool live = row < row1;
        if (row == gend) {
            ++group;
            gend += a.per;
            if constexpr (WREG) {
                if (live)
#pragma unroll
                    for (int u = 0; u < U; ++u) weight(u, group, W[u]);
            }
        }
        copies_wait<kStages - 1>();
        uint4 r[U], b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t at = ring + (stage * U + u) * slots * step;
            r[u] = ld_shared(at);
            b[u] = a.b ? ld_shared(at + step) : make_uint4(0, 0, 0, 0);
        }
        if (a.b) {
            float rstd = 1.0f;
            if (a.post) {
                float s = 0.0f;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float f[8];
                    widen8(b[u], f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) s = fmaf(f[i], f[i], s);
                }
                s = row_sum(s, T, part[(it & 1) * 2]);
                rstd = __frcp_rn(__fsqrt_rn(fmaf(s, inv_h, a.eps)));
                if (a.rstd_post && live && t == 0) a.rstd_post[row] = rstd;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float f[8], x[8], g[8], w[8];
                widen8(b[u], f);
                widen8(r[u], x);
                if constexpr (WREG) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = W[u][i];
                } else if (live) {
                    weight(u, group, w);
                }
                if (ring_gate) {
                    ring_gate8(ring + ((stage * U + u) * slots + 2) * step, step, a.gate_bf16, g);
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] *= g[i];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = fmaf(w[i], f[i] * rstd, x[i]);
                r[u] = narrow8(x);
            }
        }
        float s = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int col = (u * T + t) * 8;
            if (!live || col >= a.H) r[u] = make_uint4(0, 0, 0, 0);
            float f[8];
            widen8(r[u], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) s = fmaf(f[i], f[i], s);
        }
        // everything of this stage has been used: the row after the next ones into it
        fetch(it + kStages < a.per_strip ? row + kStages : row1, stage);
        if (++stage == kStages) stage = 0;
        if (a.ro && live) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int col = (u * T + t) * 8;
                if (col < a.H) st_v4(a.ro + row * a.H + col, r[u]);
            }
        }
        if (!a.pre) continue;
        s = row_sum(s, T, part[(it & 1) * 2 + 1]);
        const float rstd = __frcp_rn(__fsqrt_rn(fmaf(s, inv_h, a.eps)));
        if (a.rstd_pre && live && t == 0) a.rstd_pre[row] = rstd;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int col = (u * T + t) * 8;
            uint4 o = make_uint4(0, 0, 0, 0);
            if (live && col < a.H) {
                float f[8];
                widen8(r[u], f);
                if constexpr (WREG) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = f[i] * rstd * P[u][i];
                } else {
                    float g[8];
                    load8(a.pre + col, g);
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = f[i] * rstd * g[i];
                }
                o = narrow8(f);
                m2 = bf16x2_absmax(m2, bf16x2_absmax(bf16x2_absmax(o.x, o.y), bf16x2_absmax(o.z, o.w)));
                if (a.h) st_v4(a.h + row * a.H + col, o);
            }
            if constexpr (FMT != kOutNone) store_codes<FMT>(a, c8, c4, row, col, live, o);
        }
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
    copies_wait<0>();
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

__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

__device__ __forceinline__ void store_gate8(void* p, int is_bf16, int64_t at, const float (&f)[8]) {
    if (is_bf16)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = narrow8(f);
    else
        store8(static_cast<float*>(p) + at, f);
}

// Per row: one pass for the three sums, one for the gradients, both from shared
// memory (kept in registers between them, a row would spill).  With X = D n1 and W = alpha gate g1 of a column, a row
// adds X to the one sum S that dgate and dg1 share: a gate's row of dgate is
// alpha g1 S, and dg1 takes alpha gate S whenever a gate's rows end.  RING_GATE:
// each row has its own gate, which comes with it.
template <bool CLUSTER, bool RING_GATE>
__global__ void __launch_bounds__(256, 2) residual_norm_backward_kernel(const RnBwdArgs a) {
    namespace cg = cooperative_groups;
    constexpr int kStages = RING_GATE ? 2 : 3;
    extern __shared__ __align__(16) uint8_t ring_raw[];
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
    // ring: a stage holds, for each of two groups of eight columns, a slot of b, r', dr', dh and one
    // or two of the gate; behind it this thread's sums of dg1
    constexpr uint32_t kStep = 256 * 16;
    const uint32_t slots = RING_GATE ? (a.gate_bf16 ? 5 : 6) : 4;
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(ring_raw)) + threadIdx.x * 16;
    float4* const post_sum = reinterpret_cast<float4*>(ring_raw + kStages * 2 * slots * kStep) + threadIdx.x;

    auto fetch = [&](int64_t row, uint32_t stage) {
        const bool live = row < row1;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int col = c0 + (u * T + t) * 8;
            const bool on = live && col < c1;
            const int64_t at = on ? row * a.H + col : 0;
            const uint32_t dst = ring + (stage * 2 + u) * slots * kStep;
            if (a.b) copy16(dst, a.b + at, on);
            if (a.dh) {
                copy16(dst + kStep, a.ro + at, on);
                copy16(dst + 3 * kStep, a.dh + at, on);
            }
            if (a.dro) copy16(dst + 2 * kStep, a.dro + at, on);
            if (RING_GATE) {
                if (a.gate_bf16) {
                    copy16(dst + 4 * kStep, static_cast<const uint16_t*>(a.gate) + at, on);
                } else {
                    copy16(dst + 4 * kStep, static_cast<const float*>(a.gate) + at, on);
                    copy16(dst + 5 * kStep, static_cast<const float*>(a.gate) + at + (on ? 4 : 0), on);
                }
            }
        }
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) fetch(i < a.per_strip ? row0 + i : row1, i);

    int64_t group = a.gate ? row0 / a.per : 0;
    int64_t gend = a.gate ? (group + 1) * a.per : a.rows;  // first row behind the group
    bool whole = a.gate && group * a.per >= row0;          // the group began in this strip
    float Q[2][8], W[2][8], S[2][8] = {}, apre[2][8] = {};
    // alpha * gate * post of a column, without a gate that comes with the row
    auto weight = [&](int u) {
        const int col = c0 + (u * T + t) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) W[u][i] = a.alpha;
        if (col >= c1) return;
        float f[8];
        if (a.post) {
            load8(a.post + col, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) W[u][i] *= f[i];
        }
        if (a.gate && !RING_GATE) {
            load_gate8(a.gate, a.gate_bf16, group * a.H + col, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) W[u][i] *= f[i];
        }
    };
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int col = c0 + (u * T + t) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) Q[u][i] = 0.0f;
        if (a.dh && col < c1) load8(a.pre + col, Q[u]);
        if (row0 < a.rows) weight(u);
        post_sum[(2 * u) * 256] = post_sum[(2 * u + 1) * 256] = make_float4(0, 0, 0, 0);
    }

    uint32_t stage = 0;
    for (int64_t it = 0; it < a.per_strip; ++it) {
        const int64_t row = row0 + it;
        const bool live = row < row1;
        const float rstd2 = a.dh && live ? __ldg(a.rstd_pre + row) : 0.0f;
        const float rstd1 = a.post && live ? __ldg(a.rstd_post + row) : 1.0f;
        copies_wait<kStages - 1>();
        const uint32_t at_stage = ring + stage * 2 * slots * kStep;
        const uint4 none = make_uint4(0, 0, 0, 0);
        float s0 = 0.0f, s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t at = at_stage + u * slots * kStep;
            float fb[8], fo[8], fd[8], fh[8], g[8];
            widen8(a.b ? ld_shared(at) : none, fb);
            widen8(a.dh ? ld_shared(at + kStep) : none, fo);
            widen8(a.dro ? ld_shared(at + 2 * kStep) : none, fd);
            widen8(a.dh ? ld_shared(at + 3 * kStep) : none, fh);
            if (RING_GATE) ring_gate8(at + 4 * kStep, kStep, a.gate_bf16, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float n2 = fo[i] * rstd2, dn = fh[i] * Q[u][i];
                float w = W[u][i] * (fb[i] * rstd1);
                if (RING_GATE) w *= g[i];
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
        const bool flush = live && a.b && (row + 1 == gend || row + 1 == row1);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int col = c0 + (u * T + t) * 8;
            const bool on = live && col < c1;
            const int64_t at = row * a.H + col;
            float fb[8], fo[8], D[8], fh[8], e[8], g[8];
            const uint32_t from = at_stage + u * slots * kStep;
            widen8(a.b ? ld_shared(from) : none, fb);
            widen8(a.dh ? ld_shared(from + kStep) : none, fo);
            widen8(a.dro ? ld_shared(from + 2 * kStep) : none, D);
            widen8(a.dh ? ld_shared(from + 3 * kStep) : none, fh);
            if (RING_GATE) ring_gate8(from + 4 * kStep, kStep, a.gate_bf16, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float n2 = fo[i] * rstd2;
                D[i] = fmaf(rstd2, fmaf(-n2, c2, fh[i] * Q[u][i]), D[i]);
                apre[u][i] = fmaf(fh[i], n2, apre[u][i]);
                const float n1 = fb[i] * rstd1;
                S[u][i] = fmaf(D[i], n1, S[u][i]);
                const float w = RING_GATE ? W[u][i] * g[i] : W[u][i];
                e[i] = rstd1 * fmaf(-n1, m1, D[i] * w);
            }
            if (on && a.dr) st_v4(a.dr + at, narrow8(D));
            if (on && a.db) st_v4(a.db + at, narrow8(e));
            if (flush && on) {
                float p[8], f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) p[i] = 1.0f;
                if (a.post) load8(a.post + col, p);
                if (a.gate && !RING_GATE) load_gate8(a.gate, a.gate_bf16, group * a.H + col, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    S[u][i] *= a.alpha;
                    f[i] = a.gate ? S[u][i] * g[i] : S[u][i];
                    p[i] *= S[u][i];
                    S[u][i] = 0.0f;
                }
                float4 lo = post_sum[(2 * u) * 256], hi = post_sum[(2 * u + 1) * 256];
                lo.x += f[0]; lo.y += f[1]; lo.z += f[2]; lo.w += f[3];
                hi.x += f[4]; hi.y += f[5]; hi.z += f[6]; hi.w += f[7];
                post_sum[(2 * u) * 256] = lo;
                post_sum[(2 * u + 1) * 256] = hi;
                if (a.dgate) {
                    // a group that lies in this strip whole goes straight out
                    if (whole && (row + 1 == gend || row + 1 == a.rows))
                        store_gate8(a.dgate, a.gate_bf16, group * a.H + col, p);
                    else
                        store8(a.space + (2 * a.strips + 2 * strip + (whole ? 1 : 0)) * a.H + col, p);
                }
            }
        }
        // this stage has been used: the row after the next ones into it
        fetch(it + kStages < a.per_strip ? row + kStages : row1, stage);
        if (++stage == kStages) stage = 0;
        if (a.gate && row + 1 == gend) {
            ++group;
            gend += a.per;
            whole = true;
            if (!RING_GATE && row + 1 < row1) {
                weight(0);
                weight(1);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int col = c0 + (u * T + t) * 8;
        if (strip < a.strips && col < c1) {
            if (a.dpre) store8(a.space + strip * a.H + col, apre[u]);
            if (a.dpost) {
                float4* o = reinterpret_cast<float4*>(a.space + (a.strips + strip) * a.H + col);
                o[0] = post_sum[(2 * u) * 256];
                o[1] = post_sum[(2 * u + 1) * 256];
            }
        }
    }
    copies_wait<0>();
    if (CLUSTER) cg::this_cluster().sync();  // nobody's `sums` goes away while another CTA may write it
}

// 32 columns a CTA, 32 strips at a time: blockIdx.y 0 adds dpre, 1 dpost, and from
// 2 on a row of dgate that lies in several strips: row blockIdx.y - 2, where gates
// span strips, or else the one across the border behind strip blockIdx.y - 2.
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
        group = a.per >= a.per_strip ? what - 2 : (what - 1) * a.per_strip / a.per;
        const int64_t begin = group * a.per, end = min(begin + a.per, a.rows);
        const int64_t s0 = begin / a.per_strip, s1 = (end - 1) / a.per_strip;
        if (s0 == s1 || (a.per < a.per_strip && s0 != what - 2)) return;  // in one strip, or another border's
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

template <bool CLUSTER, bool RING_GATE>
fp8q_status launch_backward(const RnBwdArgs& a, unsigned ctas, unsigned slices, cudaStream_t s) {
    static std::atomic<uint64_t> devices{0};
    auto kern = residual_norm_backward_kernel<CLUSTER, RING_GATE>;
    const size_t smem = ((RING_GATE ? 2 * 2 * (a.gate_bf16 ? 5 : 6) : 3 * 2 * 4) + 4) * 4096;
    cudaError_t e = allow_smem(kern, 112 * 1024, devices);
    if (e != cudaSuccess) return cuda_fail(e, "residual_norm_backward_kernel setup");
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = slices;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = CLUSTER ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, kern, a);
    return e == cudaSuccess ? FP8Q_OK : cuda_fail(e, "residual_norm_backward_kernel");
}

template <int FMT>
fp8q_status launch_forward(RnArgs a, cudaStream_t s) {
    const int U = a.H > 16384 ? 4 : 2;
    a.T = 1024;
    while (a.T > 32 && a.H <= a.T * 4 * U) a.T /= 2;
    const int block = a.T < 256 ? 256 : a.T, per_cta = block / a.T;
    // strips: two CTAs of 256 threads an SM, one of 512 or 1024
    const int64_t most = (int64_t)(block == 256 ? 2 : 1) * 152 * per_cta;
    a.per_strip = (a.rows + most - 1) / most;
    const int64_t strips = (a.rows + a.per_strip - 1) / a.per_strip;
    const int slots = 1 + (a.b != nullptr) + (a.T < 1024 && a.gate && a.per == 1 ? (a.gate_bf16 ? 1 : 2) : 0);
    const size_t smem = (size_t)(U == 2 ? 3 : 1) * U * slots * block * 16;
    const dim3 grid((unsigned)((strips + per_cta - 1) / per_cta));
    static std::atomic<uint64_t> devices[3];
    auto kern = U == 4 ? residual_norm_kernel<FMT, 4, false> : a.T == 1024 ? residual_norm_kernel<FMT, 2, false> : residual_norm_kernel<FMT, 2, true>;
    // 3 stages of 4 slots of 512 threads, or of 2 slots of 1024
    const cudaError_t e = allow_smem(kern, 192 * 1024, devices[U == 4 ? 2 : a.T == 1024 ? 1 : 0]);
    if (e != cudaSuccess) return cuda_fail(e, "residual_norm_kernel setup");
    return launch_kernel(kern, grid, dim3(block), smem, s, "residual_norm_kernel", a);
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
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (!a.q) return launch_forward<kOutNone>(a, s);
    switch (n->fmt) {
        case FP8Q_E4M3FN: return launch_forward<FP8Q_E4M3FN>(a, s);
        case FP8Q_E5M2: return launch_forward<FP8Q_E5M2>(a, s);
        case FP8Q_MXFP4: return launch_forward<FP8Q_MXFP4>(a, s);
        default: return launch_forward<FP8Q_NVFP4>(a, s);
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
    const bool ring_gate = a.gate && a.per == 1;
    const unsigned slices = (unsigned)st.slices;
    const fp8q_status rc = slices == 1 ? (ring_gate ? launch_backward<false, true>(a, ctas, 1, s) : launch_backward<false, false>(a, ctas, 1, s))
                                       : (ring_gate ? launch_backward<true, true>(a, ctas, slices, s) : launch_backward<true, false>(a, ctas, slices, s));
    if (rc != FP8Q_OK || (!a.dpre && !a.dpost && !spread)) return rc;
    // rows of dgate to add up: those of a gate that spans strips, or the ones across their borders
    int64_t across = 0;
    if (spread && st.strips > 1 && st.per_strip % a.per != 0)
        across = a.per >= st.per_strip ? (a.rows + a.per - 1) / a.per : st.strips - 1;
    const dim3 grid((unsigned)((n->hidden + 31) / 32), (unsigned)(2 + across));
    return launch_kernel(residual_norm_sum_kernel, grid, dim3(1024), 0, s, "residual_norm_sum_kernel", a);
}

}  // extern "C"
