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
// strip to each T threads, whole warps; a thread has 16 (or 32) columns of a row,
// in groups of eight, and brings the next rows of its strip into shared memory by asynchronous
// copies of its own (it alone reads them, so they need no barrier), while the
// weights of its columns stay in shared memory (forward) or registers (backward).
//
// Measured, 8192 x 4096: e4m3 codes 42.5 us for 235 MB (5.5 TB/s), e5m2 42.3, MXFP4 43.6,
// NVFP4 48.5 us, a gate row a token 57.6 us for 302 MB; gradients 78 us for 403 MB
// (5.2 TB/s), 95 with a gate row a token.  One token of 4096 4.0 us, its gradients 6.9.
// Both issue instructions 48 to 65% of the time beside HBM at 44 to 67%: some 30 an
// element forward (NVFP4 36: a scale of every 16 elements), over two reductions a
// row that every warp of the row waits for.  (Inputs in rotation beyond L2, replayed
// from a graph.)

#include "fp4.cuh"
#include "packed_f32.cuh"

#include <cooperative_groups.h>

#include <initializer_list>

namespace {

constexpr int kRnMaxH = 32768;
constexpr int64_t kAllRows = 1ll << 32;  // more rows than there may be: rows a gate's row, held there, add up within 64 bits
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

// Eight columns of a thread, as four pairs: the arithmetic is two-lane binary32
// (packed_f32.cuh), which halves the instructions that bound these kernels.
struct Oct {
    float2 v[4];
};

__device__ __forceinline__ Oct widen8(const uint4& w) {
    Oct o;
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) o.v[i] = make_float2(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xFFFF0000u));
    return o;
}

__device__ __forceinline__ uint4 narrow8(const Oct& o) {
    return make_uint4(cvt_bf16x2(o.v[0].x, o.v[0].y), cvt_bf16x2(o.v[1].x, o.v[1].y), cvt_bf16x2(o.v[2].x, o.v[2].y),
                      cvt_bf16x2(o.v[3].x, o.v[3].y));
}

__device__ __forceinline__ Oct pairs8(const float4& a, const float4& b) {
    return {{make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)}};
}

__device__ __forceinline__ Oct splat8(float v) { return pairs8(make_float4(v, v, v, v), make_float4(v, v, v, v)); }

__device__ __forceinline__ Oct load8(const float* p) {
    return pairs8(*reinterpret_cast<const float4*>(p), *(reinterpret_cast<const float4*>(p) + 1));
}

__device__ __forceinline__ Oct load_gate8(const void* g, int is_bf16, int64_t at) {
    return is_bf16 ? widen8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(g) + at))
                   : load8(static_cast<const float*>(g) + at);
}

__device__ __forceinline__ void mul8(Oct& a, const Oct& b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) a.v[i] = mul2_rn(a.v[i], b.v[i]);
}

__device__ __forceinline__ float sum2(const float2& a, const float2& b) { return (a.x + a.y) + (b.x + b.y); }

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {  // global to shared memory
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
__device__ __forceinline__ void st_shared(uint32_t at, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ float4 as_f4(const uint4& v) {
    return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}
// Eight gate values that lie in the ring: one 16-byte slot of bf16, or two of binary32.
__device__ __forceinline__ Oct ring_gate8(uint32_t at, uint32_t step, int is_bf16) {
    return is_bf16 ? widen8(ld_shared(at)) : pairs8(as_f4(ld_shared(at)), as_f4(ld_shared(at + step)));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// A row's T threads wait for one another: the whole CTA where it has one row,
// else by a barrier of their own.
__device__ __forceinline__ void row_barrier(int T) {
    if (T == (int)blockDim.x)
        __syncthreads();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.x / T), "r"(T) : "memory");
}

// This lane's of the sums that a row's warps left in `part`: lane by lane, zeros up to the next power of two.
__device__ __forceinline__ float part_of(const float* part, int T) {
    const int warps = T >> 5, j = warps == 1 ? 0 : threadIdx.x & ((2 << (31 - __clz(warps - 1))) - 1);
    return j < warps ? part[threadIdx.x / T * warps + j] : 0.0f;
}

// Sum over the T threads of a row (T a multiple of 32 up to 1024; all of them
// call it).  `part` holds one float a warp and is not written again
// before the next barrier but one.
__device__ __forceinline__ float row_sum(float v, int T, float* part) {
    v = warp_sum(v);
    if (T == 32) return v;
    const int warp = threadIdx.x >> 5, warps = T >> 5;
    if ((threadIdx.x & 31) == 0) part[warp] = v;
    row_barrier(T);
    v = part_of(part, T);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
        if (o < warps) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// 1 / sqrt(v): the hardware's approximation and one Newton step (a relative error
// of 2^-22 goes to 1.5 times its square, so the roundings remain: 3 u at most).
// NaN for an infinite mean (an infinity in the row, or squares beyond binary32):
// a factor of 0 would pass off every finite element of such a row as a zero.
__device__ __forceinline__ float inv_sqrt(float v) {
    float y;
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(v));
    const float z = fmaf(y, fmaf(-0.5f * v * y, y, 0.5f), y);
    return v > 0x1p-126f && v < 3.4e38f ? z : __frcp_rn(__fsqrt_rn(v)) + (v - v);
}

// Codes of eight columns of h, a warp together, as fp8q_quantize_amax or
// fp8q_fp4_quantize_amax give them.  `at` is the place of the first in [rows, H].
template <int FMT>
__device__ __forceinline__ void store_codes(const RnArgs& a, const QScale& c8, const Fp4Scale& c4, int64_t row, int64_t at, int col, bool live,
                                            const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (FMT == FP8Q_E4M3FN || FMT == FP8Q_E5M2) {
        uint32_t o[2];
        if (c8.fast) {
            const float2 r = splat2(c8.r), mr = splat2(-c8.r), d = splat2(c8.s);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t x = bf16x2_clamp(w[i], c8.t2);
                const float2 f = make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u));
                const float2 y = quotient2(f, d, r, mr);  // divide<true>, two at a time
                const uint32_t q = cvt_fp8x2<FMT>(y.x, y.y);
                o[i >> 1] = i & 1 ? o[i >> 1] | (q << 16) : q;
            }
        } else {
            o[0] = quant_quad<FMT, false>(w[0], w[1], c8);
            o[1] = quant_quad<FMT, false>(w[2], w[3], c8);
        }
        if (live && col < a.H) st_v2(a.q + at, make_uint2(o[0], o[1]));
    } else if constexpr (FMT == FP8Q_MXFP4 || FMT == FP8Q_NVFP4) {
        constexpr int kLanes = Fp4<FMT>::kBlock / 8;  // lanes a block
        const uint32_t m = bf16x2_absmax(bf16x2_absmax(w[0], w[1]), bf16x2_absmax(w[2], w[3]));
        uint32_t am = max(m & 0x7FFFu, (m >> 16) & 0x7FFFu);
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, o));
        const BlockScale b = FMT == FP8Q_MXFP4 || c4.fast ? block_scale<FMT, true>(am, c4) : block_scale<FMT, false>(am, c4);
        const uint32_t codes = codes8<FMT>(w, b);
        const int64_t ld = fp4_row_bytes(a.H);
        if (live && col < 2 * ld) *reinterpret_cast<uint32_t*>(a.q + row * ld + col / 2) = codes;
        uint32_t s = b.code;
        s |= __shfl_down_sync(0xFFFFFFFFu, b.code, kLanes) << 8;
        s |= __shfl_down_sync(0xFFFFFFFFu, b.code, 2 * kLanes) << 16;
        s |= __shfl_down_sync(0xFFFFFFFFu, b.code, 3 * kLanes) << 24;
        const int64_t across = fp4_sf_tiles<FMT>(a.H), tile = col / Fp4<FMT>::kSfCols;
        if (live && (threadIdx.x & 31) % (4 * kLanes) == 0 && tile < across)
            *reinterpret_cast<uint32_t*>(a.sf + ((row / 128) * across + tile) * 512 + (row % 32) * 16 + (row % 128) / 32 * 4) = s;
    }
}

// U groups of eight columns a thread, THREADS threads a CTA.  Nothing but the
// packed sum stays in registers across the two reductions, and the weights lie in
// shared memory beside the ring (each thread's own; rows of more than 8192 columns
// read them from L1): with 16 columns' weights and values in registers 16 warps fit an SM and
// issued 59% of the time, 53 us for 8192x4096; with 24 warps it takes 49.  ROW > 0:
// the call that a block's edge makes (all parts there, a gate for several rows),
// for rows of that many threads: 42.6 us; ROW < 0: for any number of warps a row.
template <int FMT, int U, int THREADS, int ROW>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 3 : THREADS == 320 ? 2 : 1) residual_norm_kernel(const RnArgs a) {
    constexpr bool kFull = ROW != 0, kFixed = ROW > 0, kHold = THREADS < 1024;  // weights in shared memory
    constexpr int kStages = kHold ? 2 : 1;  // rows under way
    const uint32_t kStep = (kFixed ? THREADS : blockDim.x) * 16;   // from one slot to the next
    extern __shared__ __align__(16) uint8_t ring_raw[];
    __shared__ float part[4][32];
    __shared__ uint32_t red[32];
    const bool has_b = kFull || a.b, has_post = kFull || a.post, has_pre = kFull || a.pre, has_ro = kFull || a.ro;
    const int T = kFixed ? ROW : a.T, t = threadIdx.x % T;
    const uint32_t strip = blockIdx.x * ((kFixed ? THREADS : blockDim.x) / T) + threadIdx.x / T;
    const uint32_t rows = (uint32_t)a.rows, per_strip = (uint32_t)a.per_strip;
    const uint32_t row0 = strip * per_strip, row1 = min(row0 + per_strip, rows);
    const bool ring_gate = !kFull && kHold && a.gate && a.per == 1;
    const uint32_t slots = 1 + has_b + (ring_gate ? (a.gate_bf16 ? 1 : 2) : 0);
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(ring_raw)) + threadIdx.x * 16;
    const uint32_t weights = ring + kStages * U * slots * kStep;  // 2 U slots of alpha * gate * post, 2 U of pre
    const int col0 = t * 8;  // this thread's first columns; groups lie side by side across the warp
    auto off = [T](int u) { return u * T * 8; };
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) on[u] = col0 + off(u) < a.H;

    // columns that are not there stay zero in the ring, as their weights are; rows are not fetched, and
    // what the ring holds then goes nowhere
    for (uint32_t i = 0; i < kStages * U * slots + (kHold ? 4 * U : 0); ++i) st_shared(ring + i * kStep, make_uint4(0, 0, 0, 0));
    // the next kernel's CTAs only get in the way of CTAs that work on many rows (8192x4096, e4m3: 42.9 and 42.6 us)
    if (a.per_strip == 1) start_behind();
    else wait_behind();
    QScale c8;
    Fp4Scale c4;
    if constexpr (FMT == FP8Q_E4M3FN || FMT == FP8Q_E5M2) c8 = make_qscale_value(*a.scale);
    if constexpr (FMT == FP8Q_MXFP4 || FMT == FP8Q_NVFP4) c4 = make_fp4_scale(a.scale);
    uint32_t fetched = row0;
    int64_t src = (int64_t)row0 * a.H + col0;
    auto fetch = [&](uint32_t stage) {
        if (fetched < row1) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                uint32_t dst = ring + (stage * U + u) * slots * kStep;
                if (!on[u]) continue;
                copy16(dst, a.r + src + off(u));
                if (has_b) copy16(dst += kStep, a.b + src + off(u));
                if (ring_gate) {
                    if (a.gate_bf16) {
                        copy16(dst += kStep, static_cast<const uint16_t*>(a.gate) + src + off(u));
                    } else {
                        copy16(dst += kStep, static_cast<const float*>(a.gate) + src + off(u));
                        copy16(dst += kStep, static_cast<const float*>(a.gate) + src + off(u) + 4);
                    }
                }
            }
            src += a.H;
            ++fetched;
        }
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) fetch(i);

    // alpha * gate * post of a column, without the gate where it comes with the row
    auto weight = [&](int u, int64_t group) {
        Oct w = splat8(0.0f);
        if (!on[u]) return w;
        w = splat8(a.alpha);
        if (a.gate && !ring_gate) mul8(w, load_gate8(a.gate, a.gate_bf16, group * a.H + col0 + off(u)));
        if (has_post) mul8(w, load8(a.post + col0 + off(u)));
        return w;
    };
    auto keep = [&](uint32_t at, const Oct& o) {
        st_shared(at, make_uint4(__float_as_uint(o.v[0].x), __float_as_uint(o.v[0].y), __float_as_uint(o.v[1].x), __float_as_uint(o.v[1].y)));
        st_shared(at + kStep, make_uint4(__float_as_uint(o.v[2].x), __float_as_uint(o.v[2].y), __float_as_uint(o.v[3].x), __float_as_uint(o.v[3].y)));
    };
    auto kept = [&](uint32_t at) { return pairs8(as_f4(ld_shared(at)), as_f4(ld_shared(at + kStep))); };
    const uint32_t per = ring_gate || !a.gate ? rows : (uint32_t)min(a.per, (int64_t)rows);  // rows a gate's row
    uint32_t group = row0 / per, gend = (group + 1) * per;
    if (gend < row0) gend = rows;  // past 32 bits
    if (kHold && row0 < rows) {
        Oct w[U], p[U];  // all on their way before the first is waited for
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (has_b) w[u] = weight(u, group);
            if (has_pre && on[u]) p[u] = load8(a.pre + col0 + off(u));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (has_b) keep(weights + 2 * u * kStep, w[u]);
            if (has_pre && on[u]) keep(weights + (2 * U + 2 * u) * kStep, p[u]);
        }
    }
    const float inv_h = 1.0f / (float)a.H;
    uint32_t m2 = 0, stage = 0;
    int64_t at = (int64_t)row0 * a.H + col0;
    for (uint32_t it = 0; it < per_strip; ++it, at += a.H) {
        const uint32_t row = row0 + it;
        const bool live = row < row1;
        if (row == gend && live) {
            ++group;
            gend += per;
            if (kHold && has_b) {
                Oct w[U];
#pragma unroll
                for (int u = 0; u < U; ++u) w[u] = weight(u, group);
#pragma unroll
                for (int u = 0; u < U; ++u) keep(weights + 2 * u * kStep, w[u]);
            }
        }
        copies_wait<kStages - 1>();
        const uint32_t from = ring + stage * U * slots * kStep;
        uint4 o[U];
        float2 s[2] = {};
        if (has_b) {
            float rstd = 1.0f;
            if (has_post) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const Oct b = widen8(ld_shared(from + (u * slots + 1) * kStep));
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[i & 1] = fma2_rn(b.v[i], b.v[i], s[i & 1]);
                }
                rstd = inv_sqrt(fmaf(row_sum(sum2(s[0], s[1]), T, part[(it & 1) * 2]), inv_h, a.eps));
                if (a.rstd_post && live && t == 0) a.rstd_post[row] = rstd;
                s[0] = s[1] = make_float2(0.0f, 0.0f);
            }
            const float2 rs = splat2(rstd);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                Oct w = kHold ? kept(weights + 2 * u * kStep) : weight(u, live ? group : 0);
                if (ring_gate) mul8(w, ring_gate8(from + (u * slots + 2) * kStep, kStep, a.gate_bf16));
                Oct x = widen8(ld_shared(from + u * slots * kStep));
                const Oct b = widen8(ld_shared(from + (u * slots + 1) * kStep));
#pragma unroll
                for (int i = 0; i < 4; ++i) x.v[i] = fma2_rn(w.v[i], mul2_rn(b.v[i], rs), x.v[i]);
                o[u] = narrow8(x);
            }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) o[u] = ld_shared(from + u * slots * kStep);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (has_ro && live && on[u]) st_v4(a.ro + at + off(u), o[u]);
            const Oct x = widen8(o[u]);  // the norm before the next block is of what was stored
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i & 1] = fma2_rn(x.v[i], x.v[i], s[i & 1]);
        }
        float rstd = 0.0f;
        if (has_pre) {
            rstd = inv_sqrt(fmaf(row_sum(sum2(s[0], s[1]), T, part[(it & 1) * 2 + 1]), inv_h, a.eps));
            if (a.rstd_pre && live && t == 0) a.rstd_pre[row] = rstd;
        }
        // everything of this stage has been used: the row after the next ones into it
        fetch(stage);
        if (++stage == kStages) stage = 0;
        if (!has_pre) continue;
        const float2 rs = splat2(rstd);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Oct g = splat8(0.0f);
            if (kHold)
                g = kept(weights + (2 * U + 2 * u) * kStep);
            else if (on[u])
                g = load8(a.pre + col0 + off(u));
            Oct x = widen8(o[u]);
#pragma unroll
            for (int i = 0; i < 4; ++i) x.v[i] = mul2_rn(mul2_rn(x.v[i], rs), g.v[i]);
            uint4 h = narrow8(x);
            if (live && on[u]) {
                if (a.h) st_v4(a.h + at + off(u), h);
                m2 = bf16x2_absmax(m2, bf16x2_absmax(bf16x2_absmax(h.x, h.y), bf16x2_absmax(h.z, h.w)));
            } else {
                h = make_uint4(0, 0, 0, 0);  // where there is no column: 0 * NaN is not zero
            }
            if constexpr (FMT != kOutNone) store_codes<FMT>(a, c8, c4, row, at + off(u), col0 + off(u), live, h);
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
constexpr int kRnSms = 152;        // no more SMs' worth of strips than this, for which the workspace is sized: on fewer
                                   // SMs a strip is longer and there are no more of them
constexpr int kRnSlice = 4096;     // columns a CTA

struct RnStrips {
    int32_t T, slices, width, block;  // threads a strip, CTAs a row, columns and threads a CTA
    int64_t per_strip, strips;
};

RnStrips rn_strips(int64_t rows, int32_t H, int sms) {
    RnStrips s;
    s.slices = (H + kRnSlice - 1) / kRnSlice;
    s.width = ((H + s.slices - 1) / s.slices + 15) / 16 * 16;
    s.T = 256;
    while (s.T > 32 && s.width <= s.T * 8) s.T /= 2;
    // three CTAs of 160 threads an SM where 256 would leave every third idle and more (16256x2064: 76 us, 92; 6553x5120, two CTAs a row,
    // 88 and 111; a bf16 gate row a token 108 and 140, 125 and 150; few rows about the same: 777x2064 15.8 and 14.9, 15.5 and 15.6)
    if (s.T == 256 && s.width <= 160 * 16) s.T = 160;
    s.block = s.T == 160 ? 160 : 256;
    const int ctas = (sms < kRnSms ? sms : kRnSms) * (s.T == 160 ? 3 : 2), rows_at_once = ctas < s.slices ? 1 : ctas / s.slices;
    const int64_t most = (int64_t)rows_at_once * (s.block / s.T);
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

__device__ __forceinline__ void store8(float* p, const Oct& o) {
    reinterpret_cast<float4*>(p)[0] = make_float4(o.v[0].x, o.v[0].y, o.v[1].x, o.v[1].y);
    reinterpret_cast<float4*>(p)[1] = make_float4(o.v[2].x, o.v[2].y, o.v[3].x, o.v[3].y);
}

__device__ __forceinline__ void store_gate8(void* p, int is_bf16, int64_t at, const Oct& o) {
    if (is_bf16)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) = narrow8(o);
    else
        store8(static_cast<float*>(p) + at, o);
}

// Sums of three values over the warp: lane 0 has the first, 8 the second, 16 the
// third.  The lanes part the values between them as they add, so six exchanges
// do for what would take fifteen.
__device__ __forceinline__ float warp_sum3(float a, float b, float c) {
    const int lane = threadIdx.x & 31;
    // lanes below 16 keep a and b, the others c and nothing
    const float give0 = lane & 16 ? a : c, give1 = lane & 16 ? b : 0.0f;
    float k0 = lane & 16 ? c : a, k1 = lane & 16 ? 0.0f : b;
    k0 += __shfl_xor_sync(0xFFFFFFFFu, give0, 16);
    k1 += __shfl_xor_sync(0xFFFFFFFFu, give1, 16);
    const float give = lane & 8 ? k0 : k1;
    float k = lane & 8 ? k1 : k0;
    k += __shfl_xor_sync(0xFFFFFFFFu, give, 8);
#pragma unroll
    for (int o = 4; o; o >>= 1) k += __shfl_xor_sync(0xFFFFFFFFu, k, o);
    return k;
}

// Per row: one pass for the three sums, one for the gradients, both from shared
// memory (kept in registers between them, a row would spill).  With X = D n1 and
// W = alpha gate g1 of a column, a row adds X to the one sum S that dgate and dg1
// share: a gate's row of dgate is alpha g1 S, and dg1 takes alpha gate S whenever
// a gate's rows end.  RING_GATE: each row has its own gate, which comes with it.
// FULL: every part is there.  ROW > 0: strips of that many threads, in CTAs of 160 or 256.
template <bool CLUSTER, bool RING_GATE, bool FULL, int ROW>
__global__ void __launch_bounds__(ROW == 160 ? 160 : 256, ROW == 160 ? 3 : 2) residual_norm_backward_kernel(const RnBwdArgs a) {
    namespace cg = cooperative_groups;
    constexpr int kStages = RING_GATE ? 2 : 3;
    extern __shared__ __align__(16) uint8_t ring_raw[];
    __shared__ float part[2][3][8];
    __shared__ float sums[2][8][3];  // of each CTA of the cluster
    constexpr int kBlock = ROW == 160 ? 160 : 256;
    const bool has_b = FULL || a.b, has_post = FULL || a.post, has_dh = FULL || a.dh, has_dro = FULL || a.dro;
    const bool has_dr = FULL || a.dr, has_db = FULL || a.db;
    const int T = ROW > 0 ? ROW : a.T, t = threadIdx.x % T, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    int slices = 1, slice = 0;
    if (CLUSTER) {
        slices = (int)cg::this_cluster().num_blocks();
        slice = (int)cg::this_cluster().block_rank();
    }
    const int64_t strip = (int64_t)(blockIdx.x / slices) * (kBlock / T) + threadIdx.x / T;
    const int64_t row0 = strip * a.per_strip, row1 = min(row0 + a.per_strip, a.rows);
    const int c0 = slice * a.width, c1 = min(c0 + a.width, a.H);  // this CTA's columns
    const int col0 = c0 + t * 8;                                  // this thread's first, and
    const int next_u = T * 8;                                     // from one group of eight to the next
    const bool on[2] = {col0 < c1, col0 + next_u < c1};
    const float inv_h = 1.0f / (float)a.H;
    // ring: a stage holds, for each of two groups of eight columns, a slot of b, r', dr', dh and one
    // or two of the gate; behind it this thread's sums of dg1
    constexpr uint32_t kStep = kBlock * 16;
    const uint32_t slots = RING_GATE ? (a.gate_bf16 ? 5 : 6) : 4;
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(ring_raw)) + threadIdx.x * 16;
    const uint32_t post_sum = ring + kStages * 2 * slots * kStep;

    // what is not there stays zero in the ring (columns, whole tensors) or is never used (rows)
    for (uint32_t i = 0; i < kStages * 2 * slots + 4; ++i) st_shared(ring + i * kStep, make_uint4(0, 0, 0, 0));
    wait_behind();
    int64_t fetched = row0, src = row0 * a.H + col0;
    auto fetch = [&](uint32_t stage) {
        if (fetched < row1) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                if (!on[u]) continue;
                const uint32_t dst = ring + (stage * 2 + u) * slots * kStep;
                const int64_t at = src + u * next_u;
                if (has_b) copy16(dst, a.b + at);
                if (has_dh) {
                    copy16(dst + kStep, a.ro + at);
                    copy16(dst + 3 * kStep, a.dh + at);
                }
                if (has_dro) copy16(dst + 2 * kStep, a.dro + at);
                if (RING_GATE) {
                    if (a.gate_bf16) {
                        copy16(dst + 4 * kStep, static_cast<const uint16_t*>(a.gate) + at);
                    } else {
                        copy16(dst + 4 * kStep, static_cast<const float*>(a.gate) + at);
                        copy16(dst + 5 * kStep, static_cast<const float*>(a.gate) + at + 4);
                    }
                }
            }
            src += a.H;
            ++fetched;
        }
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages; ++i) fetch(i);

    int64_t group = a.gate ? row0 / a.per : 0;
    int64_t gend = a.gate ? (group + 1) * a.per : a.rows;  // first row behind the group
    bool whole = a.gate && group * a.per >= row0;          // the group began in this strip
    Oct Q[2], W[2], S[2], apre[2];
    // alpha * gate * post of a column, without a gate that comes with the row
    auto weight = [&](int u) {
        W[u] = splat8(a.alpha);
        if (has_post) mul8(W[u], load8(a.post + col0 + u * next_u));
        if (a.gate && !RING_GATE) mul8(W[u], load_gate8(a.gate, a.gate_bf16, group * a.H + col0 + u * next_u));
    };
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        Q[u] = W[u] = S[u] = apre[u] = splat8(0.0f);
        if (has_dh && on[u]) Q[u] = load8(a.pre + col0 + u * next_u);
        if (row0 < a.rows && on[u]) weight(u);
    }

    uint32_t stage = 0;
    int64_t at = row0 * a.H + col0;
    // a row's two factors are on their way while the row before it is worked on
    float next2 = has_dh && row0 < row1 ? a.rstd_pre[row0] : 0.0f;
    float next1 = has_post && row0 < row1 ? a.rstd_post[row0] : 1.0f;
    for (int64_t it = 0; it < a.per_strip; ++it, at += a.H) {
        const int64_t row = row0 + it;
        const bool live = row < row1;
        const float rstd2 = next2, rstd1 = next1;
        if (row + 1 < row1) {
            if (has_dh) next2 = a.rstd_pre[row + 1];
            if (has_post) next1 = a.rstd_post[row + 1];
        }
        const float2 r2 = splat2(rstd2), r1 = splat2(rstd1);
        copies_wait<kStages - 1>();
        const uint32_t at_stage = ring + stage * 2 * slots * kStep;
        float2 q0 = {}, q1 = {}, q2 = {};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const uint32_t from = at_stage + u * slots * kStep;
            const Oct fb = widen8(ld_shared(from)), fo = widen8(ld_shared(from + kStep)), fd = widen8(ld_shared(from + 2 * kStep)),
                      fh = widen8(ld_shared(from + 3 * kStep));
            Oct w = W[u];
            if (RING_GATE) mul8(w, ring_gate8(from + 4 * kStep, kStep, a.gate_bf16));
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 n2 = mul2_rn(fo.v[i], r2), dn = mul2_rn(fh.v[i], Q[u].v[i]);
                const float2 k = mul2_rn(w.v[i], mul2_rn(fb.v[i], r1));
                q0 = fma2_rn(dn, n2, q0);
                q1 = fma2_rn(k, fma2_rn(r2, dn, fd.v[i]), q1);
                q2 = fma2_rn(k, n2, q2);
            }
        }
        float s0, s1, s2;
        {
            const float k = warp_sum3(q0.x + q0.y, q1.x + q1.y, q2.x + q2.y);
            float(*pt)[8] = part[it & 1];
            if ((lane & 7) == 0 && lane < 24) pt[lane >> 3][warp] = k;
            if (T > 32)
                __syncthreads();
            else
                __syncwarp();
            if constexpr (ROW == 160) {
                s0 = part_of(pt[0], T);
                s1 = part_of(pt[1], T);
                s2 = part_of(pt[2], T);
            } else {  // a power of two
                const int i = (warp & ~((T >> 5) - 1)) + (lane & ((T >> 5) - 1));
                s0 = pt[0][i];
                s1 = pt[1][i];
                s2 = pt[2][i];
            }
            for (int o = ROW == 160 ? 4 : T >> 6; o; o >>= 1) {
                s0 += __shfl_xor_sync(0xFFFFFFFFu, s0, o);
                s1 += __shfl_xor_sync(0xFFFFFFFFu, s1, o);
                s2 += __shfl_xor_sync(0xFFFFFFFFu, s2, o);
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
        const float m1 = has_post ? (s1 - rstd2 * c2 * s2) * inv_h : 0.0f;  // mean(w D); no term without g1
        const float2 mc2 = splat2(-c2), mm1 = splat2(-m1);
        const bool flush = has_b && (row + 1 == gend || row + 1 == row1);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (!live) continue;  // what the ring holds is another row's
            const uint32_t from = at_stage + u * slots * kStep;
            const Oct fb = widen8(ld_shared(from)), fo = widen8(ld_shared(from + kStep)), fh = widen8(ld_shared(from + 3 * kStep));
            Oct D = widen8(ld_shared(from + 2 * kStep)), w = W[u], e, g;
            if (RING_GATE) {
                g = ring_gate8(from + 4 * kStep, kStep, a.gate_bf16);
                mul8(w, g);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 n2 = mul2_rn(fo.v[i], r2), n1 = mul2_rn(fb.v[i], r1);
                D.v[i] = fma2_rn(r2, fma2_rn(n2, mc2, mul2_rn(fh.v[i], Q[u].v[i])), D.v[i]);
                apre[u].v[i] = fma2_rn(fh.v[i], n2, apre[u].v[i]);
                S[u].v[i] = fma2_rn(D.v[i], n1, S[u].v[i]);
                e.v[i] = mul2_rn(r1, fma2_rn(n1, mm1, mul2_rn(D.v[i], w.v[i])));
            }
            if (!on[u]) continue;
            if (has_dr) st_v4(a.dr + at + u * next_u, narrow8(D));
            if (has_db) st_v4(a.db + at + u * next_u, narrow8(e));
            if (flush) {
                const int col = col0 + u * next_u;
                Oct p = splat8(1.0f);
                if (has_post) p = load8(a.post + col);
                if (a.gate && !RING_GATE) g = load_gate8(a.gate, a.gate_bf16, group * a.H + col);
                if (!a.gate) g = splat8(1.0f);
                mul8(S[u], splat8(a.alpha));
                mul8(p, S[u]);
                float4 lo = as_f4(ld_shared(post_sum + 2 * u * kStep)), hi = as_f4(ld_shared(post_sum + (2 * u + 1) * kStep));
                Oct sum = pairs8(lo, hi);
#pragma unroll
                for (int i = 0; i < 4; ++i) sum.v[i] = fma2_rn(S[u].v[i], g.v[i], sum.v[i]);
                st_shared(post_sum + 2 * u * kStep, make_uint4(__float_as_uint(sum.v[0].x), __float_as_uint(sum.v[0].y),
                                                               __float_as_uint(sum.v[1].x), __float_as_uint(sum.v[1].y)));
                st_shared(post_sum + (2 * u + 1) * kStep, make_uint4(__float_as_uint(sum.v[2].x), __float_as_uint(sum.v[2].y),
                                                                     __float_as_uint(sum.v[3].x), __float_as_uint(sum.v[3].y)));
                S[u] = splat8(0.0f);
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
        fetch(stage);
        if (++stage == kStages) stage = 0;
        if (a.gate && row + 1 == gend) {
            ++group;
            gend += a.per;
            whole = true;
            if (!RING_GATE && row + 1 < row1) {
                if (on[0]) weight(0);
                if (on[1]) weight(1);
            }
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        if (strip < a.strips && on[u]) {
            const int col = col0 + u * next_u;
            if (a.dpre) store8(a.space + strip * a.H + col, apre[u]);
            if (a.dpost)
                store8(a.space + (a.strips + strip) * a.H + col,
                       pairs8(as_f4(ld_shared(post_sum + 2 * u * kStep)), as_f4(ld_shared(post_sum + (2 * u + 1) * kStep))));
        }
    }
    copies_wait<0>();
    if (CLUSTER) cg::this_cluster().sync();  // nobody's `sums` goes away while another CTA may write it
}

// COLS columns a CTA, four a lane, 32 warps of 128 / COLS strips at a time: blockIdx.y 0 adds dpre, 1 dpost, and from 2
// on a row of dgate that lies in several strips: row blockIdx.y - 2, where gates span strips, or else the one across the
// border behind strip blockIdx.y - 2.  (32 columns a CTA where 128 would leave most SMs idle: 777x1552 13.2 us for the
// call, 15.1 by 128; 8192x1024 29.6 and 33.7; wider rows and many gates by 128: 8192x4096 77.2 us, 80 by 32.)
template <int COLS>
__global__ void __launch_bounds__(1024) residual_norm_sum_kernel(const RnBwdArgs a) {
    constexpr int kLanes = COLS / 4, kStrips = 32 / kLanes;  // a warp's
    __shared__ float4 part[32][kLanes];
    // launched while the kernel that writes the strips still runs: nothing is read before it has ended
    wait_behind();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = lane % kLanes, sub = lane / kLanes;
    const int col = blockIdx.x * COLS + c * 4;
    const int what = blockIdx.y;
    int64_t group = 0, s0 = 0, s1 = a.strips - 1;
    const float* from = a.space + what * a.strips * a.H + col;
    int64_t step = a.H;
    if (what < 2) {
        if (what == 0 ? !a.dpre : !a.dpost) return;
    } else {
        group = a.per >= a.per_strip ? what - 2 : (what - 1) * a.per_strip / a.per;
        const int64_t begin = group * a.per, end = min(begin + a.per, a.rows);
        s0 = begin / a.per_strip, s1 = (end - 1) / a.per_strip;
        if (s0 == s1 || (a.per < a.per_strip && s0 != what - 2)) return;  // in one strip, or another border's
        from = a.space + 2 * a.strips * a.H + col;
        step = 2 * a.H;
    }
    float4 v = make_float4(0, 0, 0, 0);
    auto add = [&v](const float4& x) { v.x += x.x; v.y += x.y; v.z += x.z; v.w += x.w; };
    auto across = [&] {  // the lanes of one column
#pragma unroll
        for (int o = kLanes; o < 32; o <<= 1)
            add(make_float4(__shfl_xor_sync(0xFFFFFFFFu, v.x, o), __shfl_xor_sync(0xFFFFFFFFu, v.y, o),
                            __shfl_xor_sync(0xFFFFFFFFu, v.z, o), __shfl_xor_sync(0xFFFFFFFFu, v.w, o)));
    };
    if (col < a.H) {
#pragma unroll 8
        for (int64_t s = s0 + w * kStrips + sub; s <= s1; s += 32 * kStrips)
            // a group's first rows are the tail of strip s0, the rest the heads of those that follow
            add(*reinterpret_cast<const float4*>(from + s * step + (what >= 2 && s == s0 ? a.H : 0)));
    }
    across();
    if (sub == 0) part[w][c] = v;
    __syncthreads();
    if (w > 0) return;
    v = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kLanes; ++i) add(part[sub * kLanes + i][c]);
    across();
    if (sub == 0 && col < a.H) {
        if (what == 0)
            *reinterpret_cast<float4*>(a.dpre + col) = v;
        else if (what == 1)
            *reinterpret_cast<float4*>(a.dpost + col) = v;
        else if (a.gate_bf16)
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dgate) + group * a.H + col) = make_uint2(cvt_bf16x2(v.x, v.y), cvt_bf16x2(v.z, v.w));
        else
            *reinterpret_cast<float4*>(static_cast<float*>(a.dgate) + group * a.H + col) = v;
    }
}

// The strips' sums, with `across` rows of dgate.
fp8q_status launch_sums(const RnBwdArgs& a, int64_t across, cudaStream_t s) {
    const int cols = a.H <= 2048 && across <= 4 ? 32 : 128;
    return launch_behind(cols == 32 ? residual_norm_sum_kernel<32> : residual_norm_sum_kernel<128>,
                         dim3((unsigned)((a.H + cols - 1) / cols), (unsigned)(2 + across)), dim3(1024), 0, 1, s,
                         "residual_norm_sum_kernel", a);
}

template <bool CLUSTER, bool RING_GATE, bool FULL, int ROW>
fp8q_status launch_backward(const RnBwdArgs& a, unsigned ctas, unsigned slices, cudaStream_t s) {
    static std::atomic<uint64_t> devices{0};
    constexpr int block = ROW == 160 ? 160 : 256;
    auto kern = residual_norm_backward_kernel<CLUSTER, RING_GATE, FULL, ROW>;
    const size_t smem = ((RING_GATE ? 2 * 2 * (a.gate_bf16 ? 5 : 6) : 3 * 2 * 4) + 4) * block * 16;
    cudaError_t e = allow_smem(kern, 112 * 1024, devices);
    if (e != cudaSuccess) return cuda_fail(e, "residual_norm_backward_kernel setup");
    return launch_behind(kern, dim3(ctas), dim3(block), smem, CLUSTER ? slices : 1, s, "residual_norm_backward_kernel", a);
}

template <int FMT>
fp8q_status launch_forward(RnArgs a, cudaStream_t s) {
    // rows of more than 8192 columns: 32 columns a thread, the row after next not on its way and the weights from L1, so that
    // two or three rows are under way on an SM and not one (2048x16384, e4m3: 68 us, 79; 4088x8208 70 and 108)
    const int U = a.H > 8192 ? 4 : 2;
    // As many threads a row as its columns want, whole warps: a power of two leaves up to half of them idle (6553x5120, e4m3:
    // 46.5 us, 68 with 512 threads; 8160x4112 53.7 and 82).  Where it leaves less than a quarter, or two such rows
    // would not fit an SM, the power of two is as good or better (5242x6400 57 us, 61 with 416).
    a.T = (a.H + U * 256 - 1) / (U * 256) * 32;
    if (a.T > 192 && a.T < 256) a.T = 256;
    if (U == 2 && a.T > 320 && a.T < 512) a.T = 512;
    const int per_cta = a.T < 256 ? 256 / a.T : 1, block = a.T * per_cta;
    const bool hold = U == 2;  // weights in shared memory, two rows under way
    const int slots = 1 + (a.b != nullptr) + (hold && a.gate && a.per == 1 ? (a.gate_bf16 ? 1 : 2) : 0);
    const size_t smem = (size_t)((hold ? 2 : 1) * U * slots + (hold ? 4 * U : 0)) * block * 16;
    // strips: as many as CTAs are resident, by registers (80 a thread, 24 warps; 96 in CTAs of up to 320, 20; 128 of 512, 16;
    // 64 with 32 columns a thread, 32) and shared memory
    const int64_t by_regs = (!hold ? 32 : block <= 256 ? 24 : block <= 320 ? 20 : 16) / (block / 32), by_smem = (int64_t)(224 * 1024 / (smem + 2048));
    const int64_t most = (by_regs < by_smem ? by_regs : by_smem) * sm_count() * per_cta;
    a.per_strip = (a.rows + most - 1) / most;
    const int64_t strips = (a.rows + a.per_strip - 1) / a.per_strip;
    const dim3 grid((unsigned)((strips + per_cta - 1) / per_cta));
    static std::atomic<uint64_t> devices[11];
    const int which = !hold ? 3 : block <= 256 ? 0 : block <= 320 ? 2 : 1;
    auto kern = which == 0   ? residual_norm_kernel<FMT, 2, 256, 0>
                : which == 1 ? residual_norm_kernel<FMT, 2, 512, 0>
                : which == 2 ? residual_norm_kernel<FMT, 2, 320, 0>
                             : residual_norm_kernel<FMT, 4, 1024, 0>;
    int set = which;
    if constexpr (FMT != kOutNone) {
        if (a.b && a.post && a.pre && a.ro && !(a.gate && a.per == 1) && hold) {
            set = a.T == 32 ? 4 : a.T == 64 ? 5 : a.T == 128 ? 6 : a.T == 256 ? 7 : a.T == 512 ? 8 : block <= 256 ? 9 : 10;
            kern = set == 4   ? residual_norm_kernel<FMT, 2, 256, 32>
                   : set == 5 ? residual_norm_kernel<FMT, 2, 256, 64>
                   : set == 6 ? residual_norm_kernel<FMT, 2, 256, 128>
                   : set == 7 ? residual_norm_kernel<FMT, 2, 256, 256>
                   : set == 8 ? residual_norm_kernel<FMT, 2, 512, 512>
                   : set == 9 ? residual_norm_kernel<FMT, 2, 256, -1>
                              : residual_norm_kernel<FMT, 2, 320, -1>;
        }
    }
    // at most 2 stages of 8 slots and 8 of weights of 512 threads, or 8 slots of 1024
    const cudaError_t e = allow_smem(kern, 192 * 1024, devices[set]);
    if (e != cudaSuccess) return cuda_fail(e, "residual_norm_kernel setup");
    return launch_behind(kern, grid, dim3(block), smem, 1, s, "residual_norm_kernel", a);
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
    if (rows <= 0 || hidden <= 0 || rows > kFp4MaxDim || hidden > kRnMaxH) return 0;
    const RnStrips st = rn_strips(rows, hidden, kRnSms);
    return (rows_per_gate > 1 ? 4 : 2) * st.strips * hidden * (int64_t)sizeof(float);
}

fp8q_status fp8q_residual_norm_backward(const fp8q_residual_norm_grad* n, void* stream) {
    if (!n || n->rows < 0 || n->hidden < 16 || n->hidden % 16 != 0) return FP8Q_ERR_INVALID_ARG;
    if (n->hidden > kRnMaxH || n->rows > kFp4MaxDim) return FP8Q_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (n->rows == 0) {  // the sums over no rows
        if (misaligned({n->d_pre_weight, n->d_post_weight}, 15)) return FP8Q_ERR_UNSUPPORTED;
        if (!n->d_pre_weight && !n->d_post_weight) return FP8Q_OK;
        RnBwdArgs none = {};
        none.dpre = n->d_pre_weight;
        none.dpost = n->d_post_weight;
        none.H = n->hidden;
        return launch_sums(none, 0, s);
    }
    if (!n->d_residual_out && !n->d_h) return FP8Q_ERR_INVALID_ARG;
    if (n->d_h ? (!n->residual_out || !n->rstd_pre || !n->pre_weight) : (n->pre_weight || n->d_pre_weight != nullptr))
        return FP8Q_ERR_INVALID_ARG;
    if (!n->block && (n->post_weight || n->gate || n->d_block)) return FP8Q_ERR_INVALID_ARG;
    if (n->post_weight ? !n->rstd_post : n->d_post_weight != nullptr) return FP8Q_ERR_INVALID_ARG;
    if (n->gate ? n->rows_per_gate < 1 : n->d_gate != nullptr) return FP8Q_ERR_INVALID_ARG;
    const RnStrips st = rn_strips(n->rows, n->hidden, sm_count());
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
    a.per = n->rows_per_gate < kAllRows ? n->rows_per_gate : kAllRows;
    a.per_strip = st.per_strip;
    a.strips = st.strips;
    a.H = n->hidden;
    a.T = st.T;
    a.gate_bf16 = n->gate_is_bf16 != 0;
    a.alpha = n->alpha;
    a.width = st.width;
    const int64_t per_cta = st.block / st.T;
    const unsigned ctas = (unsigned)((st.strips + per_cta - 1) / per_cta) * (unsigned)st.slices;
    const bool ring_gate = a.gate && a.per == 1;
    const unsigned slices = (unsigned)st.slices;
    // the call that a block's edge makes: everything there
    const bool full = a.b && a.post && a.dh && a.dro && a.dr && a.db;
    fp8q_status rc;
    if (a.T == 160)
        rc = ring_gate ? (slices == 1 ? launch_backward<false, true, false, 160>(a, ctas, 1, s) : launch_backward<true, true, false, 160>(a, ctas, slices, s))
             : full    ? (slices == 1 ? launch_backward<false, false, true, 160>(a, ctas, 1, s) : launch_backward<true, false, true, 160>(a, ctas, slices, s))
             : slices == 1 ? launch_backward<false, false, false, 160>(a, ctas, 1, s)
                           : launch_backward<true, false, false, 160>(a, ctas, slices, s);
    else if (ring_gate)
        rc = slices == 1 ? launch_backward<false, true, false, 0>(a, ctas, 1, s) : launch_backward<true, true, false, 0>(a, ctas, slices, s);
    else if (slices > 1)
        rc = full ? launch_backward<true, false, true, 256>(a, ctas, slices, s) : launch_backward<true, false, false, 0>(a, ctas, slices, s);
    else if (!full)
        rc = launch_backward<false, false, false, 0>(a, ctas, 1, s);
    else
        rc = a.T == 32    ? launch_backward<false, false, true, 32>(a, ctas, 1, s)
             : a.T == 64  ? launch_backward<false, false, true, 64>(a, ctas, 1, s)
             : a.T == 128 ? launch_backward<false, false, true, 128>(a, ctas, 1, s)
                          : launch_backward<false, false, true, 256>(a, ctas, 1, s);
    if (rc != FP8Q_OK || (!a.dpre && !a.dpost && !spread)) return rc;
    // rows of dgate to add up: those of a gate that spans strips, or the ones across their borders
    int64_t across = 0;
    if (spread && st.strips > 1 && st.per_strip % a.per != 0)
        across = a.per >= st.per_strip ? (a.rows - 1) / a.per + 1 : st.strips - 1;
    return launch_sums(a, across, s);
}

}  // extern "C"
