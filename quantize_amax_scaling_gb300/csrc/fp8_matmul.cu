// fp8_matmul.cu -- the product of two FP8 operands on the tensor cores, with what
// follows a linear layer in its epilogue; over rows grouped by expert; and the
// experts' weight gradients.
//
//   z = RN(sa sb) sum_k A[m][k] B[n][k] + bias[n],  D = RN(act(z) + residual),
//   q = FP8(bf16(D) / scale) with amax,  (h, h_sf) = the 8-bit checkpoint of bf16(z)
//
// Codes come into shared memory by tensor-map copies of 128 x 128 bytes (128-byte
// swizzle, zeros beyond the edges).  An operand may lie either way: where its rows
// are not along k, a box holds 128 of its rows for each of 128 k, and the tensor
// core reads it across, so the products of a backward pass need no transposed copy.
//
// Two kernels.  Few tiles: 128 rows of B by 16 to 128 of A a CTA, k split over a
// cluster while every CTA is resident; what bounds them is the operands' way from
// HBM and 4 us until it flows and the sums are out: 1 x 16384 x 4096 (67 MB) 14.1 us,
// 1 x 1024 x 4096 4.6; each megabyte more costs 0.15 us, 6.7 TB/s.  Many tiles: pairs
// of CTAs with 256 x 256.  8192 x 16384 x 4096 is 27 rounds of tiles, 442 thousand
// cycles of multiply-adds (128 for 256 x 256 x 32): 214 us at 2070 MHz.  It takes 294
// to 301 us in a burst, 3.7 PFLOP/s, and 325 to 347 in a loop at the 1400 W limit,
// where the clock falls to 1345 MHz: 466 thousand cycles, 95% of them multiply-adds.
// With zeros for operands (940 W, 2070 MHz) 239 to 255 us, 4.6 to 4.3 PFLOP/s: at
// that clock a tenth to a sixth goes to feeding them, to the start and to the end.
// So power bounds it first, their feeding next.
// Sums go out four columns of a row a lane (emit_rows), in pairs a row a lane
// (emit_row32), and a column a lane where n or an address holds no vectors
// (emit_cols); rows and columns beyond a group's or the matrix's edge are left out.

#include "checkpoint_calls.cuh"
#include "tcgen05.cuh"

namespace {

constexpr int kStepK = 128;       // codes of k a step
constexpr int kBoxBytes = 16384;  // of 128 x 128 codes
constexpr int kMaxGroups = 512;
// A k of more than kLongSteps goes by parts of kPartSteps (a multiple of every stage's steps): sum_parts().
constexpr int kPartSteps = 64, kLongSteps = 128;
constexpr int kPartK = kPartSteps * kStepK, kLongK = kLongSteps * kStepK;

struct Epilogue {
    const float *sa, *sb;
    const void *bias, *residual;
    void* d;
    uint8_t* q;
    const float* q_scale;
    float* amax;
    uint8_t *h, *h_sf;
    int32_t n;       // columns of D
    int32_t blocks;  // of 32, a row
    bool f32, bias_bf16, gelu, e5m2;
    bool vec;   // four columns a vector, and
    bool wide;   // sixteen bytes a vector, wherever a row starts, and
    bool whole;   // thirty-two of d, and
    bool whole8;  // of q and h
};

// P is the operand whose rows are the accumulator's lanes, Q the one whose rows are its columns.
struct ProductArgs {
    Epilogue e;
    const int32_t* offsets;  // [groups + 1]: group g is rows offsets[g] to offsets[g + 1] of A and D, or of k
    int32_t groups;
    int32_t rows;            // A's rows, of all groups; of ragged k: k's
    int32_t m;               // D's rows, in one group where k is ragged
    int32_t k;
    uint32_t idesc;
    int32_t p_across, q_across;  // P's, Q's rows do not lie along k
    int32_t p_tiles, q_tiles;    // tiles of a group where all have the same (pairs: of 256 columns, the last narrow ones apart)
    int32_t narrow;              // pairs: 1 where each row of tiles ends in one of half a tile's columns or fewer
    int32_t stages, per;         // stages of `per` steps
    int32_t split;               // CTAs of a cluster that share a tile's k
#ifdef FP8Q_TEST_HOOKS
    int32_t fail_role, fail_at, fail_cta;  // the wait that reports failure although what it waits for has come
#endif
};

enum PrWait { kPrNone, kPrCopyEmpty, kPrSumFull, kPrSumDrained, kPrMaskFull, kPrOutDone };
__device__ __forceinline__ bool pr_made_to_fail(const ProductArgs& a, PrWait role, uint32_t at) {
#ifdef FP8Q_TEST_HOOKS
    return a.fail_role == role && a.fail_at == (int)at && (a.fail_cta < 0 || a.fail_cta == (int)blockIdx.x);
#else
    return false;
#endif
}
// One wait of a whole warp, with one verdict.
__device__ __forceinline__ bool pr_wait(const ProductArgs& a, PrWait role, uint32_t at, uint64_t* bar, uint32_t parity) {
    return mbar_wait_all(bar, parity, pr_made_to_fail(a, role, at) && (threadIdx.x & 31) == 5);
}

__device__ __forceinline__ bool pr_wait_cluster(const ProductArgs& a, PrWait role, uint32_t at, uint64_t* bar, uint32_t parity) {
    return mbar_wait_all_cluster(bar, parity, pr_made_to_fail(a, role, at) && (threadIdx.x & 31) == 5);
}

// A group's rows; offsets that decrease or leave the tensor make it empty or end at the tensor's end.
__device__ __forceinline__ int2 group_rows(const ProductArgs& a, int g) {
    const int lo = min(max(a.offsets[g], 0), a.rows);
    return make_int2(lo, max(lo, min(a.offsets[g + 1], a.rows)));
}

// Sums of the counts up to and with each lane's, held at kManyTiles: right offsets never come near, wrong ones must not
// pass 32 bits (a tile before the tensor would be written there).
constexpr int kManyTiles = 0x3FFFFFFF;
__device__ __forceinline__ int sums_upto(int here) {
    int upto = here;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if ((threadIdx.x & 31) >= o) upto = min(upto + v, kManyTiles);
    }
    return upto;
}

// ----------------------------------------------------------------------------
// Epilogue

// x / (1 + 2^u), u = -2 sqrt(2 / pi) log2(e) (x + 0.044715 x^3), for two: exp and the reciprocal by the hardware's
// approximations, 2 and 1 units in the last place of binary32, and u off by 2 roundings, |u| 2^-23 in y: 2^-18 of y at x = -5,
// 2^-16 at -10, where y is 2^-120.  At -infinity the formula is NaN.
__device__ __forceinline__ float2 gelu2(float2 x) {
    const float2 u = mul2_rn(x, fma2_rn(mul2_rn(x, x), splat2(-0.102943239f), splat2(-2.302208198f)));
    float2 t, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t.x) : "f"(u.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t.y) : "f"(u.y));
    t = add2_rn(t, splat2(1.0f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.x) : "f"(t.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r.y) : "f"(t.y));
    return mul2_rn(x, r);
}

// Four consecutive elements of a row.
__device__ __forceinline__ void read4(const void* p, int64_t at, bool f32, float (&v)[4]) {
    if (f32) {
        const float4 x = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
        const uint2 x = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at);
        v[0] = __uint_as_float(x.x << 16), v[1] = __uint_as_float(x.x & 0xFFFF0000u);
        v[2] = __uint_as_float(x.y << 16), v[3] = __uint_as_float(x.y & 0xFFFF0000u);
    }
}
__device__ __forceinline__ float bf16_f(uint16_t w) { return __uint_as_float((uint32_t)w << 16); }

template <int FMT>
__device__ __forceinline__ uint32_t codes4(uint32_t w0, uint32_t w1, const QScale& c) {
    return c.fast ? quant_quad<FMT, true>(w0, w1, c) : quant_quad<FMT, false>(w0, w1, c);
}

// What a lane keeps over its columns.
struct Lane {
    QScale c;
    float alpha;
    uint32_t m2;  // the largest |bf16(D)|
    bool any;     // n, an address or q's scale is such that only emit_cols() holds
};

__device__ __forceinline__ Lane make_lane(const Epilogue& e) {
    Lane l;
    l.alpha = __fmul_rn(e.sa ? *e.sa : 1.0f, e.sb ? *e.sb : 1.0f);
    l.c = make_qscale_value(e.q ? *e.q_scale : 1.0f);
    l.m2 = 0;
    l.any = !e.vec || (e.q && !l.c.fast);
    return l;
}

// Eight rows from `row` on of one column a lane, the warp's a block of 32; bit i of `on` says whether the i-th is there.  For any n,
// any addresses, any scale of q.  Returns the lane's largest.  (2600x2310x512 18.6 us; four columns a lane out of line, each its
// own store into the others' sectors, 58.)
__device__ __forceinline__ uint32_t emit_cols(const Epilogue& e, Lane l, int64_t row, uint32_t on, int col, int64_t bias_at, float4 v0, float4 v1) {
    const bool in = col < e.n;
    float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
    if (!in) on = 0;
    const int64_t at = row * e.n + col;
    float b = 0.0f;
    if (in && e.bias) b = e.bias_bf16 ? bf16_f(static_cast<const uint16_t*>(e.bias)[bias_at + col]) : static_cast<const float*>(e.bias)[bias_at + col];
    uint32_t raw[8];
    if (e.residual) {  // all eight under way before the first is looked at (2600x2307x512 in bf16 28 us; 49 one after the other)
        const int64_t size = e.f32 ? 4 : 2;
        const uint8_t* p = static_cast<const uint8_t*>(e.residual) + at * size;
#pragma unroll
        for (int i = 0; i < 8; ++i, p += e.n * size) {
            raw[i] = 0;
            if (on >> i & 1) raw[i] = e.f32 ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = fmaf(v[i], l.alpha, b);
    uint32_t w[4];
    if (e.h) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = in ? cvt_bf16x2(v[2 * i], v[2 * i + 1]) : 0u;
        uint32_t mine = 0;
        uint8_t* h = e.h + at;
#pragma unroll
        for (int i = 0; i < 8; ++i, h += e.n) {
            const uint32_t x = w[i >> 1] >> 16 * (i & 1) & 0xFFFFu, code = ckpt_scale(__reduce_max_sync(0xFFFFFFFFu, x & 0x7FFFu));
            if (on >> i & 1) *h = (uint8_t)cvt_fp8x2<FP8Q_E4M3FN>(__uint_as_float(x << 16) * ckpt_factor(code), 0.0f);
            if ((col & 31) == i) mine = code;
        }
        const uint32_t there = __shfl_sync(0xFFFFFFFFu, on, 0);  // the block's first column is there if any is
        if ((col & 31) < 8 && (there >> (col & 31) & 1)) e.h_sf[(row + (col & 31)) * e.blocks + (col >> 5)] = (uint8_t)mine;
    }
    if (!(e.d || e.q || e.amax)) return l.m2;
    if (e.gelu) {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float2 y = gelu2(make_float2(v[i], v[i + 1]));
            v[i] = y.x, v[i + 1] = y.y;
        }
    }
    if (e.residual) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += __uint_as_float(e.f32 ? raw[i] : raw[i] << 16);
    }
    if (e.f32) {
        float* d = static_cast<float*>(e.d) + at;
#pragma unroll
        for (int i = 0; i < 8; ++i, d += e.n)
            if (on >> i & 1) *d = v[i];
        return l.m2;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = cvt_bf16x2(v[2 * i], v[2 * i + 1]);
    if (e.amax) {
#pragma unroll
        for (int i = 0; i < 4; ++i) l.m2 = bf16x2_absmax(l.m2, w[i] & ((on >> 2 * i & 1 ? 0xFFFFu : 0u) | (on >> 2 * i & 2 ? 0xFFFF0000u : 0u)));
    }
    if (e.d) {
        uint16_t* d = static_cast<uint16_t*>(e.d) + at;
#pragma unroll
        for (int i = 0; i < 8; ++i, d += e.n)
            if (on >> i & 1) *d = (uint16_t)(w[i >> 1] >> 16 * (i & 1));
    }
    if (e.q) {
        uint32_t four[2];
        if (e.e5m2)
            four[0] = codes4<FP8Q_E5M2>(w[0], w[1], l.c), four[1] = codes4<FP8Q_E5M2>(w[2], w[3], l.c);
        else
            four[0] = codes4<FP8Q_E4M3FN>(w[0], w[1], l.c), four[1] = codes4<FP8Q_E4M3FN>(w[2], w[3], l.c);
        uint8_t* q = e.q + at;
#pragma unroll
        for (int i = 0; i < 8; ++i, q += e.n)
            if (on >> i & 1) *q = (uint8_t)(four[i >> 2] >> 8 * (i & 3));
    }
    return l.m2;
}

// The same out of line, for pairs whose scale of q turns out to be none of the ordinary ones.
__device__ __noinline__ uint32_t emit_cols_apart(const Epilogue& e, Lane l, int64_t row, uint32_t on, int col, int64_t bias_at, float4 v0, float4 v1) {
    return emit_cols(e, l, row, on, col, bias_at, v0, v1);
}

// Columns col to col + 3 of rows row, row + step, .. of which bit i of `on` says whether the i-th is there; eight lanes side by
// side hold a block of 32 columns.  r: the residual.  All lanes of a warp come here.  For whole vectors at an ordinary scale, which
// go through the stages all rows at a time, so that a stage's latencies overlap: row by row, with the branches between,
// 8192x16384x4096 took 731 us with GELU, codes and checkpoint and 411 with bf16 alone.
template <int ROWS>
__device__ __forceinline__ void emit_rows(const Epilogue& e, Lane& l, int64_t row, int step, uint32_t on, int col, float (&v)[ROWS][4],
                                          const float (&b)[4], const float (&r)[ROWS][4]) {
    const uint32_t here = (col & ~31) < e.n ? on : 0u;  // of a block's eight lanes the first may be the only one with columns
    if (col >= e.n) on = 0;
    const float2 alpha = splat2(l.alpha), b0 = make_float2(b[0], b[1]), b1 = make_float2(b[2], b[3]);
    float2 x[ROWS][2];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        x[i][0] = fma2_rn(make_float2(v[i][0], v[i][1]), alpha, b0);
        x[i][1] = fma2_rn(make_float2(v[i][2], v[i][3]), alpha, b1);
    }
    const int64_t at = row * e.n + col, next = (int64_t)step * e.n;
    uint32_t w[ROWS][2];
    if (e.h) {
        uint32_t a[ROWS], mine = 0;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            w[i][0] = cvt_bf16x2(x[i][0].x, x[i][0].y), w[i][1] = cvt_bf16x2(x[i][1].x, x[i][1].y);
            a[i] = col < e.n ? bf16x2_absmax(w[i][0], w[i][1]) : 0u;
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1)
#pragma unroll
            for (int i = 0; i < ROWS; ++i) a[i] = bf16x2_absmax(a[i], __shfl_xor_sync(0xFFFFFFFFu, a[i], o));
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const uint32_t code = ckpt_scale(max(a[i] & 0x7FFFu, a[i] >> 16 & 0x7FFFu));
            a[i] = ckpt_codes4(w[i][0], w[i][1], ckpt_factor(code));
            if ((threadIdx.x & 7) == i) mine = code;
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (on >> i & 1) *reinterpret_cast<uint32_t*>(e.h + at + i * next) = a[i];
        // each of the eight lanes of a block stores a row's scale
        const int i = threadIdx.x & 7;
        if (i < ROWS && (here >> i & 1)) e.h_sf[(row + i * step) * e.blocks + (col >> 5)] = (uint8_t)mine;
    }
    if (e.gelu) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) x[i][0] = gelu2(x[i][0]), x[i][1] = gelu2(x[i][1]);
    }
    if (e.residual) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            x[i][0] = add2_rn(x[i][0], make_float2(r[i][0], r[i][1])), x[i][1] = add2_rn(x[i][1], make_float2(r[i][2], r[i][3]));
    }
    if (e.f32) {
        float* d = static_cast<float*>(e.d) + at;
#pragma unroll
        for (int i = 0; i < ROWS; ++i, d += next)
            if (on >> i & 1) *reinterpret_cast<float4*>(d) = make_float4(x[i][0].x, x[i][0].y, x[i][1].x, x[i][1].y);
        return;
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) w[i][0] = cvt_bf16x2(x[i][0].x, x[i][0].y), w[i][1] = cvt_bf16x2(x[i][1].x, x[i][1].y);
    if (e.amax) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            const uint32_t m = bf16x2_absmax(w[i][0], w[i][1]);
            l.m2 = bf16x2_absmax(l.m2, on >> i & 1 ? m : 0u);
        }
    }
    if (e.d) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (on >> i & 1) *reinterpret_cast<uint2*>(static_cast<uint16_t*>(e.d) + at + i * next) = make_uint2(w[i][0], w[i][1]);
    }
    if (e.q) {
        const Two s = two(l.c.s), mr = two(-l.c.r);
        uint32_t four[ROWS];
        if (e.e5m2) {
#pragma unroll
            for (int i = 0; i < ROWS; ++i) four[i] = codes4_fast<FP8Q_E5M2>(w[i][0], w[i][1], s, mr, l.c.t2);
        } else {
#pragma unroll
            for (int i = 0; i < ROWS; ++i) four[i] = codes4_fast<FP8Q_E4M3FN>(w[i][0], w[i][1], s, mr, l.c.t2);
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (on >> i & 1) *reinterpret_cast<uint32_t*>(e.q + at + i * next) = four[i];
    }
}

// Thirty-two bytes of a row in one store where rows start on whole sectors (`whole`): each of the two halves is a request of
// its own otherwise, in as many lines as there are lanes (8192x16384x4096 as below 394 us with halves, 340 whole).
__device__ __forceinline__ void st_row32(void* p, const uint4& a, const uint4& b, bool whole, bool full) {
    if (whole) {
        st_v8(p, a, b);
    } else {
        static_cast<uint4*>(p)[0] = a;
        if (full) static_cast<uint4*>(p)[1] = b;
    }
}
__device__ __forceinline__ float2 as_f2(uint32_t x, uint32_t y) { return make_float2(__uint_as_float(x), __uint_as_float(y)); }
__device__ __forceinline__ float2 bf16_f2(uint32_t w) { return as_f2(w << 16, w & 0xFFFF0000u); }

__device__ __forceinline__ uint4 ld_shared_u4(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void copy_ahead16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// Thirty-two columns from col on, or the row's last sixteen, of one row a lane, as tensor memory gives them: nothing passes
// between lanes, and a block of the checkpoint is a lane's own.  For n a multiple of 16, 16-byte addresses and an ordinary scale.
// (8192x16384x4096 with GELU, codes and checkpoint 340 us, 477 with the checkpoint's blocks over eight lanes each and codes
// through shared memory.)  Binary32 without a residual goes through shared memory: a row a lane there is 128 bytes in four
// lines a store, no faster.  res: the warp's 32 rows of the residual's columns in shared memory, their 16-byte pieces swizzled.
__device__ __forceinline__ void emit_row32(const Epilogue& e, Lane& l, int64_t row, int col, int64_t bias_at, const float (&v)[32], uint32_t res) {
    const int lane = threadIdx.x & 31;
    const bool full = col + 32 <= e.n;
    float2 x[16];
    const float2 alpha = splat2(l.alpha);
    if (e.bias && e.bias_bf16) {
        const uint4* b = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(e.bias) + bias_at + col);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 y = i < 2 || full ? b[i] : make_uint4(0, 0, 0, 0);
            x[4 * i] = fma2_rn(make_float2(v[8 * i], v[8 * i + 1]), alpha, bf16_f2(y.x));
            x[4 * i + 1] = fma2_rn(make_float2(v[8 * i + 2], v[8 * i + 3]), alpha, bf16_f2(y.y));
            x[4 * i + 2] = fma2_rn(make_float2(v[8 * i + 4], v[8 * i + 5]), alpha, bf16_f2(y.z));
            x[4 * i + 3] = fma2_rn(make_float2(v[8 * i + 6], v[8 * i + 7]), alpha, bf16_f2(y.w));
        }
    } else if (e.bias) {
        const float4* b = reinterpret_cast<const float4*>(static_cast<const float*>(e.bias) + bias_at + col);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float4 y = i < 4 || full ? b[i] : make_float4(0, 0, 0, 0);
            x[2 * i] = fma2_rn(make_float2(v[4 * i], v[4 * i + 1]), alpha, make_float2(y.x, y.y));
            x[2 * i + 1] = fma2_rn(make_float2(v[4 * i + 2], v[4 * i + 3]), alpha, make_float2(y.z, y.w));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = mul2_rn(make_float2(v[2 * i], v[2 * i + 1]), alpha);
    }
    const int64_t at = row * e.n + col;
    uint32_t w[16];
    if (e.h) {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = cvt_bf16x2(x[i].x, x[i].y);
        uint32_t m[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = full ? bf16x2_absmax(w[i], w[i + 8]) : bf16x2_absmax(w[i], 0u);
#pragma unroll
        for (int o = 4; o; o >>= 1)
#pragma unroll
            for (int i = 0; i < o; ++i) m[i] = bf16x2_absmax(m[i], m[i + o]);
        const uint32_t code = ckpt_scale(max(m[0] & 0x7FFFu, m[0] >> 16 & 0x7FFFu));
        const float f = ckpt_factor(code);
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = ckpt_codes4(w[2 * i], w[2 * i + 1], f);
        st_row32(e.h + at, make_uint4(o[0], o[1], o[2], o[3]), make_uint4(o[4], o[5], o[6], o[7]), e.whole8, full);
        e.h_sf[row * e.blocks + (col >> 5)] = (uint8_t)code;
    }
    if (e.gelu) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = gelu2(x[i]);
    }
    if (e.f32) {
        float* d = static_cast<float*>(e.d) + at;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (i >= 2 && !full) break;
            const uint4 r0 = ld_shared_u4(res + lane * 128 + (((2 * i) ^ (lane & 7)) << 4)), r1 = ld_shared_u4(res + lane * 128 + (((2 * i + 1) ^ (lane & 7)) << 4));
            const float2 a = add2_rn(x[4 * i], as_f2(r0.x, r0.y)), b = add2_rn(x[4 * i + 1], as_f2(r0.z, r0.w));
            const float2 c = add2_rn(x[4 * i + 2], as_f2(r1.x, r1.y)), g = add2_rn(x[4 * i + 3], as_f2(r1.z, r1.w));
            st_row32(d + 8 * i, make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y)),
                     make_uint4(__float_as_uint(c.x), __float_as_uint(c.y), __float_as_uint(g.x), __float_as_uint(g.y)), e.whole, true);
        }
        return;
    }
    if (e.residual) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint4 r = ld_shared_u4(res + lane * 64 + ((i ^ (lane >> 1 & 3)) << 4));
            x[4 * i] = add2_rn(x[4 * i], bf16_f2(r.x)), x[4 * i + 1] = add2_rn(x[4 * i + 1], bf16_f2(r.y));
            x[4 * i + 2] = add2_rn(x[4 * i + 2], bf16_f2(r.z)), x[4 * i + 3] = add2_rn(x[4 * i + 3], bf16_f2(r.w));
        }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = cvt_bf16x2(x[i].x, x[i].y);
    if (e.amax) {
#pragma unroll
        for (int i = 0; i < 16; ++i) l.m2 = i < 8 || full ? bf16x2_absmax(l.m2, w[i]) : l.m2;
    }
    if (e.d) {
        uint16_t* d = static_cast<uint16_t*>(e.d) + at;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (i < 1 || full)
                st_row32(d + 16 * i, make_uint4(w[8 * i], w[8 * i + 1], w[8 * i + 2], w[8 * i + 3]),
                         make_uint4(w[8 * i + 4], w[8 * i + 5], w[8 * i + 6], w[8 * i + 7]), e.whole, true);
    }
    if (e.q) {
        const Two s = two(l.c.s), mr = two(-l.c.r);
        uint32_t o[8];
        if (e.e5m2) {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = codes4_fast<FP8Q_E5M2>(w[2 * i], w[2 * i + 1], s, mr, l.c.t2);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = codes4_fast<FP8Q_E4M3FN>(w[2 * i], w[2 * i + 1], s, mr, l.c.t2);
        }
        st_row32(e.q + at, make_uint4(o[0], o[1], o[2], o[3]), make_uint4(o[4], o[5], o[6], o[7]), e.whole8, full);
    }
}

// A warp's largest, once it is through.
__device__ __forceinline__ void flush_lane(const Epilogue& e, const Lane& l) {
    if (!e.amax) return;
    const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, max(l.m2 & 0x7FFFu, l.m2 >> 16 & 0x7FFFu));
    if ((threadIdx.x & 31) == 0 && m) atomicMax(reinterpret_cast<int*>(e.amax), (int)(m << 16));
}

__device__ __forceinline__ void st_shared_v4(uint32_t at, const float* v) {
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]) : "memory");
}
__device__ __forceinline__ void ld_shared_v4(uint32_t at, float (&v)[4]) {
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(at) : "memory");
}

__device__ __forceinline__ float ld_shared_f(uint32_t at) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

// A long k goes by parts, each with one of two sets of accumulators, and the parts' sums are added here, rounded to nearest: the tensor
// cores cut off, towards zero, what lies below a sum's last place, and in one part the errors grow faster than k does.  Root mean
// square of the errors over that of the results, for activations with a few large channels: k = 4096 2.4e-7, 8192 5.8e-7, 16384
// 1.4e-6, 32768 3.7e-6 and by parts of 8192 5.8e-7, 100000 rows of a weight gradient 1.3e-5 and 4.6e-7, a million 3e-4 and 5e-7.
// By parts 4096x4096x32768 takes 348 us, 325 without, 512x4096x65536 129 and 120, 200000 rows of two experts to 512x512 238 and 216:
// the sums go through local memory, which meets the operands on their way out of shared memory.  (In registers, 128 of them, they
// make the epilogue spill: 16384 rows of 8 experts on top of a residual 180 us for 123; in shared memory with a stage less 253 for
// 216.)  Parts of 4096 from 8192 on halve the errors for twice the cost: 8192x4096x16384 343 us for 301.  So k up to 16384 is one part.
// By a warp, for COLS columns of its 32 lanes from `at` on in the first set, those of the second `gap` behind.  The whole sums come to
// lie where the last part's were.  first: the sets used before; done, drained: of both sets (PAIR: drained is the first CTA's).
template <int COLS, bool PAIR>
__device__ __forceinline__ bool sum_parts(uint32_t at, uint32_t gap, uint32_t first, int parts, uint64_t* done, uint64_t* drained, bool ok) {
    alignas(16) float sum[COLS];
    for (int j = 0; j < parts; ++j) {
        const uint32_t set = (first + j) & 1, parity = ((first + j) >> 1) & 1, from = at + set * gap;
        ok = ok && mbar_wait_warp(&done[set], parity, 32);
        tc_fence_after();
        constexpr int kAt = COLS < 32 ? COLS : 32;
#pragma unroll 1
        for (int c = 0; c < COLS; c += kAt) {
            float4* const held = reinterpret_cast<float4*>(sum + c);
            float4 y[kAt / 4];
#pragma unroll
            for (int i = 0; i < kAt / 4; ++i) y[i] = j ? held[i] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float v[kAt];
            if constexpr (kAt == 32)
                tmem_load32(from + c, v);
            else
                tmem_load16(from + c, v);
#pragma unroll
            for (int i = 0; i < kAt; i += 4) v[i] += y[i / 4].x, v[i + 1] += y[i / 4].y, v[i + 2] += y[i / 4].z, v[i + 3] += y[i / 4].w;
            if (j + 1 < parts) {
#pragma unroll
                for (int i = 0; i < kAt; i += 4) held[i / 4] = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < kAt; i += 16) tmem_store16(from + c + i, v + i);
            }
        }
        if (j + 1 < parts) {
            tc_fence_before();
            if ((threadIdx.x & 31) == 0) {
                if (PAIR)
                    arrive_cluster(in_cluster(smem_addr(&drained[set]), 0));
                else
                    arrive_local(&drained[set]);
            }
            __syncwarp();
        }
    }
    tmem_stored();
    return ok;
}

// A box of codes: 128 bytes along k by 128 rows, or 128 rows by 128 lines of k.  The multiply-adds of a step read 32 of k at
// a time, 32 bytes on in a line or 32 lines on.
__device__ __forceinline__ uint64_t k_advance(int across) { return across ? 256 : 2; }

// ----------------------------------------------------------------------------
// Few tiles: one CTA a tile, 128 rows of B by BN of A.  GROUPED: rows by expert, a kernel of its own (with both in one, what finds a
// tile's group takes 0.1 us of one token's 14.4).  LONG: k may be so long that it goes by parts; with GROUPED, for either.

template <int BN>
struct PrGeom {
    static constexpr int kSmem = (BN <= 64 ? 112 : 224) * 1024;  // two CTAs an SM, or one
    static constexpr int kMaxStages = kSmem / (kBoxBytes + BN * kStepK);
    static constexpr int kCols = BN < 32 ? 32 : BN;              // of tensor memory
};

// What the warps that carry a tile out know before its sums are there.
struct TileLane {
    Lane l;
    float b[4];
};
__device__ __forceinline__ TileLane make_tile_lane(const ProductArgs& a, int64_t group, int col) {
    TileLane t = {make_lane(a.e), {}};
    if (a.e.bias && !t.l.any && col < a.e.n) read4(a.e.bias, group * a.e.n + col, !a.e.bias_bf16, t.b);
    return t;
}

// This CTA's share of the tile's rows of A, over the SPLIT CTAs of the cluster whose sums are added in rank order, by four
// warps.  A warp takes four rows of 128 columns at a time.
template <int SPLIT, int BN>
__device__ __forceinline__ void emit_tile(const ProductArgs& a, TileLane& t, uint32_t part, int rank, int group, int p0, int q0, int q_end) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, col = p0 + lane * 4;
    const Epilogue& e = a.e;
    constexpr int kShare = BN / SPLIT;
    constexpr int kRows = kShare < 4 ? kShare : 4;
    float next[kRows][4];
    auto ask = [&](int i0) {  // the residual of a round, while the one before goes out
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (e.residual && !t.l.any && col < e.n && i0 < (rank + 1) * kShare && q0 + i0 + i < q_end)
                read4(e.residual, (int64_t)(q0 + i0 + i) * e.n + col, e.f32, next[i]);
    };
    ask(rank * kShare + warp * kRows);
#pragma unroll 1
    for (int i0 = rank * kShare + warp * kRows; i0 < (rank + 1) * kShare && q0 + i0 < q_end; i0 += 4 * kRows) {
        const int row = q0 + i0;
        float r[kRows][4], v[kRows][4] = {};
        uint32_t on = 0;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            on |= (uint32_t)(row + i < q_end) << i;
#pragma unroll
            for (int j = 0; j < 4; ++j) r[i][j] = next[i][j];
        }
        ask(i0 + 4 * kRows);
        if (SPLIT == 1) {
#pragma unroll
            for (int i = 0; i < kRows; ++i) ld_shared_v4(part + (i0 + i) * 512 + lane * 16, v[i]);
        } else {
#pragma unroll
            for (int i = 0; i < kRows; ++i) {
                float4 x[SPLIT];
#pragma unroll
                for (int j = 0; j < SPLIT; ++j) x[j] = ld_cluster_f32x4(in_cluster(part + (i0 + i) * 512 + lane * 16, j));
#pragma unroll
                for (int j = 0; j < SPLIT; ++j) v[i][0] += x[j].x, v[i][1] += x[j].y, v[i][2] += x[j].z, v[i][3] += x[j].w;
            }
        }
        if (t.l.any) {  // these rows of this CTA's sums are its own
            __syncwarp();
#pragma unroll
            for (int i = 0; i < kRows; ++i) st_shared_v4(part + (i0 + i) * 512 + lane * 16, v[i]);
            __syncwarp();
#pragma unroll 1
            for (int c = lane; p0 + (c & ~31) < e.n && c < 128; c += 32) {
                float x[4] = {};
#pragma unroll
                for (int i = 0; i < kRows; ++i) x[i] = ld_shared_f(part + (i0 + i) * 512 + c * 4);
                t.l.m2 = emit_cols(e, t.l, row, on, p0 + c, (int64_t)group * e.n, make_float4(x[0], x[1], x[2], x[3]), make_float4(0.0f, 0.0f, 0.0f, 0.0f));
            }
            continue;
        }
        emit_rows<kRows>(e, t.l, row, 1, on, col, v, t.b, r);
    }
    flush_lane(e, t.l);
}

// The rows of A of a tile, q0 < 0 for none.
struct TileRows {
    int q0, q_end, group;
};

// The groups' t-th tile where offsets decrease.  Groups may overlap then and have more tiles than the grid has CTAs, so each gives up
// the rows that a group which starts before it holds (of two that start together, the second): a row that any group holds stays with
// one, and there are no more parts of tiles than groups.
__device__ __noinline__ TileRows find_rows_apart(const int32_t* offsets, int groups, int rows, int tile_rows, int t) {
    int before = 0;
    for (int g = 0; g < groups; ++g) {
        int lo = min(max(offsets[g], 0), rows), top = 0;
        const int hi = min(offsets[g + 1], rows);
        for (int h = 0; h < groups && lo < hi; ++h) {
            const int from = min(max(offsets[h], 0), rows), to = min(offsets[h + 1], rows);
            if (from < to && (from < lo || (from == lo && h < g))) top = max(top, to);
        }
        lo = max(lo, top);
        const int here = lo < hi ? (hi - lo + tile_rows - 1) / tile_rows : 0;
        if (t - before < here) return {lo + (t - before) * tile_rows, hi, g};
        before += here;
    }
    return {-1, 0, 0};
}

// Whether offsets decrease anywhere, by the whole warp.
__device__ __forceinline__ bool offsets_fall(const ProductArgs& a) {
    bool fall = false;
    for (int g = threadIdx.x & 31; g < a.groups; g += 32) fall |= a.offsets[g] > a.offsets[g + 1];
    return __any_sync(0xFFFFFFFFu, fall) != 0;
}

template <int BN, bool GROUPED, bool LONG>
__global__ void __launch_bounds__(192) fp8_matmul_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                                                         const ProductArgs a) {
    using G = PrGeom<BN>;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full[G::kMaxStages], empty[G::kMaxStages], done[2], drained[2];
    __shared__ uint32_t tmem_slot, loads;
    __shared__ int gave_up;
    const uint32_t stages = a.stages, boxes = kBoxBytes + (a.q_across ? kBoxBytes : BN * kStepK), stage_bytes = a.per * boxes;
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    const int rank = a.split > 1 ? (int)(blockIdx.x % a.split) : 0;
    const int tile = blockIdx.x / a.split;

    if (threadIdx.x == 128) {
        if (a.k > 0) {
            prefetch_map(&map_p);
            prefetch_map(&map_q);
        }
        for (uint32_t i = 0; i < stages; ++i) {
            mbar_init(&full[i]);
            mbar_init(&empty[i]);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&done[i]);
            mbar_init_count(&drained[i], 4);
        }
        loads = 0;
        gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
    wait_behind();
    int p0, q0, q_end = a.m, group = 0;
    if (GROUPED && (!LONG || a.offsets)) {
        // this tile's group: tiles of B fastest, so that the tiles of a group's rows share its weights in L2
        const int t = tile / a.p_tiles;
        p0 = tile % a.p_tiles * 128;
        int before = 0, g0 = 0;
        bool found = false;
        for (; g0 < a.groups; g0 += 32) {
            int2 r = make_int2(0, 0);
            if (g0 + lane < a.groups) r = group_rows(a, g0 + lane);
            const int upto = sums_upto((r.y - r.x + BN - 1) / BN);
            const uint32_t past = __ballot_sync(0xFFFFFFFFu, before + upto > t);
            if (past) {
                const int i = __ffs(past) - 1;
                group = g0 + i;
                const int ahead = __shfl_sync(0xFFFFFFFFu, upto, i - (i > 0));  // tiles of the groups before, at most t - before
                q0 = __shfl_sync(0xFFFFFFFFu, r.x, i) + (t - before - (i > 0 ? ahead : 0)) * BN;
                q_end = __shfl_sync(0xFFFFFFFFu, r.y, i);
                found = true;
                break;
            }
            before = min(before + __shfl_sync(0xFFFFFFFFu, upto, 31), kManyTiles);
        }
        if (offsets_fall(a)) {
            const TileRows w = find_rows_apart(a.offsets, a.groups, a.rows, BN, t);
            q0 = w.q0, q_end = w.q_end, group = w.group;
            found = q0 >= 0;
        }
        if (!found) {  // the grid has room for a part of a tile in every group; the whole cluster ends here
            let_next_start();
            return;
        }
    } else {
        p0 = tile / a.q_tiles * 128;
        q0 = tile % a.q_tiles * BN;
    }
    // this CTA's steps
    const int steps = (a.k + kStepK - 1) / kStepK;
    const int s0 = (int)((int64_t)steps * rank / a.split), s1 = (int)((int64_t)steps * (rank + 1) / a.split);
    const int parts = LONG && s1 - s0 > kLongSteps ? (s1 - s0 + kPartSteps - 1) / kPartSteps : 1;
    const uint32_t cols = LONG ? 2 * G::kCols : G::kCols;
    if (warp == 5) {
        tmem_alloc<1>(&tmem_slot, cols);
        let_next_start();
    }
    const int col = p0 + lane * 4;
    TileLane t;
    uint32_t tmem = 0;
    if (warp != 4) {  // copies start without it
        tc_fence_before();
        some_sync<5 * 32>();
        tc_fence_after();
        tmem = tmem_slot;
    }

    if (warp == 4) {
        uint32_t st = 0, round = 0, n = 0;
        bool ok = true;
        for (int s = s0; s < s1; s += a.per, ++n) {
            if (!pr_wait(a, kPrCopyEmpty, n, &empty[st], (round & 1) ^ 1)) {
                ok = false;
                break;
            }
            const int there = min(a.per, s1 - s);
            if (elect_lane()) {
                uint32_t at = base + st * stage_bytes;
                expect_bytes(&full[st], there * boxes);
                for (int k = s * kStepK; k < (s + there) * kStepK; k += kStepK, at += boxes) {
                    if (a.p_across)
                        tile_load3(at, &map_p, p0, k, group, &full[st]);
                    else
                        tile_load3(at, &map_p, k, p0, group, &full[st]);
                    if (a.q_across)
                        tile_load3(at + kBoxBytes, &map_q, q0, k, 0, &full[st]);
                    else
                        tile_load3(at + kBoxBytes, &map_q, k, q0, 0, &full[st]);
                }
            }
            __syncwarp();
            if (++st == stages) st = 0, ++round;
        }
        // the tensor core's last arrivals land before the CTA may go
        for (uint32_t i = n > stages ? n - stages : 0; i < n && ok; ++i) ok = mbar_wait_all(&empty[i % stages], (i / stages) & 1);
        if (lane == 0) {
            if (!ok) gave_up = 1;
            loads = n;
        }
    } else if (warp == 5) {
        uint32_t st = 0, round = 0, part = 0, to = tmem;
        bool ok = true;
        const uint64_t next_p = k_advance(a.p_across), next_q = k_advance(a.q_across);
        for (int s = s0, n = 0; s < s1; s += a.per, ++n) {
            if (LONG && parts > 1 && (s - s0) % kPartSteps == 0 && s > s0) {  // the next part; stages hold 1, 2 or 4 steps
                if (elect_lane()) tc_commit(&done[part & 1]);
                __syncwarp();
                ++part;
                to = tmem + (part & 1) * G::kCols;
                if (part > 1 && !pr_wait(a, kPrSumDrained, part, &drained[part & 1], ((part >> 1) - 1) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
            }
            if (!pr_wait(a, kPrSumFull, n, &full[st], round & 1)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int end_k = min(a.k, min(s + a.per, s1) * kStepK);
            uint32_t at = base + st * stage_bytes;
            if (elect_lane()) {
                for (int k = s * kStepK; k < end_k; k += kStepK, at += boxes) {
                    const int nk = (end_k - k + 31) / 32;
                    const uint64_t dp = desc_codes(at), dq = desc_codes(at + kBoxBytes);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < nk) tc_mma_fp8<1>(to, dp + i * next_p, dq + i * next_q, a.idesc, (LONG && parts > 1 ? (k - s0 * kStepK) % kPartK : k - s0 * kStepK) | i);
                }
                tc_commit(&empty[st]);
            }
            __syncwarp();
            if (++st == stages) st = 0, ++round;
        }
        if (elect_lane()) {
            tc_commit(&done[part & 1]);
            if (!ok) gave_up = 1;
        }
    } else {
        t = make_tile_lane(a, group, col);
        const int row = q0 + rank * (BN / a.split) + (int)threadIdx.x;  // the residual on its way to L2
        if (a.e.residual && a.e.wide && (int)threadIdx.x < BN / a.split && row < q_end)
            block_prefetch(static_cast<const uint8_t*>(a.e.residual) + ((int64_t)row * a.e.n + p0) * (a.e.f32 ? 4 : 2), min(128, a.e.n - p0) * (a.e.f32 ? 4 : 2));
        const bool ok = parts > 1 ? sum_parts<BN, false>(tmem + ((uint32_t)(warp * 32) << 16), G::kCols, 0, parts, done, drained, true)
                                  : mbar_wait_warp(&done[0], 0, 0);
        if (!ok || pr_made_to_fail(a, kPrOutDone, 0)) gave_up = 1;
    }
    __syncwarp();
    __syncthreads();
    tc_fence_after();
    const int bad = gave_up;
    if (bad) {  // copies still under way end before the CTA does, and before sums (and NaN) lie where they go
        if (threadIdx.x == 0)
            for (uint32_t n = loads > stages ? loads - stages : 0; n < loads; ++n) mbar_wait(&full[n % stages], (n / stages) & 1);
        __syncthreads();
    }
    // the sums in shared memory, a row of A's 128 columns side by side; a wait that ran out (correct operation never gets there)
    // shows as NaN in the whole tile
    if (warp < 4) {
        float* part = reinterpret_cast<float*>(raw + (base - smem_addr(raw)));
        const uint32_t row = tmem + ((uint32_t)(warp * 32) << 16) + ((parts - 1) & 1) * G::kCols;
#pragma unroll 1
        for (int c = 0; c < BN; c += 16) {
            float v[16] = {};
            if (s0 < s1) tmem_load16(row + c, v);
#pragma unroll
            for (int i = 0; i < 16; ++i) part[(c + i) * 128 + warp * 32 + lane] = bad ? __uint_as_float(0x7FFFFFFFu) : v[i];
        }
    }
    tc_fence_before();
    if (a.split == 1) {
        __syncthreads();
        if (warp < 4) emit_tile<1, BN>(a, t, base, 0, group, p0, q0, q_end);
    } else {
        cluster_sync_all();
        if (warp < 4) {
            switch (a.split) {
                case 2: emit_tile<2, BN>(a, t, base, rank, group, p0, q0, q_end); break;
                case 4: emit_tile<4, BN>(a, t, base, rank, group, p0, q0, q_end); break;
                default: emit_tile<8, BN>(a, t, base, rank, group, p0, q0, q_end);
            }
        }
        cluster_sync_all();  // no CTA's sums go away while another reads them
    }
    if (warp == 5) tmem_free<1>(tmem, cols);
}

// ----------------------------------------------------------------------------
// Pairs: two CTAs of a cluster share tiles of 256 x 256.  Each holds 128 rows of
// P and of Q and the accumulators of its own rows of P; the first issues the
// multiply-adds for both, so a row of Q is read from shared memory once for 256
// rows of P.  Persistent, with two sets of accumulators: the tensor cores go on
// with the next tile while this one's sums go out.  Here P is A and Q is B.
//
// RAGGED_K: k is cut into groups that start and end anywhere, and a group's last
// step reads rows of the next one.  A warp of each CTA sees that step's codes arrive
// and puts zeros over the lines that are not the group's (both operands': zero times
// a NaN is none) before it tells the issuer.  That it tells what lies in its CTA's
// shared memory takes an arrival that releases to the cluster, which waits for
// whatever the CTA has under way: at every step it took weight gradients of 16384 rows
// of 8 experts, 4096x2048, from 113 us to 263.  Other steps' codes are announced by the
// copies alone, as without groups.

constexpr int kPrPairStages = 5;
constexpr int kPrPairThreads = 352;  // warps 0-7 carry results out, 8 copies codes, 9 multiplies, 10 puts zeros (RAGGED_K)
constexpr int kPrOut = kPrPairStages * 2 * kBoxBytes;
// Of each of the eight warps: 32 rows of 32 sums on their way out, or the residual of the next 64 (binary32) or 128 (bf16)
// columns on its way in.  It takes the place of a sixth stage, which bought nothing (8192x4096x4096 74 us either way) and left
// binary32 32 columns ahead: 3001 rows of 12 experts to weights of 2064x1040 on top of a residual 58 us, 46 with 64 ahead, 59
// without; bf16 57 us without, 35.  (With a prefetch to L2 beside it 48 and 42: twice the requests.)
constexpr int kPrRoom = 8192;
constexpr int kPrState = kPrOut + 8 * kPrRoom;

// Behind them in shared memory, which starts on 1024 bytes.  full: a stage's codes are there in both CTAs (the first
// CTA's counts); landed: they are in this one, of a group's last lines (ends: whose last use that was, and in the second byte the
// parity of each stage's next one); empty: the stage has been used; done, drained: a set of accumulators is
// complete, is in registers; stopped: the multiply-adds of an issuer that gave up have ended.
struct PairState {
    uint64_t full[kPrPairStages], landed[kPrPairStages], empty[kPrPairStages], done[2], drained[2], stopped;
    uint32_t tmem_slot, loads, ends;
    int gave_up;
    int cum[kMaxGroups + 1];  // row tiles before each group
};
constexpr int kPrPairSmem = kPrState + (int)sizeof(PairState);
static_assert(kPrPairSmem <= 227 * 1024, "");

struct PairWhere {
    int p0, p_end, q0;  // rows of A (of this CTA's pair's tile, absolute) and of B
    int cols;           // of the tile that are multiplied, a multiple of 32
    int group, k0, k;   // codes of k from k0
};
// Whether a step of `there` lines to a group's end multiplies lines that are not the group's.
template <bool RAGGED_K>
__device__ __forceinline__ bool group_ends(int there) {
    return RAGGED_K && there < kStepK && there % 32 != 0;
}
// The rows of tiles of all groups.
template <bool RAGGED_K>
__device__ __forceinline__ int pair_rows(const ProductArgs& a, const int* cum) {
    return RAGGED_K ? a.groups * a.p_tiles : a.offsets ? cum[a.groups] : a.p_tiles;
}
// Narrow tiles at the rows' ends come behind all others and are multiplied by their own width, so that a last round of them is
// shorter (2304x2176x4096 21.8 us, 24.4 with all of 256 and in their places; 8192x1040x4096 29.0 and 31.5; 3001 rows of 12 experts, n
// 1040, k 2064, 20.7 and 21.1).  Not for ragged k, which is short: there the stores bound (32.7 us, 30.9 in their places).
template <bool RAGGED_K>
__device__ __forceinline__ PairWhere pair_where(const ProductArgs& a, const int* cum, int tile) {
    PairWhere w;
    w.k0 = 0, w.k = a.k, w.group = 0, w.p_end = a.m;
    const int rows = pair_rows<RAGGED_K>(a, cum);
    const bool narrow = !RAGGED_K && a.narrow && tile >= (int64_t)rows * a.q_tiles;
    const int q_tiles = narrow ? 1 : a.q_tiles;
    if (narrow) tile -= rows * a.q_tiles;
    PairTile t;
    if (RAGGED_K) {
        const int each = a.p_tiles * q_tiles;
        w.group = tile / each;
        t = pair_tile(tile - w.group * each, a.p_tiles, q_tiles);
        const int2 r = group_rows(a, w.group);
        w.p0 = t.p, w.k0 = r.x, w.k = r.y - r.x;
    } else if (!a.offsets) {
        t = pair_tile(tile, a.p_tiles, q_tiles);
        w.p0 = t.p;
    } else {
        const int at = tile / q_tiles;
        int lo = 0, hi = a.groups;  // cum[lo] <= at < cum[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cum[mid] <= at) lo = mid; else hi = mid;
        }
        t = pair_tile(tile - cum[lo] * q_tiles, cum[lo + 1] - cum[lo], q_tiles);
        const int2 r = group_rows(a, lo);
        w.group = lo, w.p0 = r.x + t.p, w.p_end = r.y;
    }
    w.q0 = narrow ? a.q_tiles * 256 : t.q;
    w.cols = min(256, (a.e.n - w.q0 + 31) & ~31);
    return w;
}

//
// ANY: n or an address is such that only emit_cols() holds.  A kernel of its own (80 registers, and 40 bytes spilled): with both in
// one, 2600x2308x0 with a residual takes 28.5 us for 23.9, and with emit_cols() out of line 2600x2310x512 43 for 18.6.  LONG: k may be
// so long that it goes by parts.
template <bool RAGGED_K, bool ANY, bool LONG>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPrPairThreads)
    fp8_matmul_pair_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q, const ProductArgs a) {
    extern __shared__ __align__(1024) uint8_t raw[];
    PairState& sh = *reinterpret_cast<PairState*>(raw + kPrState);
    uint64_t *full = sh.full, *landed = sh.landed, *empty = sh.empty, *done = sh.done, *drained = sh.drained, &stopped = sh.stopped;
    uint32_t &tmem_slot = sh.tmem_slot, &loads = sh.loads;
    volatile int& gave_up = sh.gave_up;
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t base = smem_addr(raw);
    int* cum = sh.cum;
    const uint32_t rank = cluster_rank();
    const int stride = gridDim.x / 2, first = blockIdx.x / 2;

    if (threadIdx.x == 0) {
        if (a.k > 0) {
            prefetch_map(&map_p);
            prefetch_map(&map_q);
        }
        for (int i = 0; i < kPrPairStages; ++i) {
            mbar_init_count(&full[i], RAGGED_K ? 2 : 1);
            mbar_init(&landed[i]);
            mbar_init(&empty[i]);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&done[i]);
            mbar_init_count(&drained[i], 16);
        }
        mbar_init(&stopped);
        loads = 0;
        sh.ends = 0;
        gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers are there
    wait_behind();
    if (!RAGGED_K && a.offsets) {
        if (warp == 0) {
            int before = 0;
            for (int g0 = 0; g0 <= a.groups; g0 += 32) {
                int here = 0;
                if (g0 + lane < a.groups) {
                    const int2 r = group_rows(a, g0 + lane);
                    here = (r.y - r.x + 255) / 256;
                }
                const int upto = sums_upto(here), behind = __shfl_up_sync(0xFFFFFFFFu, upto, 1);
                if (g0 + lane <= a.groups) cum[g0 + lane] = min(before + (lane ? behind : 0), kManyTiles);
                before = min(before + __shfl_sync(0xFFFFFFFFu, upto, 31), kManyTiles);
            }
        }
        __syncthreads();
    }
    const int tiles = (int)min((int64_t)pair_rows<RAGGED_K>(a, cum) * (a.q_tiles + a.narrow), (int64_t)kManyTiles);
    if (warp == 9) {
        tmem_alloc<2>(&tmem_slot, 512);
        let_next_start();
    }
    uint32_t tmem = 0;
    if (warp != 8) {  // copies start without it
        tc_fence_before();
        some_sync<kPrPairThreads - 32>();
        tc_fence_after();
        tmem = *(volatile uint32_t*)&tmem_slot;
    }
    cluster_sync_all();  // both CTAs have tensor memory before the first multiplies into it

    if (warp == 8) {
        uint32_t st = 0, round = 0, n = 0, ends = 0;
        bool ok = true;
        const uint32_t bars = in_cluster(smem_addr(&full[0]), 0);
        for (int tile = first; tile < tiles && ok; tile += stride) {
            const PairWhere w = pair_where<RAGGED_K>(a, cum, tile);
            const int p0 = w.p0 + (int)rank * 128, q0 = w.q0 + (int)rank * (w.cols / 2);
            const int bg = RAGGED_K ? 0 : w.group;
            for (int k = 0; k < w.k; k += kStepK, ++n) {
                if (!pr_wait(a, kPrCopyEmpty, n, &empty[st], (round & 1) ^ 1)) {
                    ok = false;
                    break;
                }
                const uint32_t at = base + st * 2 * kBoxBytes, bar = bars + st * 8;
                const int px = a.p_across ? p0 : k, py = a.p_across ? w.k0 + k : p0;
                const int qx = a.q_across ? q0 : k, qy = a.q_across ? w.k0 + k : q0;
                if (group_ends<RAGGED_K>(w.k - k)) {
                    if (elect_lane()) {
                        expect_bytes(&landed[st], 2 * kBoxBytes);
                        tile_load3(at, &map_p, px, py, 0, &landed[st]);
                        tile_load3(at + kBoxBytes, &map_q, qx, qy, bg, &landed[st]);
                    }
                    ends = (ends | 1u << st) ^ 256u << st;
                } else {
                    if (elect_lane()) {
                        if (rank == 0) {
                            expect_bytes(&full[st], 4 * kBoxBytes);
                            if (RAGGED_K) arrive_local(&full[st]);  // for both that arrive at a group's end
                        }
                        tile_load3_pair(at, &map_p, px, py, 0, bar);
                        tile_load3_pair(at + kBoxBytes, &map_q, qx, qy, bg, bar);
                    }
                    ends &= ~(1u << st);
                }
                __syncwarp();
                if (++st == kPrPairStages) st = 0, ++round;
            }
        }
        // The tensor cores' last arrivals land before this CTA may go.
        for (uint32_t i = 0; i < kPrPairStages && i < n && ok; ++i) {
            st = st ? st - 1 : kPrPairStages - 1;
            ok = mbar_wait_all(&empty[st], ((n - 1 - i) / kPrPairStages) & 1);
        }
        if (lane == 0) {
            if (!ok) gave_up = 1;
            loads = n;
            sh.ends = ends;
        }
    } else if (warp == 9) {
        if (rank == 0) {
            uint32_t st = 0, round = 0, it = 0, n = 0;
            bool ok = true;
            const uint64_t next_p = k_advance(a.p_across), next_q = k_advance(a.q_across);
            for (int tile = first; tile < tiles && ok; tile += stride, ++it) {
                const PairWhere w = pair_where<RAGGED_K>(a, cum, tile);
                const uint32_t idesc = mma_desc_cols(a.idesc, w.cols);
                uint32_t set = it & 1, to = tmem + set * 256;
                if (it > 1 && !pr_wait(a, kPrSumDrained, it, &drained[set], ((it >> 1) - 1) & 1)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                for (int k = 0; k < w.k; k += kStepK, ++n) {
                    if (LONG && w.k > kLongK && k % kPartK == 0 && k > 0) {  // the next part
                        if (elect_lane()) tc_commit_pair(&done[set], 3);
                        __syncwarp();
                        set = ++it & 1, to = tmem + set * 256;
                        if (it > 1 && !pr_wait(a, kPrSumDrained, it, &drained[set], ((it >> 1) - 1) & 1)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                    }
                    if (!(group_ends<RAGGED_K>(w.k - k) ? pr_wait_cluster(a, kPrSumFull, n, &full[st], round & 1) : pr_wait(a, kPrSumFull, n, &full[st], round & 1))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const int nk = min(4, (w.k - k + 31) / 32);
                    const uint32_t at = base + st * 2 * kBoxBytes;
                    const uint64_t dp = desc_codes(at), dq = desc_codes(at + kBoxBytes);
                    if (elect_lane()) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (i < nk) tc_mma_fp8<2>(to, dp + i * next_p, dq + i * next_q, idesc, (LONG && w.k > kLongK ? k % kPartK : k) | i);
                        tc_commit_pair(&empty[st], 3);
                    }
                    __syncwarp();
                    if (++st == kPrPairStages) st = 0, ++round;
                }
                // An unfinished tile is never announced as done: those who carry results out run out of time in their
                // turn, in both CTAs, and write NaN.
                if (ok && elect_lane()) tc_commit_pair(&done[set], 3);
                __syncwarp();
            }
            // The other CTA's last arrivals land before this one may go.
            for (uint32_t i = it > 2 ? it - 2 : 0; i < it && ok; ++i) ok = mbar_wait_all(&drained[i & 1], (i >> 1) & 1);
            if (!ok) {
                if (elect_lane()) {
                    tc_commit_pair(&stopped, 1);
                    gave_up = 1;
                }
                __syncwarp();
                mbar_wait_all(&stopped, 0);
            }
        }
    } else if (warp == 10) {
        if constexpr (RAGGED_K) {
            uint32_t st = 0, n = 0, phase = 0;
            bool ok = true;
            const uint32_t bars = in_cluster(smem_addr(&full[0]), 0);
            for (int tile = first; tile < tiles && ok; tile += stride) {
                const PairWhere w = pair_where<RAGGED_K>(a, cum, tile);
                for (int k = 0; k < w.k; k += kStepK, ++n) {
                    const int there = w.k - k, upto = (there + 31) & ~31;  // lines of the group, and those that are multiplied
                    const bool ends = group_ends<RAGGED_K>(there);
                    // all steps of the group go by meanwhile, which may take longer than a wait
                    if (pr_made_to_fail(a, kPrMaskFull, n) ||
                        (ends && !mbar_wait_warp(&landed[st], phase >> st & 1, 32) && !mbar_wait_on(&landed[st], phase >> st & 1, empty, kPrPairStages))) {
                        ok = false;
                        break;
                    }
                    if (ends) {
                        const uint32_t at = base + st * 2 * kBoxBytes;
                        const float zero[4] = {};
                        for (int i = there * 8 + lane; i < upto * 8; i += 32) {
                            st_shared_v4(at + i * 16, zero);
                            st_shared_v4(at + kBoxBytes + i * 16, zero);
                        }
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) arrive_cluster_release(bars + st * 8);
                        phase ^= 1u << st;
                    }
                    __syncwarp();
                    if (++st == kPrPairStages) st = 0;
                }
            }
            if (!ok && lane == 0) gave_up = 1;
        }
    } else {
        const Epilogue& e = a.e;
        const uint32_t from = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (warp >> 2) * 128;
        const uint32_t room = base + kPrOut + warp * kPrRoom;
        const int sub = lane >> 3, c4 = (lane & 7) * 4;
        Lane l = make_lane(e);
        const bool rows_in_lanes = !ANY && e.wide && (!e.f32 || e.residual) && (!e.q || l.c.fast);
        const bool ahead = rows_in_lanes && e.residual;
        bool ok = true;
        uint32_t it = 0;
        const auto first_row = [&](const PairWhere& w) { return w.p0 + (int)rank * 128 + (warp & 3) * 32; };
        const auto d_row = [&](const PairWhere& w) { return (int64_t)first_row(w) + (RAGGED_K ? (int64_t)w.group * a.m : 0); };
        // 32 columns of a tile's residual on their way, by rows' lengths; a lane finds its row's as emit_row32() reads them
        const auto ask = [&](const PairWhere& w, int c, uint32_t to) {
            const int q = w.q0 + (warp >> 2) * 128 + c, rows = w.p_end - first_row(w);
            const uint8_t* from = static_cast<const uint8_t*>(e.residual) + (d_row(w) * e.n + q) * (e.f32 ? 4 : 2);
            if (e.f32) {
                if (q + c4 < e.n) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int row = i * 4 + sub;
                        if (row < rows) copy_ahead16(to + row * 128 + (((lane & 7) ^ (row & 7)) << 4), from + ((int64_t)row * e.n + c4) * 4);
                    }
                }
            } else if (q + (lane & 3) * 8 < e.n) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = i * 8 + (lane >> 2);
                    if (row < rows) copy_ahead16(to + row * 64 + (((lane & 3) ^ (row >> 1 & 3)) << 4), from + ((int64_t)row * e.n + (lane & 3) * 8) * 2);
                }
            }
        };
        PairWhere w = {}, then = {};
        if (first < tiles) w = pair_where<RAGGED_K>(a, cum, first);
        if (ahead && first < tiles) {
#pragma unroll
            for (int c = 0; c < kPrRoom / 64; c += 32) {
                if (e.f32 && c >= kPrRoom / 128) break;
                ask(w, c, room + c * (e.f32 ? 128 : 64));
                asm volatile("cp.async.commit_group;" ::: "memory");
            }
        }
        for (int tile = first; tile < tiles; tile += stride, ++it, w = then) {
            const bool more = tile + stride < tiles;
            if (more) then = pair_where<RAGGED_K>(a, cum, tile + stride);
            const int parts = LONG && w.k > kLongK ? (w.k + kPartK - 1) / kPartK : 1;
            const uint32_t before = it;
            it += parts - 1;
            const uint32_t set = it & 1;
            const uint32_t bar = in_cluster(smem_addr(&drained[set]), 0);
            const int p_first = first_row(w);
            const int64_t d_first = d_row(w);
            if (e.residual && !ahead && e.wide && p_first + lane < w.p_end) {  // on its way to L2 while the tensor cores work
                const int q = w.q0 + (warp >> 2) * 128, there = min(128, e.n - q), size = e.f32 ? 4 : 2;
                if (there > 0) block_prefetch(static_cast<const uint8_t*>(e.residual) + ((d_first + lane) * e.n + q) * size, there * size);
            }
            if (parts > 1)
                ok = sum_parts<128, true>(from, 256, before, parts, done, drained, ok);
            else
                ok = ok && mbar_wait_warp(&done[set], (it >> 1) & 1, 32);
            ok = ok && !pr_made_to_fail(a, kPrOutDone, it);
            if (!ok) gave_up = 1;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 128; c += 32) {
                const int q = w.q0 + (warp >> 2) * 128 + c, col = q + c4;
                float v[32];
                const bool staged = !rows_in_lanes && q < e.n && p_first < w.p_end;
                float b[4] = {}, r[8][4];
                if (!ANY && staged && !l.any) {  // on their way while tensor memory is read
                    if (e.bias && col < e.n) read4(e.bias, (int64_t)w.group * e.n + col, !e.bias_bf16, b);
                    if (e.residual) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            if (col < e.n && p_first + i * 4 + sub < w.p_end)
                                read4(e.residual, (d_first + i * 4 + sub) * e.n + col, e.f32, r[i]);
                        }
                    }
                }
                if (w.k > 0) {
                    tmem_load32(from + set * 256 + c, v);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0.0f;
                }
                if (c == 96) {  // the accumulators are in registers
                    tc_fence_before();
                    if (lane == 0) arrive_cluster(bar);
                }
                if (rows_in_lanes) {
                    const uint32_t res = room + (e.f32 ? c * 128 : c * 64) % kPrRoom;
                    if (ahead) {
                        if (e.f32)
                            asm volatile("cp.async.wait_group %0;" ::"n"(kPrRoom / 4096 - 1) : "memory");
                        else
                            asm volatile("cp.async.wait_group %0;" ::"n"(kPrRoom / 2048 - 1) : "memory");
                        __syncwarp();
                    }
                    if (!ok) {  // a wait that ran out shows as NaN
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(0x7FFFFFFFu);
                    }
                    if (q < e.n && p_first + lane < w.p_end) emit_row32(e, l, d_first + lane, q, (int64_t)w.group * e.n, v, res);
                    if (ahead) {
                        __syncwarp();
                        const int on = c + kPrRoom / (e.f32 ? 128 : 64);  // what this room holds next, of this tile or the one behind
                        if (on < 128)
                            ask(w, on, res);
                        else if (more)
                            ask(then, on - 128, res);
                        asm volatile("cp.async.commit_group;" ::: "memory");
                    }
                    continue;
                }
                if (q >= e.n || p_first >= w.p_end) continue;
                // through shared memory: a thread has a row's sums, and four of eight rows go out
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j) st_shared_v4(room + lane * 128 + ((j ^ (lane & 7)) << 4), v + 4 * j);
                __syncwarp();
                if (ANY || l.any) {  // a column a lane, eight rows at a time
#pragma unroll 1
                    for (int i0 = 0; i0 < 32 && p_first + i0 < w.p_end; i0 += 8) {
                        float y[8];
                        uint32_t on = 0;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            y[i] = ld_shared_f(room + (i0 + i) * 128 + (((lane >> 2) ^ i) << 4) + (lane & 3) * 4);
                            if (!ok) y[i] = __uint_as_float(0x7FFFFFFFu);  // a wait that ran out
                            on |= (uint32_t)(p_first + i0 + i < w.p_end) << i;
                        }
                        const float4 y0 = make_float4(y[0], y[1], y[2], y[3]), y1 = make_float4(y[4], y[5], y[6], y[7]);
                        l.m2 = ANY ? emit_cols(e, l, d_first + i0, on, q + lane, (int64_t)w.group * e.n, y0, y1)
                                   : emit_cols_apart(e, l, d_first + i0, on, q + lane, (int64_t)w.group * e.n, y0, y1);
                    }
                    continue;
                }
                if (ANY) continue;
                float x[8][4];
                uint32_t on = 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int row = i * 4 + sub;
                    ld_shared_v4(room + row * 128 + (((lane & 7) ^ (row & 7)) << 4), x[i]);
                    on |= (uint32_t)(p_first + row < w.p_end) << i;
                }
                if (!ok) {  // a wait that ran out shows as NaN
#pragma unroll
                    for (int i = 0; i < 8; ++i) x[i][0] = x[i][1] = x[i][2] = x[i][3] = __uint_as_float(0x7FFFFFFFu);
                }
                emit_rows<8>(e, l, d_first + sub, 4, on, col, x, b, r);
            }
        }
        flush_lane(e, l);
    }
    __syncwarp();
    __syncthreads();
    if (gave_up && threadIdx.x == 0) {  // copies still under way end before their CTAs do
        for (uint32_t n = loads > kPrPairStages ? loads - kPrPairStages : 0; n < loads; ++n) {
            const uint32_t st = n % kPrPairStages;
            if (RAGGED_K && (sh.ends >> st & 1))
                mbar_wait(&landed[st], (sh.ends >> (8 + st) & 1) ^ 1);
            else if (rank == 0)
                mbar_wait(&full[st], (n / kPrPairStages) & 1);
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (warp == 9) tmem_free<2>(tmem, 512);
    cluster_sync_all();
}

// ----------------------------------------------------------------------------
// Host

// An operand of `rows` rows, `groups` times; across: its rows do not lie along k.  Boxes of 128 bytes by 128 lines or box_rows
// rows, zeros beyond the edges.
bool operand_map(CUtensorMap* map, const uint8_t* q, int64_t rows, int64_t k, int64_t ld, int64_t groups, bool across, int box_rows) {
    const int64_t lines = across ? k : rows;
    return make_map<3>(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, {(cuuint64_t)(across ? rows : k), (cuuint64_t)lines, (cuuint64_t)groups},
                       {(cuuint64_t)ld, (cuuint64_t)(ld * lines)}, {kStepK, (cuuint32_t)(across ? kStepK : box_rows), 1},
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

template <int BN, bool GROUPED, bool LONG>
fp8q_status launch_product(const CUtensorMap& mp, const CUtensorMap& mq, ProductArgs a, unsigned grid, cudaStream_t s) {
    static std::atomic<uint64_t> devices{0};
    auto kern = fp8_matmul_kernel<BN, GROUPED, LONG>;
    const cudaError_t e = allow_smem(kern, PrGeom<BN>::kSmem, devices);
    if (e != cudaSuccess) return cuda_fail(e, "fp8_matmul_kernel setup");
    // Stages of up to four steps, two stages or more: a stage's waits and its arrival take its issuers 150 cycles each, and
    // a step 150 beside (24x4096x16384 with clusters of two: 16.3 us, 18.5 with a step a stage).
    const int steps = ((a.k + kStepK - 1) / kStepK + a.split - 1) / a.split;
    const int boxes = kBoxBytes + (a.q_across ? kBoxBytes : BN * kStepK), room = (PrGeom<BN>::kSmem - 1024) / boxes;
    a.per = room >= 12 ? 4 : room >= 5 ? 2 : 1;
    a.stages = room / a.per;
    const int most = (steps + a.per - 1) / a.per;  // what a short k leaves free lets the next kernel start
    if (a.stages > most) a.stages = most > 1 ? most : 1;
    const int need = a.stages * a.per * boxes;
    return launch_behind(kern, dim3(grid), dim3(192), (need > BN * 512 ? need : BN * 512) + 1024, (unsigned)a.split, s, "fp8_matmul_kernel", mp, mq, a);
}

template <int BN>
auto launch_product_of(bool grouped, bool parts) {
    return parts ? launch_product<BN, true, true> : grouped ? launch_product<BN, true, false> : launch_product<BN, false, false>;
}

template <bool RAGGED_K, bool ANY, bool LONG>
fp8q_status launch_product_pairs(const CUtensorMap& mp, const CUtensorMap& mq, const ProductArgs& a, int64_t tiles, cudaStream_t s) {
    static std::atomic<uint64_t> devices{0};
    auto kern = fp8_matmul_pair_kernel<RAGGED_K, ANY, LONG>;
    const cudaError_t e = allow_smem(kern, kPrPairSmem, devices);
    if (e != cudaSuccess) return cuda_fail(e, "fp8_matmul_pair_kernel setup");
    const int64_t pairs = sm_count() / 2;
    const unsigned grid = 2u * (unsigned)(tiles < pairs ? tiles : pairs);
    return launch_behind(kern, dim3(grid), dim3(kPrPairThreads), kPrPairSmem, 1, s, "fp8_matmul_pair_kernel", mp, mq, a);
}

#ifdef FP8Q_TEST_HOOKS
int g_pr_fail_role = 0, g_pr_fail_at = 0, g_pr_fail_cta = -1;
#endif

enum Grouping { kWhole, kGroupedRows, kGroupedK };

fp8q_status product(const fp8q_product* p, const int32_t* offsets, int32_t groups, Grouping how, void* stream) {
    if (!p || p->m < 0 || p->n < 0 || p->k < 0 || (how != kWhole && groups < 0)) return FP8Q_ERR_INVALID_ARG;
    if (!valid_fmt(p->a_fmt) || !valid_fmt(p->b_fmt) || (p->out != FP8Q_OUT_BF16 && p->out != FP8Q_OUT_F32)) return FP8Q_ERR_INVALID_ARG;
    if (p->act != FP8Q_ACT_NONE && p->act != FP8Q_ACT_GELU) return FP8Q_ERR_INVALID_ARG;
    if (p->m > kFp4MaxDim || p->n > kFp4MaxDim || p->k > kFp4MaxDim || (how != kWhole && groups > kMaxGroups)) return FP8Q_ERR_UNSUPPORTED;
    if (p->m == 0 || p->n == 0 || (how != kWhole && groups == 0)) return FP8Q_OK;
    if (!p->d && !p->q && !p->h && !p->amax) return FP8Q_ERR_INVALID_ARG;
    if (p->q ? (!valid_fmt(p->q_fmt) || !p->q_scale) : p->q_scale != nullptr) return FP8Q_ERR_INVALID_ARG;
    if (p->out == FP8Q_OUT_F32 && (!p->d || p->q || p->amax)) return FP8Q_ERR_INVALID_ARG;
    if ((p->h != nullptr) != (p->h_sf != nullptr)) return FP8Q_ERR_INVALID_ARG;
    if (how == kGroupedK && (p->bias || p->act != FP8Q_ACT_NONE || p->q || p->amax || p->h || !p->a_trans || !p->b_trans))
        return FP8Q_ERR_INVALID_ARG;
    if ((how == kGroupedRows && p->a_trans) || (how != kWhole && !offsets)) return FP8Q_ERR_INVALID_ARG;
    if (p->k > 0) {
        if (!p->a || !p->b) return FP8Q_ERR_INVALID_ARG;
        if (p->lda < (p->a_trans ? p->m : p->k) || p->ldb < (p->b_trans ? p->n : p->k)) return FP8Q_ERR_INVALID_ARG;
    }
    const uintptr_t odd2 = (uintptr_t)(p->out == FP8Q_OUT_BF16 ? p->d : nullptr) | (uintptr_t)(p->out == FP8Q_OUT_BF16 ? p->residual : nullptr) |
                           (uintptr_t)(p->bias_is_bf16 ? p->bias : nullptr);
    const uintptr_t odd4 = (uintptr_t)(p->out == FP8Q_OUT_F32 ? p->d : nullptr) | (uintptr_t)(p->out == FP8Q_OUT_F32 ? p->residual : nullptr) |
                           (uintptr_t)(p->bias_is_bf16 ? nullptr : p->bias) | (uintptr_t)p->a_scale | (uintptr_t)p->b_scale |
                           (uintptr_t)p->q_scale | (uintptr_t)p->amax | (uintptr_t)offsets;
    if ((odd2 & 1u) || (odd4 & 3u)) return FP8Q_ERR_INVALID_ARG;
    if (p->k > 0 && ((((uintptr_t)p->a | (uintptr_t)p->b) & 15u) || ((p->lda | p->ldb) & 15))) return FP8Q_ERR_UNSUPPORTED;
    // a tensor map's strides have 40 bits
    if (p->k > 0 && (p->lda >= (1ll << 31) || p->ldb >= (1ll << 31) ||
                     (how == kGroupedRows && groups > 1 && p->ldb * (p->b_trans ? p->k : p->n) >= (1ll << 40))))
        return FP8Q_ERR_UNSUPPORTED;

    ProductArgs a = {};
#ifdef FP8Q_TEST_HOOKS
    a.fail_role = g_pr_fail_role;
    a.fail_at = g_pr_fail_at;
    a.fail_cta = g_pr_fail_cta;
#endif
    Epilogue& e = a.e;
    e.sa = p->a_scale;
    e.sb = p->b_scale;
    e.bias = p->bias;
    e.residual = p->residual;
    e.d = p->d;
    e.q = p->q;
    e.q_scale = p->q_scale;
    e.amax = p->amax;
    e.h = p->h;
    e.h_sf = p->h_sf;
    e.n = (int32_t)p->n;
    e.blocks = (int32_t)((p->n + 31) / 32);
    e.f32 = p->out == FP8Q_OUT_F32;
    e.bias_bf16 = p->bias_is_bf16 != 0;
    e.gelu = p->act == FP8Q_ACT_GELU;
    e.e5m2 = p->q_fmt == FP8Q_E5M2;
    // four columns at a time
    const uintptr_t wide = (uintptr_t)p->d | (uintptr_t)p->residual;
    e.vec = p->n % 4 == 0 && (wide & (e.f32 ? 15u : 7u)) == 0 && ((uintptr_t)p->bias & (e.bias_bf16 ? 7u : 15u)) == 0 &&
            (((uintptr_t)p->q | (uintptr_t)p->h) & 3u) == 0;
    e.wide = e.vec && p->n % 16 == 0 && ((wide | (uintptr_t)p->bias | (uintptr_t)p->q | (uintptr_t)p->h) & 15u) == 0;
    e.whole = e.wide && ((uintptr_t)p->d & 31u) == 0;
    e.whole8 = e.wide && p->n % 32 == 0 && (((uintptr_t)p->q | (uintptr_t)p->h) & 31u) == 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    a.offsets = offsets;
    a.groups = how == kWhole ? 1 : groups;
    a.rows = (int32_t)(how == kGroupedK ? p->k : p->m);
    a.m = (int32_t)p->m;
    a.k = (int32_t)p->k;
    const int fa = p->a_fmt == FP8Q_E5M2, fb = p->b_fmt == FP8Q_E5M2, ta = p->a_trans != 0, tb = p->b_trans != 0;
    const int64_t b_groups = how == kGroupedRows ? groups : 1;
    const int sms = sm_count();
    // Pairs of CTAs where 128-row tiles of one CTA each would not all be resident at once.  (A grouped call does not know its
    // groups: at most a part of a tile in each beside full ones.)
    const int64_t across = (p->n + 127) / 128, blocks = (how == kGroupedRows ? p->m / 128 + groups : (p->m + 127) / 128) * across;
    const bool pairs = how == kGroupedK || (blocks > sms && (how == kGroupedRows ? p->m > 64 * (int64_t)groups : p->m > 128 && p->n > 128));
    CUtensorMap mp = {}, mq = {};
    if (pairs) {
        a.idesc = mma_desc_fp8(256, 256, fa, fb, ta, tb);
        a.p_across = ta;
        a.q_across = tb;
        a.split = 1;
        a.p_tiles = (int32_t)((p->m + 255) / 256);
        a.narrow = how != kGroupedK && p->n > 256 && p->n % 256 > 0 && p->n % 256 <= 128;
        a.q_tiles = (int32_t)(a.narrow ? p->n / 256 : (p->n + 255) / 256);
        const int64_t tiles = (how == kGroupedRows ? p->m / 256 + groups : (int64_t)a.p_tiles * (how == kGroupedK ? groups : 1)) * (a.q_tiles + a.narrow);
        if (tiles > kManyTiles) return FP8Q_ERR_UNSUPPORTED;
        if (p->k > 0 && (!operand_map(&mp, p->a, p->m, p->k, p->lda, 1, ta, 128) || !operand_map(&mq, p->b, p->n, p->k, p->ldb, b_groups, tb, 128)))
            return cuda_fail(cudaErrorInvalidValue, "fp8_matmul_pair_kernel tensor map");
        const auto launch = how == kGroupedK ? (a.k > kLongK ? (e.vec ? launch_product_pairs<true, false, true> : launch_product_pairs<true, true, true>)
                                                            : (e.vec ? launch_product_pairs<true, false, false> : launch_product_pairs<true, true, false>))
                                             : (a.k > kLongK ? (e.vec ? launch_product_pairs<false, false, true> : launch_product_pairs<false, true, true>)
                                                            : (e.vec ? launch_product_pairs<false, false, false> : launch_product_pairs<false, true, false>));
        return launch(mp, mq, a, tiles, s);
    }
    // P is B and Q is A.  Fewer rows of A a CTA while two thirds of the SMs have room for all CTAs: a tile goes out sooner
    // the smaller it is (300x1024x1024 5.3 us with 32 rows, 6.9 with 128; 278x208x64 5.5 and 14), but reads B once more, and
    // takes the SMs that would share a longer k (1003x1040x2064 9.4 us with 128, 10.3 with 64).
    const int64_t each = how == kGroupedRows ? (p->m + groups - 1) / groups : p->m;
    int bn = each <= 16 ? 16 : each <= 32 ? 32 : each <= 64 ? 64 : 128;
    while (bn > 32 && (how == kGroupedRows ? p->m * 2 / bn + groups : (p->m * 2 + bn - 1) / bn) * across * 3 <= sms * 2) bn /= 2;
    const int steps = (int)((p->k + kStepK - 1) / kStepK);
    a.idesc = mma_desc_fp8(128, bn, fb, fa, tb, ta);
    a.p_across = tb;
    a.q_across = ta;
    a.q_tiles = (int32_t)((p->m + bn - 1) / bn);
    // a grouped call does not know its groups: at most as many tiles as full ones and one part of a tile in each
    const int64_t q_tiles = how == kGroupedRows ? p->m / bn + (groups < p->m ? groups : p->m) : a.q_tiles;
    a.p_tiles = (int32_t)across;
    const int64_t tiles = across * q_tiles;
    // The CTAs of a cluster share a tile's sums, as many as are resident at once (two an SM up to 64 rows of A; clusters
    // of 4 and 8 reach 19 and 17 of 20 of them) and have four steps or more, where the steps that a CTA saves are worth the
    // cluster and its sums: 1x4096x4096 7.2 us on clusters of 8, 7.9 on 2; 1x1024x4096 4.7, 5.6 on 4; but two rounds of
    // CTAs cost more than they save, 1x16384x4096 18 us on clusters of 4, 13.9 on 2.
    const int64_t room = (bn <= 64 ? 2 : 1) * sms;
    int split = 1, most = 1;
    while (most < 8 && tiles * most * 2 <= room * (most == 1 ? 20 : most == 2 ? 19 : 17) / 20 && steps >= most * 8) most *= 2;
    if (steps - steps / most > 3 + bn / 32) split = most;
    a.split = split;
    if (tiles * split > kManyTiles) return FP8Q_ERR_UNSUPPORTED;
    if (p->k > 0 && (!operand_map(&mp, p->b, p->n, p->k, p->ldb, b_groups, tb, 128) || !operand_map(&mq, p->a, p->m, p->k, p->lda, 1, ta, bn)))
        return cuda_fail(cudaErrorInvalidValue, "fp8_matmul_kernel tensor map");
    const unsigned grid = (unsigned)(tiles * split);
    const bool grouped = how == kGroupedRows, parts = steps > kLongSteps * split;
    switch (bn) {
        case 16: return launch_product_of<16>(grouped, parts)(mp, mq, a, grid, s);
        case 32: return launch_product_of<32>(grouped, parts)(mp, mq, a, grid, s);
        case 64: return launch_product_of<64>(grouped, parts)(mp, mq, a, grid, s);
        default: return launch_product_of<128>(grouped, parts)(mp, mq, a, grid, s);
    }
}

}  // namespace

extern "C" {

#ifdef FP8Q_TEST_HOOKS  // the wait of that role (PrWait) at that step or tile reports failure, in one CTA or (cta < 0) in all
void fp8q_test_set_product_give_up(int role, int at, int cta) {
    g_pr_fail_role = role;
    g_pr_fail_at = at;
    g_pr_fail_cta = cta;
}
#endif

fp8q_status fp8q_matmul(const fp8q_product* args, void* stream) { return product(args, nullptr, 0, kWhole, stream); }

fp8q_status fp8q_grouped_matmul(const fp8q_product* args, const int32_t* offsets, int32_t groups, void* stream) {
    return product(args, offsets, groups, kGroupedRows, stream);
}

fp8q_status fp8q_grouped_weight_gradient(const fp8q_product* args, const int32_t* offsets, int32_t groups, void* stream) {
    return product(args, offsets, groups, kGroupedK, stream);
}

}  // extern "C"
