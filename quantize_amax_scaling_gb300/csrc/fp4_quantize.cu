// fp4_quantize.cu -- bf16 -> microscaled 4-bit operands, of a matrix and of its
// transpose in one pass, and back.
//
// Four kernels, which stream HBM.
//   fp4_quantize_kernel         with the transpose, or of rows that start anywhere:
//       tiles of 128 x 128.  128 rows are what a scale tile spans, so a CTA writes
//       whole scale tiles (512 contiguous bytes) and, for the transpose, 64
//       contiguous bytes of each of its 128 code rows.  A thread quantizes 16
//       columns of a row from registers; the transpose reads the same tile back
//       from shared memory by pairs of columns.  Rows that do not start on
//       32-byte boundaries pass through shared memory by 16 aligned bytes.
//   fp4_quantize_rows_kernel    one direction of rows on 32-byte boundaries: tiles of
//       32 x 512, from registers alone.
//   fp4_dequantize_rows_kernel  rows on 16-byte boundaries: tiles of 8 x 1024.
//   fp4_dequantize_kernel       rows that start anywhere: tiles of 64 x 128, out
//       through shared memory by 16 aligned bytes.
//
// Measured, 8192 x 4096, 86 MB for one direction (105 MB for both): NVFP4 15.9 us
// (26.9), MXFP4 14.3 us (19.9), back 14.2 and 13.9 us, 3.9 to 6.1 TB/s; 1187 x 2731
// both ways, where rows start anywhere, 7.1 and 5.5 us, back 4.7.  NVFP4 both ways
// issues in 64 % of its cycles, with 24 warps an SM that load, compute and store in
// turn (DRAM 33 %): a scale of every 16 elements costs a conversion there and back,
// two products and a reciprocal, twice over.  (Inputs in rotation beyond L2,
// replayed from a graph.)

#include "fp4.cuh"

#include <type_traits>

namespace {

constexpr int kTile = 128;  // rows and columns of a CTA's tile

// Rows that start anywhere pass through shared memory as they lie in memory, by
// groups of 16 aligned bytes: element e of a row's part of the tile is half-word
// e + shift there, `shift` the part's place within its 16 bytes.
constexpr int kGroups = kTile / 8 + 1;  // a row's
__device__ __forceinline__ int shift_of(const uint16_t* first) { return (int)(((uintptr_t)first >> 1) & 7); }

// Rows [r0, r0 + 128) of x, columns [c0, c0 + 128), into `raw`, zeros where there are none; nine groups a thread,
// all on their way at once.  A group takes its neighbours' elements along, where they belong to x.
// (8192x4095, NVFP4: 27.9 us, both ways 38.8; 31.7 and 47.7 by 32-bit words.)
__device__ __forceinline__ void load_rows(uint4* raw, const uint16_t* x, int64_t r0, int64_t rows, int64_t c0, int64_t cols) {
    constexpr int kLoads = (kTile * kGroups + kThreads - 1) / kThreads;
    const int n = (int)min((int64_t)kTile, cols - c0);
    const uint16_t* end = x + rows * cols;
    uint4 v[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
        const int i = j * kThreads + threadIdx.x, k = i / kGroups;
        v[j] = make_uint4(0, 0, 0, 0);
        if (k < kTile && r0 + k < rows) {
            const uint16_t* first = x + (r0 + k) * cols + c0;
            const int e = (i - k * kGroups) * 8 - shift_of(first);
            const uint16_t* at = first + e;
            if (e < n) {
                if (at >= x && at + 8 <= end) {
                    v[j] = *reinterpret_cast<const uint4*>(at);
                } else {  // x's first or last
                    uint32_t u[4];
#pragma unroll
                    for (int h = 0; h < 4; ++h)
                        u[h] = (at + 2 * h >= x && at + 2 * h < end ? (uint32_t)at[2 * h] : 0u) |
                               (at + 2 * h + 1 >= x && at + 2 * h + 1 < end ? (uint32_t)at[2 * h + 1] << 16 : 0u);
                    v[j] = make_uint4(u[0], u[1], u[2], u[3]);
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
        const int i = j * kThreads + threadIdx.x, k = i / kGroups;
        if (n < kTile && r0 + k < rows) {  // columns past the last
            const int keep = n - ((i - k * kGroups) * 8 - shift_of(x + (r0 + k) * cols + c0));  // elements of the group
            uint32_t u[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
            for (int h = 0; h < 4; ++h) u[h] &= (keep > 2 * h ? 0xFFFFu : 0u) | (keep > 2 * h + 1 ? 0xFFFF0000u : 0u);
            v[j] = make_uint4(u[0], u[1], u[2], u[3]);
        }
        if (k < kTile) raw[i] = v[j];
    }
}

struct Fp4QuantArgs {
    const uint16_t* x;
    uint8_t *q, *sf, *qt, *sft;
    const float* scale;
    float* amax;
    int64_t rows, cols, tile_cols;
};

// The 512-byte scale tiles gathered in `s` go out by 32-bit words (four blocks
// of one row); words of rows at or past `rows` and tiles past the last are not
// written.
template <int FMT>
__device__ __forceinline__ void store_sf(uint8_t* sf, const uint32_t* s, int64_t r0, int64_t rows, int64_t c0,
                                         int64_t cols) {
    constexpr int kTiles = kTile / Fp4<FMT>::kSfCols;
    const int64_t across = fp4_sf_tiles<FMT>(cols), t0 = c0 / Fp4<FMT>::kSfCols;
    const int i = threadIdx.x & 127, t = threadIdx.x >> 7;
    if (t < kTiles && t0 + t < across && r0 + (i & 3) * 32 + (i >> 2) < rows)
        reinterpret_cast<uint32_t*>(sf)[((r0 / 128) * across + t0 + t) * 128 + i] = s[t * 128 + i];
}

__device__ __forceinline__ int sf_byte(int row, int block) {
    return (block >> 2) * 512 + (row & 31) * 16 + (row >> 5) * 4 + (block & 3);
}

template <int FMT, bool ROW, bool COL, bool VEC>
__global__ void __launch_bounds__(kThreads) fp4_quantize_kernel(const Fp4QuantArgs a) {
    constexpr int kBlock = Fp4<FMT>::kBlock;
    __shared__ uint32_t red[kThreads / 32];
    __shared__ __align__(16) uint32_t sfs[2 * 128];
    __shared__ __align__(16) uint32_t xs[VEC ? kTile * kTile / 2 : kTile * kGroups * 4];
    __shared__ __align__(16) uint2 qts[COL ? kTile * 9 : 1];  // 72 bytes a code row: 2-way conflicts at most
    const int tid = threadIdx.x;
    const uint32_t tr = blockIdx.x / (uint32_t)a.tile_cols;
    const int64_t r0 = (int64_t)tr * kTile, c0 = (int64_t)(blockIdx.x - tr * (uint32_t)a.tile_cols) * kTile;

    start_behind();
    Fp4Scale sc;
    if (!VEC) sc = make_fp4_scale(a.scale);  // on its way before the barriers of load_rows() (1187x2731, NVFP4: 7.1 us; 1 us more behind them)
    uint32_t w[4][8];
    // a thread's four chunks lie 32 rows apart
    const int ck = tid & 7, left = (int)min(a.rows - r0, (int64_t)kTile) - (tid >> 3);
    if constexpr (VEC) {
        const bool in = c0 + ck * 16 < a.cols;
        const uint16_t* x = a.x + (r0 + (tid >> 3)) * a.cols + c0 + ck * 16;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
            if (in && u * 32 < left) ld_once_v8(x, lo, hi);
            x += 32 * a.cols;
            w[u][0] = lo.x; w[u][1] = lo.y; w[u][2] = lo.z; w[u][3] = lo.w;
            w[u][4] = hi.x; w[u][5] = hi.y; w[u][6] = hi.z; w[u][7] = hi.w;
        }
    } else {
        load_rows(reinterpret_cast<uint4*>(xs), a.x, r0, a.rows, c0, a.cols);
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int id = u * kThreads + tid, row = id >> 3;
            const int shift = shift_of(a.x + (r0 + row) * a.cols + c0), odd = shift & 1;
            const uint32_t* p = xs + row * kGroups * 4 + (id & 7) * 8 + (shift >> 1);
            uint32_t v = p[0];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t next = odd || i < 7 ? p[i + 1] : 0u;
                w[u][i] = odd ? __byte_perm(v, next, 0x5432) : v;
                v = next;
            }
        }
        if (COL) __syncthreads();  // xs is laid out again
    }
    if (VEC) sc = make_fp4_scale(a.scale);  // behind the loads of x (8192x4096: half a us less than before them)
    uint32_t m2 = 0;
    auto run = [&](auto fast) {
        const int64_t ld = fp4_row_bytes(a.cols);
        uint8_t* q = a.q + (r0 + (tid >> 3)) * ld + c0 / 2 + ck * 8;
        const bool out = c0 + ck * 16 < 2 * ld;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int row = u * 32 + (tid >> 3);
            const uint32_t m = absmax16(w[u]);
            m2 = bf16x2_absmax(m2, m);
            if (ROW) {
                uint32_t am = max(m & 0x7FFFu, (m >> 16) & 0x7FFFu);
                if (FMT == FP8Q_MXFP4) am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
                const BlockScale b = block_scale<FMT, decltype(fast)::value>(am, sc);
                const uint2 o = block_codes<FMT>(w[u], b);
                if (out && u * 32 < left) *reinterpret_cast<uint2*>(q) = o;
                q += 32 * ld;
                if (FMT == FP8Q_NVFP4 || (ck & 1) == 0)
                    reinterpret_cast<uint8_t*>(sfs)[sf_byte(row, ck * 16 / kBlock)] = (uint8_t)b.code;
            }
            if (COL) {
                uint4* d = reinterpret_cast<uint4*>(xs + row * (kTile / 2) + ck * 8);
                d[0] = make_uint4(w[u][0], w[u][1], w[u][2], w[u][3]);
                d[1] = make_uint4(w[u][4], w[u][5], w[u][6], w[u][7]);
            }
        }
        __syncthreads();
        if (ROW) store_sf<FMT>(a.sf, sfs, r0, a.rows, c0, a.cols);
        if (COL) {
            if (ROW) __syncthreads();  // sfs is used again
            constexpr int kHalves = kBlock / 16, kUnits = kTile / kBlock;  // blocks down a column
#pragma unroll 1
            for (int id = tid; id < kUnits * (kTile / 2); id += kThreads) {
                const int p = id & 63, rb = id >> 6;  // column pair, block of rows
                uint32_t v[kHalves * 16];  // a row's two neighbours each
                uint32_t m = 0;
#pragma unroll
                for (int i = 0; i < kHalves * 16; ++i) v[i] = xs[(rb * kBlock + i) * (kTile / 2) + p];
#pragma unroll
                for (int i = 0; i < kHalves * 16; i += 2) m = bf16x2_absmax(m, bf16x2_absmax(v[i], v[i + 1]));
                const BlockScale bl = block_scale<FMT, decltype(fast)::value>(m & 0x7FFFu, sc);
                const BlockScale bh = block_scale<FMT, decltype(fast)::value>((m >> 16) & 0x7FFFu, sc);
#pragma unroll
                for (int h = 0; h < kHalves; ++h) {
                    uint32_t lo[2], hi[2];
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        Two f[4], e[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t v0 = v[h * 16 + g * 8 + 2 * i], v1 = v[h * 16 + g * 8 + 2 * i + 1];
                            f[i] = two(v0 << 16, v1 << 16);
                            e[i] = two(v0 & 0xFFFF0000u, v1 & 0xFFFF0000u);
                        }
                        lo[g] = codes8<FMT>(f, bl);
                        hi[g] = codes8<FMT>(e, bh);
                    }
                    qts[(2 * p) * 9 + rb * kHalves + h] = make_uint2(lo[0], lo[1]);
                    qts[(2 * p + 1) * 9 + rb * kHalves + h] = make_uint2(hi[0], hi[1]);
                }
                reinterpret_cast<uint8_t*>(sfs)[sf_byte(2 * p, rb)] = (uint8_t)bl.code;
                reinterpret_cast<uint8_t*>(sfs)[sf_byte(2 * p + 1, rb)] = (uint8_t)bh.code;
            }
            __syncthreads();
            store_sf<FMT>(a.sft, sfs, c0, a.cols, r0, a.rows);
            const int64_t ldt = fp4_row_bytes(a.rows);
            const int cols_left = (int)min(a.cols - c0, (int64_t)kTile) - (tid >> 3);
            uint8_t* qt = a.qt + (c0 + (tid >> 3)) * ldt + r0 / 2 + ck * 8;
            const bool in_t = r0 / 2 + ck * 8 < ldt;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (in_t && u * 32 < cols_left) *reinterpret_cast<uint2*>(qt) = qts[((tid >> 3) + u * 32) * 9 + ck];
                qt += 32 * ldt;
            }
        }
    };
    if (FMT == FP8Q_MXFP4 || sc.fast)  // the same for every thread
        run(std::true_type());
    else
        run(std::false_type());
    if (a.amax) flush_amax(m2, 0u, a.amax, red);
}

// One direction of rows that start on 32-byte boundaries: the same work on tiles
// of kWideRows x kWide columns, from registers alone, so that a CTA reads longer
// stretches of memory; scales go out by words of four blocks.  (8192x4096, NVFP4:
// 15.9 us; 2 us more, and 2.5 on tiles of 128 x 128, with every address worked out
// anew; 1024 columns measure the same.)
constexpr int kWide = 512, kWideRows = kTile * kTile / kWide;

template <int FMT>
__global__ void __launch_bounds__(kThreads) fp4_quantize_rows_kernel(const Fp4QuantArgs a) {
    constexpr int kBlock = Fp4<FMT>::kBlock, kSf = Fp4<FMT>::kSfCols;
    __shared__ uint32_t red[kThreads / 32];
    __shared__ uint32_t sfs[kWideRows * kWide / kSf];
    // a warp takes a row of the tile, every eighth: addresses advance by eight rows
    static_assert(kWide == 512 && kThreads == 256, "a warp a row");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t tr = blockIdx.x / (uint32_t)a.tile_cols;
    const int64_t r0 = (int64_t)tr * kWideRows, c0 = (int64_t)(blockIdx.x - tr * (uint32_t)a.tile_cols) * kWide;
    const int64_t ld = fp4_row_bytes(a.cols);
    const int left = (int)min(a.rows - r0, (int64_t)kWideRows) - warp;  // rows from this warp's first on
    const bool in = c0 + lane * 16 < a.cols, out = c0 + lane * 16 < 2 * ld;
    const uint16_t* x = a.x + (r0 + warp) * a.cols + c0 + lane * 16;
    uint8_t* q = a.q + (r0 + warp) * ld + c0 / 2 + lane * 8;
    start_behind();
    uint4 lo[4], hi[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        lo[u] = hi[u] = make_uint4(0, 0, 0, 0);
        if (in && u * 8 < left) ld_once_v8(x, lo[u], hi[u]);
        x += 8 * a.cols;
    }
    const Fp4Scale sc = make_fp4_scale(a.scale);
    uint32_t m2 = 0;
    auto run = [&](auto fast) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t w[8] = {lo[u].x, lo[u].y, lo[u].z, lo[u].w, hi[u].x, hi[u].y, hi[u].z, hi[u].w};
            const uint32_t m = absmax16(w);
            m2 = bf16x2_absmax(m2, m);
            uint32_t am = max(m & 0x7FFFu, (m >> 16) & 0x7FFFu);
            if (FMT == FP8Q_MXFP4) am = max(am, __shfl_xor_sync(0xFFFFFFFFu, am, 1));
            const BlockScale b = block_scale<FMT, decltype(fast)::value>(am, sc);
            const uint2 o = block_codes<FMT>(w, b);
            if (out && u * 8 < left) st_v2(q, o);
            q += 8 * ld;
            if (FMT == FP8Q_NVFP4 || (lane & 1) == 0)
                reinterpret_cast<uint8_t*>(sfs)[(warp + u * 8) * (kWide / kBlock) + lane * 16 / kBlock] = (uint8_t)b.code;
        }
    };
    if (FMT == FP8Q_MXFP4 || sc.fast)  // the same for every thread
        run(std::true_type());
    else
        run(std::false_type());
    __syncthreads();
    const int64_t across = fp4_sf_tiles<FMT>(a.cols);
    if (tid < kWideRows * kWide / kSf) {
        const int64_t r = r0 + tid / (kWide / kSf), t = c0 / kSf + tid % (kWide / kSf);
        if (r < a.rows && t < across)
            *reinterpret_cast<uint32_t*>(a.sf + ((r / 128) * across + t) * 512 + (r % 32) * 16 + (r % 128) / 32 * 4) = sfs[tid];
    }
    if (a.amax) flush_amax(m2, 0u, a.amax, red);
}

struct Fp4DequantArgs {
    const uint8_t *q, *sf;
    uint16_t* y;
    const float* scale;
    int64_t rows, cols, tile_cols;
};

// Eight codes and their block's scale byte -> eight bf16.
template <int FMT>
__device__ __forceinline__ uint4 values8(uint32_t w, uint32_t code, float s) {
    uint32_t h[4], o[4];
    e2m1x8_to_f16(w, h);
    if (FMT == FP8Q_MXFP4) {
        const float2 b = splat2(sf_value<FMT>(code));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 y = mul2_rn(make_float2(f16_lo(h[i]), f16_hi(h[i])), b);
            o[i] = cvt_bf16x2(y.x, y.y);
        }
    } else {
        // code times block scale is exact in binary16: six bits at most, from 2^-10 to 2688
        const uint32_t b = fp8x2_to_f16x2<FP8Q_E4M3FN>(code | code << 8);
        const float2 ss = splat2(s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t v;
            asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(v) : "r"(h[i]), "r"(b));
            const float2 y = mul2_rn(make_float2(f16_lo(v), f16_hi(v)), ss);
            o[i] = cvt_bf16x2(y.x, y.y);
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// Rows that start anywhere: tiles of kOddRows x kTile columns, kOddChunks of 16 a thread, through shared memory.
// (1187x2731, 8192x4095: 4.7 and 25.9 us; 5.3 and 27.5 with one chunk, 6.3 and 27.0 with four.)
constexpr int kOddChunks = 2, kOddRows = kThreads * kOddChunks * 16 / kTile;

template <int FMT>
__global__ void __launch_bounds__(kThreads) fp4_dequantize_kernel(const Fp4DequantArgs a) {
    __shared__ uint4 raw[kOddRows * kGroups];
    const int ck = threadIdx.x & 7;
    const uint32_t tr = blockIdx.x / (uint32_t)a.tile_cols;
    const int64_t r0 = (int64_t)tr * kOddRows, c0 = (int64_t)(blockIdx.x - tr * (uint32_t)a.tile_cols) * kTile;
    const int64_t c = c0 + ck * 16, block = c / Fp4<FMT>::kBlock;
    start_behind();
    const float s = a.scale ? *a.scale : 1.0f;
    uint2 w[kOddChunks];
    uint32_t code[kOddChunks];
#pragma unroll
    for (int u = 0; u < kOddChunks; ++u) {
        const int64_t r = r0 + u * (kThreads / 8) + (threadIdx.x >> 3);
        w[u] = make_uint2(0, 0);
        code[u] = 0;
        if (r < a.rows && c < a.cols) {
            w[u] = ld_once_v2(a.q + r * fp4_row_bytes(a.cols) + c / 2);
            code[u] = a.sf[(r / 128 * fp4_sf_tiles<FMT>(a.cols) + block / 4) * 512 + (r % 32) * 16 + (r % 128) / 32 * 4 + block % 4];
        }
    }
#pragma unroll
    for (int u = 0; u < kOddChunks; ++u) {
        const int row = u * (kThreads / 8) + (threadIdx.x >> 3);
        const uint4 v0 = values8<FMT>(w[u].x, code[u], s), v1 = values8<FMT>(w[u].y, code[u], s);
        const uint32_t o[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
        const int shift = shift_of(a.y + (r0 + row) * a.cols + c0);
        uint32_t* p = reinterpret_cast<uint32_t*>(raw + row * kGroups) + ck * 8 + (shift >> 1);
        if (shift & 1) {  // half a word on: this chunk's first element is its neighbour's last half-word
            uint16_t* h = reinterpret_cast<uint16_t*>(p);
            h[1] = (uint16_t)o[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) p[i] = __byte_perm(o[i - 1], o[i], 0x5432);
            h[16] = (uint16_t)(o[7] >> 16);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = o[i];
        }
    }
    __syncthreads();
    const int n = (int)min(a.cols - c0, (int64_t)kTile);
#pragma unroll
    for (int i = threadIdx.x; i < kOddRows * kGroups; i += kThreads) {
        const int k = i / kGroups;
        if (r0 + k >= a.rows) break;
        uint16_t* first = a.y + (r0 + k) * a.cols + c0;
        const int e = (i - k * kGroups) * 8 - shift_of(first);  // the group's first element
        const uint4 v = raw[i];
        if (e >= 0 && e + 8 <= n) {
            st_v4(first + e, v);
        } else {
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int f = e + 2 * j;
                if (f >= 0 && f + 1 < n) {
                    *reinterpret_cast<uint32_t*>(first + f) = u[j];
                } else {
                    if (f >= 0 && f < n) first[f] = (uint16_t)u[j];
                    if (f + 1 >= 0 && f + 1 < n) first[f + 1] = (uint16_t)(u[j] >> 16);
                }
            }
        }
    }
}

// Rows that start on 16-byte boundaries: tiles of kOutRows x kOut columns, eight
// columns a thread at a time, so that a warp's stores are one stretch (8192x4096,
// NVFP4: 14.0 us; half a us more with two chunks a thread, 2.5 with sixteen columns at a time).
constexpr int kOut = 1024, kOutChunks = 4, kOutRows = kThreads * kOutChunks * 8 / kOut;

template <int FMT>
__global__ void __launch_bounds__(kThreads) fp4_dequantize_rows_kernel(const Fp4DequantArgs a) {
    constexpr int kBlock = Fp4<FMT>::kBlock, kSf = Fp4<FMT>::kSfCols;
    __shared__ uint32_t sfs[kOutRows * kOut / kSf];
    // half a CTA takes a row of the tile, every second: addresses advance by two rows
    static_assert(kOut == 1024 && kThreads == 256, "128 threads a row");
    const int tid = threadIdx.x, t = tid & 127, row0 = tid >> 7;
    const uint32_t tr = blockIdx.x / (uint32_t)a.tile_cols;
    const int64_t r0 = (int64_t)tr * kOutRows, c0 = (int64_t)(blockIdx.x - tr * (uint32_t)a.tile_cols) * kOut;
    const int64_t ld = fp4_row_bytes(a.cols), across = fp4_sf_tiles<FMT>(a.cols);
    const int left = (int)min(a.rows - r0, (int64_t)kOutRows) - row0;
    const bool in = c0 + t * 8 < a.cols;
    const uint8_t* q = a.q + (r0 + row0) * ld + c0 / 2 + t * 4;
    uint16_t* y = a.y + (r0 + row0) * a.cols + c0 + t * 8;
    start_behind();
    const float s = a.scale ? *a.scale : 1.0f;
    uint32_t w[kOutChunks];
#pragma unroll
    for (int u = 0; u < kOutChunks; ++u) {
        w[u] = 0;
        if (in && u * 2 < left) w[u] = *reinterpret_cast<const unsigned int*>(q);
        q += 2 * ld;
    }
    for (int i = tid; i < kOutRows * kOut / kSf; i += kThreads) {
        const int64_t r = r0 + i / (kOut / kSf), k = c0 / kSf + i % (kOut / kSf);
        if (r < a.rows && k < across)
            sfs[i] = *reinterpret_cast<const unsigned int*>(a.sf + ((r / 128) * across + k) * 512 + (r % 32) * 16 + (r % 128) / 32 * 4);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kOutChunks; ++u) {
        if (in && u * 2 < left)
            st_v4(y, values8<FMT>(w[u], reinterpret_cast<const uint8_t*>(sfs)[(row0 + u * 2) * (kOut / kBlock) + t * 8 / kBlock], s));
        y += 2 * a.cols;
    }
}

template <int FMT, bool VEC>
fp8q_status launch_quantize(const Fp4QuantArgs& a, unsigned grid, cudaStream_t s) {
    auto kern = fp4_quantize_kernel<FMT, false, true, VEC>;
    if (a.q && a.qt)
        kern = fp4_quantize_kernel<FMT, true, true, VEC>;
    else if constexpr (!VEC) {
        if (a.q) kern = fp4_quantize_kernel<FMT, true, false, false>;
    }
    return launch_behind(kern, dim3(grid), dim3(kThreads), 0, 1, s, "fp4_quantize_kernel", a);
}

// Tiles of an [rows, cols] matrix; 0 where there are more than a grid holds.
unsigned tile_grid(int64_t rows, int64_t cols, int64_t tile_rows = kTile) {
    const int64_t tr = (rows + tile_rows - 1) / tile_rows, tc = (cols + kTile - 1) / kTile;
    return tr <= 0x7FFFFFFF / tc ? (unsigned)(tr * tc) : 0u;
}

}  // namespace

extern "C" {

int64_t fp8q_fp4_row_bytes(int64_t cols) { return cols > 0 && cols <= kFp4MaxDim ? fp4_row_bytes(cols) : 0; }

int64_t fp8q_fp4_scale_bytes(int64_t rows, int64_t cols, fp8q_format fmt) {
    if (rows <= 0 || cols <= 0 || rows > kFp4MaxDim || cols > kFp4MaxDim || !valid_fp4(fmt)) return 0;
    return (rows + 127) / 128 * (fmt == FP8Q_MXFP4 ? fp4_sf_tiles<FP8Q_MXFP4>(cols) : fp4_sf_tiles<FP8Q_NVFP4>(cols)) * 512;
}

fp8q_status fp8q_fp4_quantize_amax(const void* x_bf16, int64_t rows, int64_t cols, uint8_t* q, uint8_t* sf, uint8_t* qt,
                                   uint8_t* sft, fp8q_format fmt, const float* scale, float* amax, void* stream) {
    if (!valid_fp4(fmt) || rows < 0 || cols < 0) return FP8Q_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return FP8Q_OK;
    if (rows > kFp4MaxDim || cols > kFp4MaxDim) return FP8Q_ERR_UNSUPPORTED;
    if (!x_bf16 || (!q != !sf) || (!qt != !sft) || (!q && !qt)) return FP8Q_ERR_INVALID_ARG;
    if (fmt == FP8Q_MXFP4 && scale) return FP8Q_ERR_INVALID_ARG;
    if (((uintptr_t)x_bf16 & 1u) || ((uintptr_t)scale & 3u) || ((uintptr_t)amax & 3u)) return FP8Q_ERR_INVALID_ARG;
    if (((uintptr_t)q | (uintptr_t)sf | (uintptr_t)qt | (uintptr_t)sft) & 15u) return FP8Q_ERR_UNSUPPORTED;
    const unsigned grid = tile_grid(rows, cols);
    if (!grid) return FP8Q_ERR_UNSUPPORTED;
    Fp4QuantArgs a;
    a.x = static_cast<const uint16_t*>(x_bf16);
    a.q = q;
    a.sf = sf;
    a.qt = qt;
    a.sft = sft;
    a.scale = scale;
    a.amax = amax;
    a.rows = rows;
    a.cols = cols;
    a.tile_cols = (cols + kTile - 1) / kTile;
    // rows of whole 16-column chunks on 32-byte boundaries load straight into registers
    const bool vec = cols % 16 == 0 && ((uintptr_t)x_bf16 & 31u) == 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (vec && !qt) {
        a.tile_cols = (cols + kWide - 1) / kWide;
        const int64_t tiles = (rows + kWideRows - 1) / kWideRows * a.tile_cols;
        if (tiles > 0x7FFFFFFF) return FP8Q_ERR_UNSUPPORTED;
        return launch_behind(fmt == FP8Q_MXFP4 ? fp4_quantize_rows_kernel<FP8Q_MXFP4> : fp4_quantize_rows_kernel<FP8Q_NVFP4>,
                             dim3((unsigned)tiles), dim3(kThreads), 0, 1, s, "fp4_quantize_rows_kernel", a);
    }
    if (fmt == FP8Q_MXFP4) return vec ? launch_quantize<FP8Q_MXFP4, true>(a, grid, s) : launch_quantize<FP8Q_MXFP4, false>(a, grid, s);
    return vec ? launch_quantize<FP8Q_NVFP4, true>(a, grid, s) : launch_quantize<FP8Q_NVFP4, false>(a, grid, s);
}

fp8q_status fp8q_fp4_dequantize(const uint8_t* q, const uint8_t* sf, void* y_bf16, int64_t rows, int64_t cols,
                                fp8q_format fmt, const float* scale, void* stream) {
    if (!valid_fp4(fmt) || rows < 0 || cols < 0) return FP8Q_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return FP8Q_OK;
    if (rows > kFp4MaxDim || cols > kFp4MaxDim) return FP8Q_ERR_UNSUPPORTED;
    if (!q || !sf || !y_bf16 || (fmt == FP8Q_MXFP4 && scale)) return FP8Q_ERR_INVALID_ARG;
    if (((uintptr_t)y_bf16 & 1u) || ((uintptr_t)scale & 3u)) return FP8Q_ERR_INVALID_ARG;
    if (((uintptr_t)q | (uintptr_t)sf) & 15u) return FP8Q_ERR_UNSUPPORTED;
    const unsigned grid = tile_grid(rows, cols, kOddRows);
    if (!grid) return FP8Q_ERR_UNSUPPORTED;
    Fp4DequantArgs a;
    a.q = q;
    a.sf = sf;
    a.y = static_cast<uint16_t*>(y_bf16);
    a.scale = scale;
    a.rows = rows;
    a.cols = cols;
    a.tile_cols = (cols + kTile - 1) / kTile;
    const bool vec = cols % 16 == 0 && ((uintptr_t)y_bf16 & 15u) == 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (vec) {
        a.tile_cols = (cols + kOut - 1) / kOut;
        const int64_t tiles = (rows + kOutRows - 1) / kOutRows * a.tile_cols;
        if (tiles > 0x7FFFFFFF) return FP8Q_ERR_UNSUPPORTED;
        return launch_behind(fmt == FP8Q_MXFP4 ? fp4_dequantize_rows_kernel<FP8Q_MXFP4> : fp4_dequantize_rows_kernel<FP8Q_NVFP4>,
                             dim3((unsigned)tiles), dim3(kThreads), 0, 1, s, "fp4_dequantize_rows_kernel", a);
    }
    auto kern = fmt == FP8Q_MXFP4 ? fp4_dequantize_kernel<FP8Q_MXFP4> : fp4_dequantize_kernel<FP8Q_NVFP4>;
    return launch_behind(kern, dim3(grid), dim3(kThreads), 0, 1, s, "fp4_dequantize_kernel", a);
}

}  // extern "C"
