// fp4_matmul.cu -- the product of two microscaled 4-bit operands on the tensor
// cores.
//
//   D[m][n] = RN_out( (sum_k A[m][k] B[n][k]) * RN(sa * sb) )
//
// Both operands are packed along k (fp4.cuh).  Codes come into shared memory by
// tensor-map copies (256 codes of k a step, 128 bytes a row, 128-byte swizzle,
// zeros beyond the edges), block scales by plain bulk copies of whole scale
// tiles, which already lie as tensor memory takes them; one thread issues the
// copies, another the block-scaled multiply-adds; other warps
// store the scales to tensor memory and carry the accumulators out.
//
// Two kernels.  Few tiles: 128 rows of P by 16 to 128 of Q a CTA, k split over a
// cluster while every CTA is resident; what bounds them is the operands' way from
// HBM, and at these sizes the time until it flows: 1 x 16384 x 4096 (37.7 MB) 9.5 us,
// 4.0 TB/s; 1 x 4096 x 4096 (9.4 MB) 4.6 us; each megabyte more costs 0.17 us, 5.8 TB/s.
// Many tiles: pairs of CTAs with 256 x 256 (below).  8192 x 16384 x 4096 takes 173 us
// (MXFP4 166), 6.4 PFLOP/s, of which the multiply-adds alone, 128 cycles for
// 256 x 256 x 64, are 107 us at 2070 MHz: a step of 256 codes takes 0.29 us where they
// take 0.25, and between tiles the tensor cores wait 0.9 to 1.4 us for the accumulators'
// way out.  In a loop seconds long the power limit comes on top: 198 us at 1400 W and 1690 MHz.
// Single CTAs take 507 us of it; pairs from more 128 x 128 tiles than SMs
// on, 2560 x 1280 x 4096 10.5 us (17.1 on single CTAs), 2560 x 2560 x 4096 16.5 (26.7).
// (All with operands in rotation beyond L2, replayed from a graph.)

#include "tcgen05.cuh"

namespace {

constexpr int kStepBytes = 128;  // bytes of codes a row and step
constexpr int kStages = 4;

// "P" is the operand whose rows are the accumulator's 128 lanes, "Q" the one
// whose rows are its BN columns.
struct MmArgs {
    const uint8_t *p_sf, *q_sf;
    const float *sa, *sb;
    void* d;
    int64_t ld;          // D's row length
    int32_t p_rows, q_rows;
    int32_t ksteps;      // steps of 64 codes
    int32_t sf_across;   // scale tiles along k
    int32_t q_tiles;     // tiles of Q
    int32_t split;       // CTAs (of one cluster) that share a tile's k
    int32_t p_is_m;      // P's rows are D's rows
    int32_t vec;         // D's rows hold 16-byte groups
#ifdef FP8Q_TEST_HOOKS
    int32_t fail_role, fail_at, fail_cta;  // the wait that reports failure although what it waits for has come
#endif
};

// The waits, by who waits for what; a test makes one of them run out.
enum MmWait { kNoWait, kCopyEmpty, kSumFull, kSumScaled, kScaleFull, kOutDone, kScaleCopyEmpty, kSumDrained };
__device__ __forceinline__ bool made_to_fail(const MmArgs& a, MmWait role, uint32_t at) {
#ifdef FP8Q_TEST_HOOKS
    return a.fail_role == role && a.fail_at == (int)at && (a.fail_cta < 0 || a.fail_cta == (int)blockIdx.x);
#else
    return false;
#endif
}
// One wait of a whole warp, with one verdict.
__device__ __forceinline__ bool wait_of(const MmArgs& a, MmWait role, uint32_t at, uint64_t* bar, uint32_t parity) {
    return mbar_wait_all(bar, parity, made_to_fail(a, role, at) && (threadIdx.x & 31) == 5);
}

template <int FMT, int BN>
struct MmGeom {
    static constexpr int kSfTiles = FMT == FP8Q_MXFP4 ? 2 : 4;  // scale tiles a step and 128 rows
    static constexpr int kPBytes = 128 * kStepBytes, kQBytes = BN * kStepBytes;
    static constexpr int kStageBytes = kPBytes + kQBytes + 2 * kSfTiles * 512;
    static constexpr int kSmem = kStages * kStageBytes + 1024;  // and room to start on 1024 bytes
    static constexpr int kAccCols = BN < 32 ? 32 : BN;
    static constexpr int kSfCols = kSfTiles * 4 * 2;          // tensor memory columns a stage
    static constexpr int kNeed = kAccCols + kStages * kSfCols;
    static constexpr int kCols = kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
};

template <bool F32>
__device__ __forceinline__ void store_one(void* d, int64_t at, float v) {
    if (F32)
        static_cast<float*>(d)[at] = v;
    else
        static_cast<uint16_t*>(d)[at] = (uint16_t)(cvt_bf16x2(v, 0.0f) & 0xFFFFu);
}

// Sixteen columns of one row of D.
template <bool F32>
__device__ __forceinline__ void store_row16(void* d, int64_t at, const float (&v)[16], int n, bool vec) {
    if (vec && n >= 16) {
        if (F32) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(d) + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        } else {
            uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(d) + at);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                o[i] = make_uint4(cvt_bf16x2(v[8 * i], v[8 * i + 1]), cvt_bf16x2(v[8 * i + 2], v[8 * i + 3]),
                                  cvt_bf16x2(v[8 * i + 4], v[8 * i + 5]), cvt_bf16x2(v[8 * i + 6], v[8 * i + 7]));
        }
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (i < n) store_one<F32>(d, at + i, v[i]);
    }
}

// This CTA's share of a tile's sums, added over the SPLIT CTAs of the cluster in rank order, four rows a thread, BATCH such
// groups on their way at a time: a read of another CTA's memory takes hundreds of cycles (256x4096x8192 11.1 us,
// 12.7 with one group at a time).
template <bool F32, int SPLIT, int BATCH>
__device__ __forceinline__ void add_shares(const MmArgs& a, uint32_t part, int bn, int rank, int p0, int q0, float alpha) {
    const int share = bn * 32 / SPLIT, end = (rank + 1) * share;
    for (int i0 = rank * share + (int)threadIdx.x; i0 < end; i0 += 192 * BATCH) {
        float4 v[BATCH][SPLIT];
#pragma unroll
        for (int b = 0; b < BATCH; ++b)
            if (i0 + 192 * b < end)
#pragma unroll
                for (int r = 0; r < SPLIT; ++r) v[b][r] = ld_cluster_f32x4(in_cluster(part + (i0 + 192 * b) * 16, r));
#pragma unroll
        for (int b = 0; b < BATCH; ++b) {
            const int i = i0 + 192 * b, q = q0 + (i >> 5), p = p0 + (i & 31) * 4;
            if (i >= end) break;
            float f[4] = {v[b][0].x, v[b][0].y, v[b][0].z, v[b][0].w};
#pragma unroll
            for (int r = 1; r < SPLIT; ++r) f[0] += v[b][r].x, f[1] += v[b][r].y, f[2] += v[b][r].z, f[3] += v[b][r].w;
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = __fmul_rn(f[k], alpha);
            const int64_t at = (int64_t)q * a.ld + p;  // split tiles have D's rows along P
            if (q < a.q_rows && a.vec && p < a.p_rows) {
                if (F32)
                    *reinterpret_cast<float4*>(static_cast<float*>(a.d) + at) = make_float4(f[0], f[1], f[2], f[3]);
                else
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.d) + at) = make_uint2(cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]));
            } else if (q < a.q_rows) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (p + k < a.p_rows) store_one<F32>(a.d, at + k, f[k]);
            }
        }
    }
}

template <int FMT, int BN, bool F32>
__global__ void __launch_bounds__(192) fp4_matmul_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                                                         const MmArgs a) {
    using G = MmGeom<FMT, BN>;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full[kStages], scaled[kStages], empty[kStages], done;
    __shared__ uint32_t tmem_slot, loads;
    __shared__ int gave_up;
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    const int rank = a.split > 1 ? (int)(blockIdx.x % a.split) : 0;
    const int tile = blockIdx.x / a.split;
    const int p0 = tile / a.q_tiles * 128, q0 = tile % a.q_tiles * BN;
    // this CTA's steps of 256 codes
    const int steps = (a.ksteps + 3) / 4;
    const int s0 = (int)((int64_t)steps * rank / a.split), s1 = (int)((int64_t)steps * (rank + 1) / a.split);

    if (threadIdx.x == 128) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i]);
            mbar_init_count(&scaled[i], 4);
            mbar_init(&empty[i]);
        }
        mbar_init(&done);
        loads = 0;
        gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
    wait_behind();
    if (warp == 5) {
        tmem_alloc<1>(&tmem_slot, G::kCols);
        let_next_start();
    }
    uint32_t tmem = 0;
    if (warp != 4) {  // copies start without it
        tc_fence_before();
        some_sync<5 * 32>();
        tc_fence_after();
        tmem = tmem_slot;
    }

    if (warp == 4) {
        const uint8_t* psf = a.p_sf + (int64_t)(p0 / 128) * a.sf_across * 512;
        const uint8_t* qsf = a.q_sf + (int64_t)(q0 / 128) * a.sf_across * 512;
        uint32_t st = 0, round = 0, n = 0;
        bool ok = true;
        for (int s = s0; s < s1; ++s, ++n) {
            if (!wait_of(a, kCopyEmpty, n, &empty[st], (round & 1) ^ 1)) {
                ok = false;
                break;
            }
            const uint32_t at = base + st * G::kStageBytes, sf = at + G::kPBytes + G::kQBytes;
            const int t0 = s * G::kSfTiles, nt = min(G::kSfTiles, a.sf_across - t0);
            if (elect_lane()) {
                expect_bytes(&full[st], G::kPBytes + G::kQBytes + nt * 512 * 2);
                tile_load(at, &map_p, s * kStepBytes, p0, &full[st]);
                tile_load(at + G::kPBytes, &map_q, s * kStepBytes, q0, &full[st]);
                block_load(sf, psf + (int64_t)t0 * 512, nt * 512, &full[st]);
                block_load(sf + G::kSfTiles * 512, qsf + (int64_t)t0 * 512, nt * 512, &full[st]);
            }
            __syncwarp();
            if (++st == kStages) st = 0, ++round;
        }
        // the tensor core's last arrivals land before the CTA may go
        for (uint32_t i = n > kStages ? n - kStages : 0; i < n && ok; ++i) ok = mbar_wait_all(&empty[i % kStages], (i / kStages) & 1);
        if (lane == 0) {
            if (!ok) gave_up = 1;
            loads = n;
        }
    } else if (warp == 5) {
        uint32_t st = 0, round = 0;
        bool ok = true;
        for (int s = s0; s < s1; ++s) {
            if (!wait_of(a, kSumFull, s - s0, &full[st], round & 1) || !wait_of(a, kSumScaled, s - s0, &scaled[st], round & 1)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const int nk = min(4, a.ksteps - s * 4);
            const uint32_t at = base + st * G::kStageBytes;
            const uint64_t dp = desc_codes(at), dq = desc_codes(at + G::kPBytes);
            const uint32_t tp = tmem + G::kAccCols + st * G::kSfCols, tq = tp + G::kSfTiles * 4;
            if (elect_lane()) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int t = FMT == FP8Q_MXFP4 ? k >> 1 : k;
                    constexpr uint32_t kEven = mma_desc<FMT>(128, BN, 0), kOdd = mma_desc<FMT>(128, BN, 2);
                    if (k < nk)  // a step of 64 codes is 32 bytes on
                        tc_mma<FMT, 1>(tmem, dp + k * 2, dq + k * 2, FMT == FP8Q_MXFP4 && (k & 1) ? kOdd : kEven, tp + t * 4, tq + t * 4,
                                       (s - s0) | k);
                }
                tc_commit(&empty[st]);
                if (s == s1 - 1) tc_commit(&done);
            }
            __syncwarp();
            if (++st == kStages) st = 0, ++round;
        }
        if (!ok && elect_lane()) {
            tc_commit(&done);
            gave_up = 1;
        }
    } else {
        uint32_t st = 0, round = 0;
        bool ok = true;
        for (int s = s0; s < s1; ++s) {
            if (!wait_of(a, kScaleFull, s - s0, &full[st], round & 1)) {
                ok = false;
                break;
            }
            const uint32_t sf = base + st * G::kStageBytes + G::kPBytes + G::kQBytes;
            const uint32_t to = tmem + ((uint32_t)(warp * 32) << 16) + G::kAccCols + st * G::kSfCols;
            if constexpr (FMT == FP8Q_MXFP4) {
                store_scales4(to, sf, 512);  // P's and Q's two
            } else {
                store_scales4(to, sf, 512);
                store_scales4(to + 16, sf + 2048, 512);
            }
            scales_stored();
            if (lane == 0) arrive_local(&scaled[st]);
            if (++st == kStages) st = 0, ++round;
        }
        if (!mbar_wait_warp(&done, 0, 0) || made_to_fail(a, kOutDone, 0) || !ok) gave_up = 1;
    }
    __syncwarp();
    __syncthreads();
    tc_fence_after();
    const float alpha = __fmul_rn(a.sa ? *a.sa : 1.0f, a.sb ? *a.sb : 1.0f);
    // A wait that ran out (correct operation never gets there) shows as NaN in the whole tile.
    const float nan = __uint_as_float(0x7FFFFFFFu);
    const int bad = gave_up;
    if (bad) {  // copies still under way end before the CTA does, and before sums (and NaN) lie where they go
        if (threadIdx.x == 0)
            for (uint32_t n = loads > kStages ? loads - kStages : 0; n < loads; ++n) mbar_wait(&full[n % kStages], (n / kStages) & 1);
        __syncthreads();
    }
    if (a.split == 1) {
        if (warp < 4) {
            const int p = p0 + warp * 32 + lane;
            const uint32_t row = tmem + ((uint32_t)(warp * 32) << 16);
#pragma unroll 1
            for (int c = 0; c < BN; c += 16) {
                float v[16];
                tmem_load16(row + c, v);
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = bad ? nan : __fmul_rn(v[i], alpha);
                const int left = a.q_rows - (q0 + c);
                if (p < a.p_rows && left > 0) {
                    if (a.p_is_m) {
                        store_row16<F32>(a.d, (int64_t)p * a.ld + q0 + c, v, left, a.vec);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (i < left) store_one<F32>(a.d, (int64_t)(q0 + c + i) * a.ld + p, v[i]);
                    }
                }
                __syncwarp();
            }
        }
    } else {
        // the partial sums in shared memory, a column's 128 rows side by side; each CTA adds its
        // share of them over the cluster in rank order, four rows a thread
        if (warp < 4) {
            float* part = reinterpret_cast<float*>(raw + (base - smem_addr(raw)));
            const uint32_t row = tmem + ((uint32_t)(warp * 32) << 16);
#pragma unroll 1
            for (int c = 0; c < BN; c += 16) {
                float v[16];
                tmem_load16(row + c, v);
#pragma unroll
                for (int i = 0; i < 16; ++i) part[(c + i) * 128 + warp * 32 + lane] = bad ? nan : v[i];
            }
        }
        cluster_sync_all();
        switch (a.split) {
            case 2: add_shares<F32, 2, 4>(a, base, BN, rank, p0, q0, alpha); break;
            case 4: add_shares<F32, 4, 2>(a, base, BN, rank, p0, q0, alpha); break;
            default: add_shares<F32, 8, 2>(a, base, BN, rank, p0, q0, alpha);
        }
        cluster_sync_all();  // no CTA's sums go away while another reads them
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) tmem_free<1>(tmem, G::kCols);
}

// ----------------------------------------------------------------------------
// Pairs: two CTAs of a cluster share tiles of 256 x 256.  Each holds 128 rows of
// P and of Q and the accumulators of its own rows of P; the first issues the
// multiply-adds for both, so a row of Q is read from shared memory once for 256
// rows of P.  Persistent: the copies of the next tile run on while this one's
// accumulators go out, and the tensor cores wait only until these are in
// registers.

constexpr int kPairStages = 5;
constexpr int kPairThreads = 608;  // warps 0-7 carry results out, 8 copies codes, 9 multiplies, 10-17 store scales, 18 copies scales

template <int FMT>
struct PairGeom {
    static constexpr int kSfTiles = FMT == FP8Q_MXFP4 ? 2 : 4;
    static constexpr int kCodeBytes = 128 * kStepBytes;  // of P and of Q
    static constexpr int kStageBytes = 2 * kCodeBytes + 3 * kSfTiles * 512;
    static constexpr int kOutBytes = 8 * 4096;  // 32 rows of 128 bytes for each warp that carries results out
    static constexpr int kSmem = kPairStages * kStageBytes + kOutBytes + 1024;
    static constexpr int kSfCols = 3 * kSfTiles * 4;
};

// Rows of D that start anywhere: 32 swizzled lines of 128 bytes in shared memory go out a line at a time, a lane a
// 32-bit word, the words as they are aligned in D.  `rows` and `n` elements of a row are there, from `first` on.
// (8192 x 16383 x 4096: 240 us; 362 by single elements, whose half-filled sectors cost the memory a read each.)
template <bool F32>
__device__ __forceinline__ void store_rows(void* d, int64_t first, int64_t ld, int rows, int n, uint32_t lines) {
    const int lane = threadIdx.x & 31;
    uint8_t* row = static_cast<uint8_t*>(d) + first * (F32 ? 4 : 2);
    for (int r0 = 0; r0 < min(rows, 32); r0 += 8) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[j]) : "r"(lines + (r0 + j) * 128 + ((((uint32_t)lane >> 2) ^ j) << 4) + (lane & 3) * 4) : "memory");
#pragma unroll
        for (int j = 0; j < 8; ++j, row += ld * (F32 ? 4 : 2)) {
            if (r0 + j >= rows) break;
            uint16_t* h = reinterpret_cast<uint16_t*>(row);
            if (F32) {
                if (lane < n) reinterpret_cast<uint32_t*>(row)[lane] = w[j];
            } else if (n < 64) {  // elements 2 lane and 2 lane + 1
                if (2 * lane < n) h[2 * lane] = (uint16_t)w[j];
                if (2 * lane + 1 < n) h[2 * lane + 1] = (uint16_t)(w[j] >> 16);
            } else if ((uintptr_t)row & 2) {  // the same for the warp: a word in D holds elements 2 lane - 1 and 2 lane
                const uint32_t v = __byte_perm(__shfl_up_sync(0xFFFFFFFFu, w[j], 1), w[j], 0x5432);
                if (lane) reinterpret_cast<uint32_t*>(h - 1)[lane] = v;
                if (lane == 0) h[0] = (uint16_t)w[j];
                if (lane == 31) h[63] = (uint16_t)(w[j] >> 16);
            } else {
                reinterpret_cast<uint32_t*>(row)[lane] = w[j];
            }
        }
    }
}

template <int FMT, bool F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads)
    fp4_matmul_pair_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                           const __grid_constant__ CUtensorMap map_psf, const __grid_constant__ CUtensorMap map_qsf,
                           const __grid_constant__ CUtensorMap map_d, const MmArgs a) {
    using G = PairGeom<FMT>;
    extern __shared__ uint8_t raw[];
    // full: the codes of a stage are there in both CTAs and its scales in both tensor memories (the first CTA's counts);
    // sf_full: this CTA's scales are in shared memory; empty: the stage has been used; done: a tile's sums are
    // complete; stopped: the multiply-adds of an issuer that gave up have ended
    __shared__ uint64_t full[kPairStages], sf_full[kPairStages], empty[kPairStages], done, drained, stopped;
    __shared__ uint32_t tmem_slot, loads, sf_loads;
    __shared__ int gave_up;
    const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    const uint32_t rank = cluster_rank();
    const int p_tiles = (a.p_rows + 255) / 256, tiles = p_tiles * a.q_tiles, stride = gridDim.x / 2;
    const int steps = (a.ksteps + 3) / 4;

    if (threadIdx.x == 0) {
        prefetch_map(&map_p);
        prefetch_map(&map_q);
        prefetch_map(&map_psf);
        prefetch_map(&map_qsf);
        for (int i = 0; i < kPairStages; ++i) {
            mbar_init_count(&full[i], 1 + 8);
            mbar_init(&sf_full[i]);
            mbar_init(&empty[i]);
        }
        mbar_init(&done);
        mbar_init(&stopped);
        mbar_init_count(&drained, 16);
        loads = sf_loads = 0;
        gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
    cluster_sync_all();  // both CTAs' barriers are there
    wait_behind();
    if (warp == 9) {
        tmem_alloc<2>(&tmem_slot, 512);
        let_next_start();
    }
    uint32_t tmem = 0;
    if (warp != 8 && warp != 18) {  // copies start without it; no multiply-add starts before both CTAs' scale warps come from here
        tc_fence_before();
        some_sync<kPairThreads - 2 * 32>();
        tc_fence_after();
        tmem = tmem_slot;
    }

    if (warp == 8) {
        uint32_t st = 0, round = 0, n = 0;
        bool ok = true;
        const uint32_t bars = in_cluster(smem_addr(&full[0]), 0);
        for (int tile = blockIdx.x / 2; tile < tiles && ok; tile += stride) {
            const PairTile t = pair_tile(tile, p_tiles, a.q_tiles);
            const int p0 = t.p + (int)rank * 128, q0 = t.q + (int)rank * 128;
            for (int s = 0; s < steps; ++s, ++n) {
                if (!wait_of(a, kCopyEmpty, n, &empty[st], (round & 1) ^ 1)) {
                    ok = false;
                    break;
                }
                const uint32_t at = base + st * G::kStageBytes, bar = bars + st * 8;
                if (elect_lane()) {
                    if (rank == 0) expect_bytes(&full[st], 4 * G::kCodeBytes);
                    tile_load_pair(at, &map_p, s * kStepBytes, p0, bar);
                    tile_load_pair(at + G::kCodeBytes, &map_q, s * kStepBytes, q0, bar);
                }
                __syncwarp();
                if (++st == kPairStages) st = 0, ++round;
            }
        }
        // The tensor cores' last arrivals land before this CTA may go.
        for (uint32_t i = 0; i < kPairStages && i < n && ok; ++i) {
            st = st ? st - 1 : kPairStages - 1;
            ok = mbar_wait_all(&empty[st], ((n - 1 - i) / kPairStages) & 1);
        }
        if (lane == 0) {
            if (!ok) gave_up = 1;
            loads = n;
        }
    } else if (warp == 18) {
        uint32_t st = 0, round = 0, n = 0;
        bool ok = true;
        for (int tile = blockIdx.x / 2; tile < tiles && ok; tile += stride) {
            const PairTile t = pair_tile(tile, p_tiles, a.q_tiles);
            for (int s = 0; s < steps; ++s, ++n) {
                if (!wait_of(a, kScaleCopyEmpty, n, &empty[st], (round & 1) ^ 1)) {
                    ok = false;
                    break;
                }
                const uint32_t sf = base + st * G::kStageBytes + 2 * G::kCodeBytes;
                if (elect_lane()) {
                    expect_bytes(&sf_full[st], 3 * G::kSfTiles * 512);
                    tile_load(sf, &map_psf, s * G::kSfTiles * 64, t.p / 128 + (int)rank, &sf_full[st]);
                    tile_load(sf + G::kSfTiles * 512, &map_qsf, s * G::kSfTiles * 64, t.q / 128, &sf_full[st]);
                }
                __syncwarp();
                if (++st == kPairStages) st = 0, ++round;
            }
        }
        if (lane == 0) {
            if (!ok) gave_up = 1;
            sf_loads = n;
        }
    } else if (warp == 9) {
        if (rank == 0) {
            uint32_t st = 0, round = 0, it = 0;
            bool ok = true;
            for (int tile = blockIdx.x / 2; tile < tiles && ok; tile += stride, ++it) {
                if (it > 0 && !wait_of(a, kSumDrained, it, &drained, (it - 1) & 1)) {
                    ok = false;
                    break;
                }
                for (int s = 0; s < steps; ++s) {
                    if (!wait_of(a, kSumFull, it * steps + s, &full[st], round & 1)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const int nk = min(4, a.ksteps - s * 4);
                    const uint32_t at = base + st * G::kStageBytes;
                    const uint64_t dp = desc_codes(at), dq = desc_codes(at + G::kCodeBytes);
                    const uint32_t tp = tmem + 256 + st * G::kSfCols, tq = tp + G::kSfTiles * 4;
                    if (elect_lane()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int t = FMT == FP8Q_MXFP4 ? k >> 1 : k;
                            constexpr uint32_t kEven = mma_desc<FMT>(256, 256, 0), kOdd = mma_desc<FMT>(256, 256, 2);
                            if (k < nk)  // a step of 64 codes is 32 bytes on
                                tc_mma<FMT, 2>(tmem, dp + k * 2, dq + k * 2, FMT == FP8Q_MXFP4 && (k & 1) ? kOdd : kEven, tp + t * 4,
                                               tq + t * 8, s | k);
                        }
                        tc_commit_pair(&empty[st], 3);
                        if (s == steps - 1) tc_commit_pair(&done, 3);
                    }
                    __syncwarp();
                    if (++st == kPairStages) st = 0, ++round;
                }
            }
            // The other CTA's last arrivals land before this one may go.
            if (ok && it > 0) ok = mbar_wait_all(&drained, (it - 1) & 1);
            // An unfinished tile is never announced as done: those who carry results out run out of time in their
            // turn, in both CTAs, and write NaN.
            if (!ok) {
                if (elect_lane()) {
                    tc_commit_pair(&stopped, 1);
                    gave_up = 1;
                }
                __syncwarp();
                mbar_wait_all(&stopped, 0);
            }
        }
    } else if (warp >= 10) {
        // two groups of four warps in turn; a warp reaches the lanes of its number modulo 4
        const uint32_t group = (warp - 10) >> 2;
        const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16) + 256;
        const uint32_t bars = in_cluster(smem_addr(&full[0]), 0);
        uint32_t st = 0, round = 0, n = 0;
        bool ok = true;
        for (int tile = blockIdx.x / 2; tile < tiles && ok; tile += stride) {
            for (int s = 0; s < steps; ++s, ++n) {
                if ((n & 1) == group) {
                    // The stage's last round went to the other group; its use has to be over before a
                    // parity tells this round's scales from the last but one's.
                    if (!mbar_wait_all(&empty[st], (round & 1) ^ 1) || !wait_of(a, kScaleFull, n, &sf_full[st], round & 1)) {
                        ok = false;
                        break;
                    }
                    const uint32_t sf = base + st * G::kStageBytes + 2 * G::kCodeBytes, to = lanes + st * G::kSfCols;
                    // Q's scales for its first and second 128 rows lie side by side for each step of 64
                    if constexpr (FMT == FP8Q_MXFP4) {
                        store_scales2(to, sf);
                        store_scales4(to + 8, sf + 1024, 1024);
                    } else {
                        store_scales4(to, sf, 512);
                        store_scales4(to + 16, sf + 4 * 512, 4 * 512);
                        store_scales4(to + 32, sf + 6 * 512, 4 * 512);
                    }
                    scales_stored();
                    if (lane == 0) arrive_cluster(bars + st * 8);
                }
                if (++st == kPairStages) st = 0, ++round;
            }
        }
        if (!ok) gave_up = 1;
    } else {
        const float alpha = __fmul_rn(a.sa ? *a.sa : 1.0f, a.sb ? *a.sb : 1.0f);
        const uint32_t from = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (warp >> 2) * 128;
        const uint32_t bar = in_cluster(smem_addr(&drained), 0);
        bool ok = true;
        uint32_t it = 0;
        constexpr int kLine = F32 ? 32 : 64;  // columns of a 128-byte line
        const uint32_t out = base + kPairStages * G::kStageBytes + warp * 4096, line = out + lane * 128;
        for (int tile = blockIdx.x / 2; tile < tiles; tile += stride, ++it) {
            const PairTile t = pair_tile(tile, p_tiles, a.q_tiles);
            const int p_first = t.p + (int)rank * 128 + (warp & 3) * 32;
            const int q = t.q + (warp >> 2) * 128, left = a.q_rows - q;
            ok = ok && mbar_wait_warp(&done, it & 1, 32) && !made_to_fail(a, kOutDone, it);
            if (!ok) gave_up = 1;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < 128; c += kLine) {
                uint32_t o[32];
#pragma unroll
                for (int h = 0; h < kLine; h += 32) {
                    float v[32];
                    tmem_load32(from + c + h, v);
                    // a wait that ran out shows as NaN in the tile
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = ok ? __fmul_rn(v[i], alpha) : __uint_as_float(0x7FFFFFFFu);
                    if constexpr (F32) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(v[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[h / 2 + i] = cvt_bf16x2(v[2 * i], v[2 * i + 1]);
                    }
                }
                if (c + kLine == 128) {  // the accumulators are in registers
                    tc_fence_before();
                    if (lane == 0) arrive_cluster(bar);
                }
                // through shared memory (128-byte swizzle)
                if (a.vec && lane == 0) store_read_wait();
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(line + ((j ^ (lane & 7)) << 4)), "r"(o[4 * j]),
                                 "r"(o[4 * j + 1]), "r"(o[4 * j + 2]), "r"(o[4 * j + 3])
                                 : "memory");
                if (a.vec) {  // out by a tensor-map store
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    __syncwarp();
                    if (lane == 0 && left > c && p_first < a.p_rows) tile_store(&map_d, q + c, p_first, out);
                } else {
                    __syncwarp();
                    store_rows<F32>(a.d, (int64_t)p_first * a.ld + q + c, a.ld, a.p_rows - p_first, left - c, out);
                }
                __syncwarp();
            }
        }
        if (lane == 0) store_wait();
    }
    __syncwarp();
    __syncthreads();
    if (gave_up && threadIdx.x == 0) {  // copies still under way end before their CTAs do
        for (uint32_t n = loads > kPairStages ? loads - kPairStages : 0; n < loads && rank == 0; ++n)
            mbar_wait(&full[n % kPairStages], (n / kPairStages) & 1);
        for (uint32_t n = sf_loads > kPairStages ? sf_loads - kPairStages : 0; n < sf_loads; ++n)
            mbar_wait(&sf_full[n % kPairStages], (n / kPairStages) & 1);
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (warp == 9) tmem_free<2>(tmem, 512);
    cluster_sync_all();
}

// ----------------------------------------------------------------------------
// Host

// Codes [rows, cols]: boxes of 128 bytes x box_rows rows, zeros beyond the edges.
bool codes_map(CUtensorMap* map, const uint8_t* q, int64_t rows, int64_t cols, int box_rows) {
    const cuuint64_t ld = (cuuint64_t)fp4_row_bytes(cols);
    return make_map<2>(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, q, {ld, (cuuint64_t)rows}, {ld}, {kStepBytes, (cuuint32_t)box_rows},
                       CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// Block scales: rows of scale tiles along k, boxes of `tiles` of them x box_rows, zeros beyond the edges.
bool scales_map(CUtensorMap* map, const uint8_t* sf, int64_t rows, int64_t across, int tiles, int box_rows) {
    return make_map<2>(map, CU_TENSOR_MAP_DATA_TYPE_UINT64, sf, {(cuuint64_t)across * 64, (cuuint64_t)((rows + 127) / 128)},
                       {(cuuint64_t)across * 512}, {(cuuint32_t)tiles * 64, (cuuint32_t)box_rows}, CU_TENSOR_MAP_SWIZZLE_NONE,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}

// D: boxes of 32 rows of 128 bytes.
template <bool F32>
bool result_map(CUtensorMap* map, void* d, int64_t rows, int64_t cols) {
    constexpr int kBytes = F32 ? 4 : 2;
    return make_map<2>(map, F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, d, {(cuuint64_t)cols, (cuuint64_t)rows},
                       {(cuuint64_t)cols * kBytes}, {128 / kBytes, 32}, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE);
}

template <int FMT, int BN, bool F32>
fp8q_status launch_tiles(const CUtensorMap& mp, const CUtensorMap& mq, const MmArgs& a, unsigned grid, cudaStream_t s) {
    static std::atomic<uint64_t> devices{0};
    auto kern = fp4_matmul_kernel<FMT, BN, F32>;
    cudaError_t e = allow_smem(kern, MmGeom<FMT, BN>::kSmem, devices);
    if (e != cudaSuccess) return cuda_fail(e, "fp4_matmul_kernel setup");
    return launch_behind(kern, dim3(grid), dim3(192), MmGeom<FMT, BN>::kSmem, (unsigned)a.split, s, "fp4_matmul_kernel", mp, mq, a);
}

template <int FMT, bool F32>
fp8q_status launch_pairs(const uint8_t* p, const uint8_t* q, int64_t k, MmArgs g, cudaStream_t s) {
    static std::atomic<uint64_t> devices{0};
    using G = PairGeom<FMT>;
    auto kern = fp4_matmul_pair_kernel<FMT, F32>;
    const cudaError_t e = allow_smem(kern, G::kSmem, devices);
    if (e != cudaSuccess) return cuda_fail(e, "fp4_matmul_pair_kernel setup");
    CUtensorMap mp, mq, ms, mt, md = {};
    if (!codes_map(&mp, p, g.p_rows, k, 128) || !codes_map(&mq, q, g.q_rows, k, 128) ||
        !scales_map(&ms, g.p_sf, g.p_rows, g.sf_across, G::kSfTiles, 1) || !scales_map(&mt, g.q_sf, g.q_rows, g.sf_across, G::kSfTiles, 2))
        return cuda_fail(cudaErrorInvalidValue, "fp4_matmul_pair_kernel tensor map");
    if (g.vec && !result_map<F32>(&md, g.d, g.p_rows, g.q_rows))
        return cuda_fail(cudaErrorInvalidValue, "fp4_matmul_pair_kernel tensor map");
    g.q_tiles = (g.q_rows + 255) / 256;
    const int64_t tiles = (int64_t)((g.p_rows + 255) / 256) * g.q_tiles;
    if (tiles > 0x3FFFFFFF) return FP8Q_ERR_UNSUPPORTED;
    const int64_t pairs = sm_count() / 2;
    const unsigned grid = 2u * (unsigned)(tiles < pairs ? tiles : pairs);
    return launch_behind(kern, dim3(grid), dim3(kPairThreads), G::kSmem, 1, s, "fp4_matmul_pair_kernel", mp, mq, ms, mt, md, g);
}

#ifdef FP8Q_TEST_HOOKS
int g_fail_role = 0, g_fail_at = 0, g_fail_cta = -1;
#endif

template <int FMT, bool F32>
fp8q_status matmul(const uint8_t* a, const uint8_t* a_sf, const uint8_t* b, const uint8_t* b_sf, void* d, int64_t m, int64_t n, int64_t k,
                   const float* sa, const float* sb, cudaStream_t s) {
    MmArgs g;
#ifdef FP8Q_TEST_HOOKS
    g.fail_role = g_fail_role;
    g.fail_at = g_fail_at;
    g.fail_cta = g_fail_cta;
#endif
    g.sa = sa;
    g.sb = sb;
    g.d = d;
    g.ld = n;
    g.ksteps = (int32_t)((k + 63) / 64);
    g.sf_across = (int32_t)fp4_sf_tiles<FMT>(k);
    g.vec = ((uintptr_t)d & 15u) == 0 && n % (F32 ? 4 : 8) == 0;
    // Pairs of CTAs where 128-row tiles of one CTA each would not all be resident at once.
    const int sms = sm_count();
    // (Odd rows of bf16, which a pair stores slowly at the end, stay with single CTAs where both tiles and steps are few:
    // 1033x2071x1000 7.5 us, 10.2 on pairs; 2560x2561x1000 14.4 and 16.7, but 2560x2561x4096 25.5 and 22.6.)
    const int64_t blocks = (m + 127) / 128 * ((n + 127) / 128);
    const bool pairs = m > 128 && n > 128 && blocks > sms && (F32 || n % 2 == 0 || blocks > 3 * sms || g.ksteps >= 32);
    // Otherwise the CTAs of a cluster share a tile's sums, as many as are resident at once (two an SM up to 32 rows of Q;
    // clusters of 4 and 8 reach 144 and 120 of the 152 SMs) and have two steps or more, where the steps that a CTA
    // saves are worth the cluster and its sums, 1 us for 16 rows of Q to 2.5 for 128, a step 0.3: 1x4096x4096
    // takes 4.7 us on clusters of 4, 6.6 without; 128x4096x4096 7.0 and 8.5, 128x8192x4096 9.0 and 9.6, but 128x4096x2048 6.3 and 5.7.
    // The more of the GPU the tiles take anyway, the longer k has to be.  Above two fifths of the SMs, 16 steps: 128x8192x2048 (8)
    // takes 6.3 us, 6.9 on clusters of 2; 128x8192x4096 9.7 and 9.2.  Above two thirds, 32: 24x16384x2048 6.9 and 7.4,
    // 24x16384x4096 10.3 and 10.2, 24x16384x8192 16.9 and 15.6.
    const int bn = m <= 16 ? 16 : m <= 32 ? 32 : m <= 64 ? 64 : 128, steps = (g.ksteps + 3) / 4;
    int split = 1;
    if (!pairs) {
        const int64_t tiles = (n + 127) / 128 * ((m + bn - 1) / bn), room = (bn <= 32 ? 2 : 1) * sms;
        int most = 1;
        while (most < 8 && tiles * most * 2 <= room * (most == 1 ? 20 : most == 2 ? 19 : 16) / 20 && steps >= most * 4) most *= 2;
        if (steps - steps / most > 3 + bn / 32 && steps >= (tiles * 3 > sms * 2 ? 32 : tiles * 5 > sms * 2 ? 16 : 0)) split = most;
    }
    g.split = split;
    // P, whose rows are the accumulators' 128 lanes, is A, and a thread holds part of a row of D, where
    // pairs write it through shared memory and where D's rows hold whole vectors; otherwise the lanes run along
    // D's rows, so that a warp's stores are contiguous, as they are where few rows of A leave the lanes to B.
    g.p_is_m = pairs || (g.vec && split == 1 && m >= n);
    const uint8_t *p = g.p_is_m ? a : b, *q = g.p_is_m ? b : a;
    g.p_sf = g.p_is_m ? a_sf : b_sf;
    g.q_sf = g.p_is_m ? b_sf : a_sf;
    g.p_rows = (int32_t)(g.p_is_m ? m : n);
    g.q_rows = (int32_t)(g.p_is_m ? n : m);
    if (pairs) return launch_pairs<FMT, F32>(p, q, k, g, s);
    const int qn = g.p_is_m ? (n <= 16 ? 16 : n <= 32 ? 32 : n <= 64 ? 64 : 128) : bn;
    g.q_tiles = (g.q_rows + qn - 1) / qn;
    const int64_t tiles = (int64_t)((g.p_rows + 127) / 128) * g.q_tiles;
    if (tiles * split > 0x7FFFFFFF) return FP8Q_ERR_UNSUPPORTED;
    CUtensorMap mp, mq;
    if (!codes_map(&mp, p, g.p_rows, k, 128) || !codes_map(&mq, q, g.q_rows, k, qn))
        return cuda_fail(cudaErrorInvalidValue, "fp4_matmul_kernel tensor map");
    const unsigned grid = (unsigned)(tiles * split);
    switch (qn) {
        case 16: return launch_tiles<FMT, 16, F32>(mp, mq, g, grid, s);
        case 32: return launch_tiles<FMT, 32, F32>(mp, mq, g, grid, s);
        case 64: return launch_tiles<FMT, 64, F32>(mp, mq, g, grid, s);
        default: return launch_tiles<FMT, 128, F32>(mp, mq, g, grid, s);
    }
}

}  // namespace

extern "C" {

#ifdef FP8Q_TEST_HOOKS  // the wait of that role (MmWait) at that step or tile reports failure, in one CTA or (cta < 0) in all
void fp8q_test_set_matmul_give_up(int role, int at, int cta) {
    g_fail_role = role;
    g_fail_at = at;
    g_fail_cta = cta;
}
#endif

fp8q_status fp8q_fp4_matmul(const uint8_t* a, const uint8_t* a_sf, const uint8_t* b, const uint8_t* b_sf, void* d,
                            int64_t m, int64_t n, int64_t k, fp8q_format fmt, fp8q_out_type out, const float* a_scale,
                            const float* b_scale, void* stream) {
    if (!valid_fp4(fmt) || m < 0 || n < 0 || k < 0) return FP8Q_ERR_INVALID_ARG;
    if (out != FP8Q_OUT_BF16 && out != FP8Q_OUT_F32) return FP8Q_ERR_INVALID_ARG;
    if (m == 0 || n == 0) return FP8Q_OK;
    if (m > kFp4MaxDim || n > kFp4MaxDim || k > kFp4MaxDim) return FP8Q_ERR_UNSUPPORTED;
    if (!d || (k > 0 && (!a || !a_sf || !b || !b_sf))) return FP8Q_ERR_INVALID_ARG;
    if (fmt == FP8Q_MXFP4 && (a_scale || b_scale)) return FP8Q_ERR_INVALID_ARG;
    if (((uintptr_t)d & (out == FP8Q_OUT_F32 ? 3u : 1u)) || ((uintptr_t)a_scale & 3u) || ((uintptr_t)b_scale & 3u))
        return FP8Q_ERR_INVALID_ARG;
    if (((uintptr_t)a | (uintptr_t)a_sf | (uintptr_t)b | (uintptr_t)b_sf) & 15u) return FP8Q_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (k == 0) {  // an empty sum
        const cudaError_t e = cudaMemsetAsync(d, 0, (size_t)(m * n) * (out == FP8Q_OUT_F32 ? 4 : 2), s);
        return e == cudaSuccess ? FP8Q_OK : cuda_fail(e, "fp8q_fp4_matmul");
    }
    if (fmt == FP8Q_MXFP4)
        return out == FP8Q_OUT_F32 ? matmul<FP8Q_MXFP4, true>(a, a_sf, b, b_sf, d, m, n, k, a_scale, b_scale, s)
                                   : matmul<FP8Q_MXFP4, false>(a, a_sf, b, b_sf, d, m, n, k, a_scale, b_scale, s);
    return out == FP8Q_OUT_F32 ? matmul<FP8Q_NVFP4, true>(a, a_sf, b, b_sf, d, m, n, k, a_scale, b_scale, s)
                               : matmul<FP8Q_NVFP4, false>(a, a_sf, b, b_sf, d, m, n, k, a_scale, b_scale, s);
}

}  // extern "C"
