// fp4_matmul.cu -- the product of two microscaled 4-bit operands on the tensor
// cores.
//
//   D[m][n] = RN_out( (sum_k A[m][k] B[n][k]) * RN(sa * sb) )
//
// Both operands are packed along k (fp4.cuh).  Codes come into shared memory by
// tensor-map copies (256 codes of k a step, 128 bytes a row, 128-byte swizzle,
// zeros beyond the edges), block scales by plain bulk copies of whole scale
// tiles, which already lie as tensor memory takes them; one thread issues the
// copies, another the scale copies to tensor memory and the block-scaled
// multiply-adds, and four warps carry the accumulators out.

#include "tcgen05.cuh"

#include <atomic>

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
};

template <int FMT, int BN>
struct MmGeom {
    static constexpr int kSfTiles = FMT == FP8Q_MXFP4 ? 2 : 4;  // scale tiles a step and 128 rows
    static constexpr int kQSf = (BN + 127) / 128;
    static constexpr int kPBytes = 128 * kStepBytes, kQBytes = BN * kStepBytes;
    static constexpr int kStageBytes = kPBytes + kQBytes + (1 + kQSf) * kSfTiles * 512;
    static constexpr int kSmem = kStages * kStageBytes + 1024;  // and room to start on 1024 bytes
    static constexpr int kAccCols = BN < 32 ? 32 : BN;
    static constexpr int kSfCols = kSfTiles * 4 * (1 + kQSf);   // tensor memory columns a stage
    static constexpr int kNeed = kAccCols + kStages * kSfCols;
    static constexpr int kCols = kNeed <= 128 ? 128 : kNeed <= 256 ? 256 : 512;
};

__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t at, uint32_t rank) {
    uint32_t r;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(r) : "memory");
    return v;
}

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

template <int FMT, int BN, bool F32>
__global__ void __launch_bounds__(192) fp4_matmul_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                                                         const MmArgs a) {
    using G = MmGeom<FMT, BN>;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t full[kStages], empty[kStages], done;
    __shared__ uint32_t tmem_slot, loads;
    __shared__ int gave_up;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = (smem_addr(raw) + 1023u) & ~1023u;
    const int rank = a.split > 1 ? (int)(blockIdx.x % a.split) : 0;
    const int tile = blockIdx.x / a.split;
    const int p0 = tile / a.q_tiles * 128, q0 = tile % a.q_tiles * BN;
    // this CTA's steps of 256 codes
    const int steps = (a.ksteps + 3) / 4;
    const int s0 = (int)((int64_t)steps * rank / a.split), s1 = (int)((int64_t)steps * (rank + 1) / a.split);

    if (warp == 5) tmem_alloc<1>(&tmem_slot, G::kCols);
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&full[i]);
            mbar_init(&empty[i]);
        }
        mbar_init(&done);
        loads = 0;
        gave_up = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    if (warp == 4 && lane == 0) {
        const int q_sf_tiles = min(G::kQSf, (a.q_rows - q0 + 127) / 128);  // scale tiles of Q's rows that exist
        const uint8_t* psf = a.p_sf + (int64_t)(p0 / 128) * a.sf_across * 512;
        const uint8_t* qsf = a.q_sf + (int64_t)(q0 / 128) * a.sf_across * 512;
        uint32_t n = 0;
        for (int s = s0; s < s1; ++s, ++n) {
            const uint32_t st = n % kStages, at = base + st * G::kStageBytes;
            if (!mbar_wait(&empty[st], ((n / kStages) & 1) ^ 1)) {
                gave_up = 1;
                break;
            }
            const int t0 = s * G::kSfTiles, nt = min(G::kSfTiles, a.sf_across - t0);
            expect_bytes(&full[st], G::kPBytes + G::kQBytes + nt * 512 * (1 + q_sf_tiles));
            tile_load(at, &map_p, s * kStepBytes, p0, &full[st]);
            tile_load(at + G::kPBytes, &map_q, s * kStepBytes, q0, &full[st]);
            const uint32_t sf = at + G::kPBytes + G::kQBytes;
            block_load(sf, psf + (int64_t)t0 * 512, nt * 512, &full[st]);
            for (int j = 0; j < q_sf_tiles; ++j)
                block_load(sf + (1 + j) * G::kSfTiles * 512, qsf + ((int64_t)j * a.sf_across + t0) * 512, nt * 512, &full[st]);
        }
        loads = n;
    } else if (warp == 5 && lane == 0) {
        uint32_t n = 0;
        for (int s = s0; s < s1; ++s, ++n) {
            const uint32_t st = n % kStages, at = base + st * G::kStageBytes;
            if (!mbar_wait(&full[st], (n / kStages) & 1)) {
                gave_up = 1;
                break;
            }
            tc_fence_after();
            const int nk = min(4, a.ksteps - s * 4), nt = min(G::kSfTiles, a.sf_across - s * G::kSfTiles);
            const uint32_t sf = at + G::kPBytes + G::kQBytes;
            const uint32_t tp = tmem + G::kAccCols + st * G::kSfCols, tq = tp + G::kSfTiles * 4;
            for (int t = 0; t < nt; ++t) {
                tc_copy_scales<1>(tp + t * 4, desc_scales(sf + t * 512));
#pragma unroll
                for (int j = 0; j < G::kQSf; ++j)
                    tc_copy_scales<1>(tq + t * 4 * G::kQSf + j * 4, desc_scales(sf + ((1 + j) * G::kSfTiles + t) * 512));
            }
            for (int k = 0; k < nk; ++k) {
                const int t = FMT == FP8Q_MXFP4 ? k >> 1 : k;
                const uint32_t idesc = FMT == FP8Q_MXFP4 && (k & 1) ? mma_desc<FMT>(128, BN, 2) : mma_desc<FMT>(128, BN, 0);
                tc_mma<FMT, 1>(tmem, desc_codes(at + k * 32), desc_codes(at + G::kPBytes + k * 32), idesc, tp + t * 4,
                               tq + t * 4 * G::kQSf, n | k);
            }
            tc_commit(&empty[st]);
        }
        tc_commit(&done);
    }
    __syncwarp();
    if (warp < 4 && !mbar_wait(&done, 0)) gave_up = 1;
    __syncthreads();
    tc_fence_after();
    const float alpha = __fmul_rn(a.sa ? __ldg(a.sa) : 1.0f, a.sb ? __ldg(a.sb) : 1.0f);
    // A wait that ran out (correct operation never gets there) shows as NaN in the whole tile.
    const float nan = __uint_as_float(0x7FFFFFFFu);
    const int p = p0 + warp * 32 + lane;
    if (a.split == 1) {
        if (warp < 4) {
            const uint32_t row = tmem + ((uint32_t)(warp * 32) << 16);
#pragma unroll 1
            for (int c = 0; c < BN; c += 16) {
                float v[16];
                tmem_load16(row + c, v);
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = gave_up ? nan : __fmul_rn(v[i], alpha);
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
        // the partial sums in shared memory, a column's 128 rows side by side; each CTA adds
        // its share of the columns over the cluster in rank order
        float* part = reinterpret_cast<float*>(raw + (base - smem_addr(raw)));
        if (warp < 4) {
            const uint32_t row = tmem + ((uint32_t)(warp * 32) << 16);
#pragma unroll 1
            for (int c = 0; c < BN; c += 16) {
                float v[16];
                tmem_load16(row + c, v);
#pragma unroll
                for (int i = 0; i < 16; ++i) part[(c + i) * 128 + warp * 32 + lane] = gave_up ? nan : v[i];
            }
        }
        cluster_sync_all();
        if (warp < 4) {
            for (int c = rank; c < BN && q0 + c < a.q_rows; c += a.split) {
                const uint32_t at = base + (c * 128 + warp * 32 + lane) * 4;
                float v = 0.0f;
                for (int r = 0; r < a.split; ++r) v += ld_cluster_f32(at, r);
                v = __fmul_rn(v, alpha);
                if (p < a.p_rows) {
                    if (a.p_is_m)
                        store_one<F32>(a.d, (int64_t)p * a.ld + q0 + c, v);
                    else
                        store_one<F32>(a.d, (int64_t)(q0 + c) * a.ld + p, v);
                }
            }
        }
        cluster_sync_all();  // no CTA's sums go away while another reads them
    }
    if (gave_up && threadIdx.x == 0)  // copies still under way end before the CTA does
        for (uint32_t n = loads > kStages ? loads - kStages : 0; n < loads; ++n) mbar_wait(&full[n % kStages], (n / kStages) & 1);
    tc_fence_before();
    __syncthreads();
    if (warp == 5) tmem_free<1>(tmem, G::kCols);
}

// ----------------------------------------------------------------------------
// Host

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static std::atomic<EncodeTiled> known{nullptr};
    EncodeTiled f = known.load(std::memory_order_acquire);
    if (!f) {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            (void)cudaGetLastError();
            return nullptr;
        }
        f = reinterpret_cast<EncodeTiled>(p);
        known.store(f, std::memory_order_release);
    }
    return f;
}

// Codes [rows, cols]: boxes of 128 bytes x box_rows rows, zeros beyond the edges.
bool codes_map(CUtensorMap* map, const uint8_t* q, int64_t rows, int64_t cols, int box_rows) {
    const EncodeTiled f = encode_tiled();
    if (!f) return false;
    const int64_t ld = fp4_row_bytes(cols);
    const cuuint64_t dim[2] = {(cuuint64_t)ld, (cuuint64_t)rows}, stride[1] = {(cuuint64_t)ld};
    const cuuint32_t box[2] = {kStepBytes, (cuuint32_t)box_rows}, one[2] = {1, 1};
    return f(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(q), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

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

template <int FMT, int BN, bool F32>
fp8q_status launch_tiles(const CUtensorMap& mp, const CUtensorMap& mq, const MmArgs& a, unsigned grid, cudaStream_t s) {
    static std::atomic<uint64_t> devices{0};
    auto kern = fp4_matmul_kernel<FMT, BN, F32>;
    cudaError_t e = allow_smem(kern, MmGeom<FMT, BN>::kSmem, devices);
    if (e != cudaSuccess) return cuda_fail(e, "fp4_matmul_kernel setup");
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)a.split;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(192);
    cfg.dynamicSmemBytes = MmGeom<FMT, BN>::kSmem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kern, mp, mq, a);
    return e == cudaSuccess ? FP8Q_OK : cuda_fail(e, "fp4_matmul_kernel");
}

template <int FMT, bool F32>
fp8q_status matmul(const uint8_t* a, const uint8_t* a_sf, const uint8_t* b, const uint8_t* b_sf, void* d, int64_t m, int64_t n, int64_t k,
                   const float* sa, const float* sb, cudaStream_t s) {
    MmArgs g;
    g.sa = sa;
    g.sb = sb;
    g.d = d;
    g.ld = n;
    g.ksteps = (int32_t)((k + 63) / 64);
    g.sf_across = (int32_t)fp4_sf_tiles<FMT>(k);
    g.vec = ((uintptr_t)d & 15u) == 0 && n % (F32 ? 4 : 8) == 0;
    // P, the 128 lanes, is the operand with more rows; with D's rows too short for whole
    // vectors the lanes run along D's rows, so that a warp's stores are contiguous
    g.p_is_m = m >= n && g.vec;
    const uint8_t *p = g.p_is_m ? a : b, *q = g.p_is_m ? b : a;
    g.p_sf = g.p_is_m ? a_sf : b_sf;
    g.q_sf = g.p_is_m ? b_sf : a_sf;
    g.p_rows = (int32_t)(g.p_is_m ? m : n);
    g.q_rows = (int32_t)(g.p_is_m ? n : m);
    const int bn = g.q_rows <= 16 ? 16 : g.q_rows <= 32 ? 32 : g.q_rows <= 64 ? 64 : g.q_rows <= 128 ? 128 : 256;
    g.q_tiles = (g.q_rows + bn - 1) / bn;
    const int64_t tiles = (int64_t)((g.p_rows + 127) / 128) * g.q_tiles;
    const int steps = (g.ksteps + 3) / 4;
    int split = 1;
    while (split < 8 && tiles * split * 2 <= 2 * 152 && steps >= split * 4) split *= 2;
    g.split = split;
    if (tiles * split > 0x7FFFFFFF) return FP8Q_ERR_UNSUPPORTED;
    CUtensorMap mp, mq;
    if (!codes_map(&mp, p, g.p_rows, k, 128) || !codes_map(&mq, q, g.q_rows, k, bn))
        return cuda_fail(cudaErrorInvalidValue, "fp4_matmul_kernel tensor map");
    const unsigned grid = (unsigned)(tiles * split);
    switch (bn) {
        case 16: return launch_tiles<FMT, 16, F32>(mp, mq, g, grid, s);
        case 32: return launch_tiles<FMT, 32, F32>(mp, mq, g, grid, s);
        case 64: return launch_tiles<FMT, 64, F32>(mp, mq, g, grid, s);
        case 128: return launch_tiles<FMT, 128, F32>(mp, mq, g, grid, s);
        default: return launch_tiles<FMT, 256, F32>(mp, mq, g, grid, s);
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
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (fmt == FP8Q_MXFP4)
        return out == FP8Q_OUT_F32 ? matmul<FP8Q_MXFP4, true>(a, a_sf, b, b_sf, d, m, n, k, a_scale, b_scale, s)
                                   : matmul<FP8Q_MXFP4, false>(a, a_sf, b, b_sf, d, m, n, k, a_scale, b_scale, s);
    return out == FP8Q_OUT_F32 ? matmul<FP8Q_NVFP4, true>(a, a_sf, b, b_sf, d, m, n, k, a_scale, b_scale, s)
                               : matmul<FP8Q_NVFP4, false>(a, a_sf, b, b_sf, d, m, n, k, a_scale, b_scale, s);
}

}  // extern "C"
