// tcgen05.cuh -- the fifth-generation tensor core's instructions that the 4-bit
// and the 8-bit products use: tensor memory, the multiply-adds, and the copies
// that feed them.  Documented PTX only.

#pragma once

#include "fp4.cuh"
#include "mbarrier.cuh"

#include <cuda.h>

#include <atomic>

namespace {

// mbar_wait() for a whole warp: one lane looks at the barrier (32 lanes looking,
// in many warps, take the barriers' time from the threads that everything waits
// for), with pauses of `pause` ns where the wait is long anyway.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity, uint32_t pause) {
    uint32_t ok = 0;
    if ((threadIdx.x & 31) == 0) {
        WaitClock clock;
        while (!(ok = mbar_try(bar, parity))) {
            if (!clock.more()) break;
            if (pause) __nanosleep(pause);
        }
    }
    return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
}

// For a wait that lasts as long as a loop over `stages` barriers does, once mbar_wait_warp() has given up: goes on while one of them
// completes a phase within the limit.  Out of line: no short loop comes here.
__device__ __noinline__ bool mbar_wait_on(uint64_t* bar, uint32_t parity, uint64_t* loop, uint32_t stages) {
    uint32_t ok = 0;
    if ((threadIdx.x & 31) == 0) {
        WaitClock clock;
        uint32_t seen = 0;
        while (!(ok = mbar_try(bar, parity))) {
            uint32_t now = 0;
            for (uint32_t i = 0; i < stages; ++i) now |= (uint32_t)mbar_test(&loop[i], 0) << i;
            if (now != seen) clock = WaitClock();
            seen = now;
            if (!clock.more()) break;
        }
    }
    return __shfl_sync(0xFFFFFFFFu, ok, 0) != 0;
}

// mbar_wait() where each lane looks, with one verdict for the warp: every lane's
// clock runs out for itself, and a warp of which some lanes went on and some
// left would never come together again at the warp-wide instructions behind
// the wait (elect, the .aligned ones of tensor memory).
__device__ __forceinline__ bool mbar_wait_all(uint64_t* bar, uint32_t parity, bool fail_lane = false) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity) && !fail_lane);
}

// The same for a barrier at which the cluster's other CTA arrives for what it has in its own shared memory (arrive_cluster_release()).
__device__ __forceinline__ bool mbar_wait_all_cluster(uint64_t* bar, uint32_t parity, bool fail_lane = false) {
    WaitClock clock;
    uint32_t done;
    for (;;) {
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(smem_addr(bar)), "r"(parity)
            : "memory");
        if (done || !clock.more()) break;
    }
    return __all_sync(0xFFFFFFFFu, done && !fail_lane);
}

// One lane of a converged warp.  The warps that issue copies and multiply-adds
// run their loops whole and let one lane issue: addresses and descriptors then
// stay in uniform registers, and a step costs its issuer tens of cycles, not
// hundreds.
__device__ __forceinline__ bool elect_lane() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// ----------------------------------------------------------------------------
// Tensor memory

// A whole warp.  The only allocation of its CTA: others on the SM may go on at once.
// Behind wait_behind() and before let_next_start(): a kernel that held tensor memory
// while it waits for the kernel ahead could keep that one's CTAs from theirs, and
// both would wait for ever; and so could the next kernel, if it took tensor memory
// at its start, before this one's CTAs all had theirs.
template <int PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t* slot, uint32_t cols) {
    if (PAIR == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
}

template <int PAIR>
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t cols) {  // a whole warp
    if (PAIR == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols));
    else
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols));
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Sixteen consecutive columns of the calling warp's 32 lanes, one lane a thread.
// The values are there after tmem_wait().
__device__ __forceinline__ void tmem_load16(uint32_t at, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Thirty-two columns.
__device__ __forceinline__ void tmem_load32(uint32_t at, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
        "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Sixteen columns back; they are there after tmem_stored().
__device__ __forceinline__ void tmem_store16(uint32_t at, const float* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]),
        "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15])
        : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ----------------------------------------------------------------------------
// Shared-memory descriptors

// Rows of 128 bytes along k, 128-byte swizzle, atoms of 8 rows (1024 bytes) one
// after another.  A step of 64 codes along k adds 32 bytes to the start.
__device__ __forceinline__ uint64_t desc_codes(uint32_t at) {
    return (uint64_t)((at & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// ----------------------------------------------------------------------------
// Instructions

// Four scale tiles (512 bytes each) to sixteen columns of the calling warp's 32
// lanes: line l of a tile, 16 bytes, is lane l's four columns.  The tiles lie one
// behind another (gap 512), or the second and fourth `gap` behind the first and
// third, which lie one behind the other.  Each of the four warps that reach the four groups of
// lanes stores the same.  Copying them by the tensor core's own shared-to-tensor
// memory copies holds up the multiply-adds behind them (1162 cycles for four
// multiply-adds of 256x256x64 and their twelve tiles, 512 without); stored by
// eight warps beside them, twelve tiles take 445.
__device__ __forceinline__ void store_scales4(uint32_t to, uint32_t from, uint32_t gap) {
    uint32_t v[16];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[4 * i]), "=r"(v[4 * i + 1]), "=r"(v[4 * i + 2]), "=r"(v[4 * i + 3])
                     : "r"(from + (gap == 512 ? i * 512 : (i >> 1) * 512 + (i & 1) * gap) + (threadIdx.x & 31) * 16)
                     : "memory");
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(to),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]),
        "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

__device__ __forceinline__ void store_scales2(uint32_t to, uint32_t from) {
    uint32_t v[8];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[4 * i]), "=r"(v[4 * i + 1]), "=r"(v[4 * i + 2]), "=r"(v[4 * i + 3])
                     : "r"(from + i * 512 + (threadIdx.x & 31) * 16)
                     : "memory");
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(to), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                 "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

__device__ __forceinline__ void scales_stored() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
    tc_fence_before();
}

// Instruction descriptor: e2m1 operands along k, N columns, M rows, the scale
// format, and which pair of the four scale bytes is used (32-blocks only).
template <int FMT>
__host__ __device__ constexpr uint32_t mma_desc(uint32_t m, uint32_t n, uint32_t pair) {
    return (pair << 4) | (1u << 7) | (1u << 10) | ((n >> 3) << 17) | ((FMT == FP8Q_MXFP4 ? 1u : 0u) << 23) | ((m >> 4) << 24) |
           (pair << 29);
}

// d (+)= A B^T over 64 codes with their block scales.
template <int FMT, int PAIR>
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb, uint32_t add) {
#define FP8Q_MMA(group, kind)                                                                                       \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                                  \
                 "tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),  \
                 "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(add)                                           \
                 : "memory")
    if (FMT == FP8Q_MXFP4) {
        if (PAIR == 2)
            FP8Q_MMA("2", "mxf4.block_scale.scale_vec::2X");
        else
            FP8Q_MMA("1", "mxf4.block_scale.scale_vec::2X");
    } else {
        if (PAIR == 2)
            FP8Q_MMA("2", "mxf4nvf4.block_scale.scale_vec::4X");
        else
            FP8Q_MMA("1", "mxf4nvf4.block_scale.scale_vec::4X");
    }
#undef FP8Q_MMA
}

// Instruction descriptor of the FP8 product: formats (0 e4m3, 1 e5m2), whether
// an operand's rows lie along m or n (transposed) and not along k, N columns, M rows.
__host__ __device__ constexpr uint32_t mma_desc_fp8(uint32_t m, uint32_t n, uint32_t fa, uint32_t fb, uint32_t ta, uint32_t tb) {
    return (1u << 4) | (fa << 7) | (fb << 10) | (ta << 15) | (tb << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

// The same with another number of columns.
__device__ __forceinline__ uint32_t mma_desc_cols(uint32_t idesc, uint32_t n) { return (idesc & ~(63u << 17)) | (n >> 3) << 17; }

// d (+)= A B^T over 32 FP8 codes.  Sums are binary32, but what lies below the last place of the largest addend is cut off, not
// rounded: 8e-8 to 2.4e-7 of the results' root mean square over a k of 4096, three times what additions that round leave.
template <int PAIR>
__device__ __forceinline__ void tc_mma_fp8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add) {
#define FP8Q_MMA(group)                                                                                   \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"                                        \
                 "tcgen05.mma.cta_group::" group ".kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),      \
                 "l"(a), "l"(b), "r"(idesc), "r"(add)                                                     \
                 : "memory")
    if (PAIR == 2)
        FP8Q_MMA("2");
    else
        FP8Q_MMA("1");
#undef FP8Q_MMA
}

// *bar completes a phase when everything this thread has given to the tensor core is done.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}

// The same for the pair: the barrier at this place in each CTA of `mask`.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar, uint32_t mask) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(smem_addr(bar)),
                 "h"((uint16_t)mask)
                 : "memory");
}

// ----------------------------------------------------------------------------
// Clusters

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync_all() {
    __syncwarp();  // the barrier is a warp's instruction: its lanes may come from loops of unlike lengths
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// The address in the cluster of what lies at `at` in the CTA of that rank.
__device__ __forceinline__ uint32_t in_cluster(uint32_t at, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
    return r;
}

// What it announces lies in tensor memory (stored or read before tcgen05's own
// wait and fence), so it need not order other memory over the cluster: with
// .release.cluster it reached the barrier 1600 cycles late.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}

// arrive_cluster() for what this CTA has in shared memory, copied there or stored: it happens before what follows
// mbar_wait_all_cluster() in the other CTA.
__device__ __forceinline__ void arrive_cluster_release(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A barrier of THREADS of the CTA's threads, whole warps.
template <int THREADS>
__device__ __forceinline__ void some_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

__device__ __forceinline__ void arrive_local(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void mbar_init_count(uint64_t* bar, uint32_t n) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(n) : "memory");
}

// ----------------------------------------------------------------------------
// Copies

__device__ __forceinline__ void expect_bytes(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}

__device__ __forceinline__ void tile_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}

// The same in a pair: the barrier, a cluster address, may lie in either of its CTAs.
__device__ __forceinline__ void tile_load_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Of three dimensions.
__device__ __forceinline__ void tile_load3(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}
__device__ __forceinline__ void tile_load3_pair(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void block_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}

// Bytes (a multiple of 16, from a 16-byte address) on their way to L2.
__device__ __forceinline__ void block_prefetch(const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

// A box from shared memory, clipped at the tensor's edges; one thread's stores
// are done reading shared memory after store_read_wait(), done altogether after
// store_wait().
__device__ __forceinline__ void tile_store(const CUtensorMap* map, int x, int y, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map), "r"(x), "r"(y), "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// A tensor map on its way before its first copy.
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
__device__ __forceinline__ void store_read_wait() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// ----------------------------------------------------------------------------
// Tiles of 256 x 256, and tensor maps

// Tiles go in bands of eight along P, along Q within a band, so that the tiles
// under way at one time share rows of both operands in L2.
struct PairTile {
    int p, q;
};
__device__ __forceinline__ PairTile pair_tile(int tile, int p_tiles, int q_tiles) {
    const int band = tile / (8 * q_tiles), in = tile - band * 8 * q_tiles;
    const int high = min(8, p_tiles - band * 8);
    return {(band * 8 + in % high) * 256, in / high * 256};
}

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

// A tensor map of DIMS dimensions: sizes and strides (in bytes, of all but the first) and the box.  A thread that has made no
// call of the runtime yet has no context, without which no map is made: the current device's is taken up then.
template <int DIMS>
bool make_map(CUtensorMap* map, CUtensorMapDataType type, const void* p, const cuuint64_t (&dim)[DIMS], const cuuint64_t (&stride)[DIMS - 1],
              const cuuint32_t (&box)[DIMS], CUtensorMapSwizzle swizzle, CUtensorMapL2promotion promotion) {
    const EncodeTiled f = encode_tiled();
    if (!f) return false;
    cuuint32_t one[DIMS];
    for (int i = 0; i < DIMS; ++i) one[i] = 1;
    const auto make = [&] {
        return f(map, type, DIMS, const_cast<void*>(p), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promotion,
                 CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    CUresult r = make();
    if (r == CUDA_ERROR_INVALID_CONTEXT || r == CUDA_ERROR_NOT_INITIALIZED || r == CUDA_ERROR_CONTEXT_IS_DESTROYED) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess) {
            (void)cudaGetLastError();
            return false;
        }
        r = make();
    }
    return r == CUDA_SUCCESS;
}

}  // namespace
