// tensor_memory_neighbours.cu -- kernels beside which the 4-bit product runs in a stream, for the order in which
// neighbours take tensor memory.  Both take all of an SM's 512 columns and give them back at once.
//   ahead   lets the next kernel start first, and takes tensor memory some time later
//   behind  may start while the kernel before it still runs, takes tensor memory at once and holds it while it waits
//           for that kernel
#include <cstdint>

#include <cuda_runtime.h>

__device__ __forceinline__ uint32_t take(uint32_t* slot) {
    const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(slot));
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(at) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    __syncwarp();
    return *static_cast<volatile uint32_t*>(slot);
}
__device__ __forceinline__ void give_back(uint32_t at) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(at));
}
__device__ __forceinline__ uint64_t now() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__global__ void __launch_bounds__(32) ahead(unsigned long long* count) {
    __shared__ uint32_t slot;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (const uint64_t t = now(); now() - t < 50000;) __nanosleep(1000);  // 50 us
    give_back(take(&slot));
    if (threadIdx.x == 0) atomicAdd(count, 1ull);
}

__global__ void __launch_bounds__(32) behind(unsigned long long* count) {
    __shared__ uint32_t slot;
    const uint32_t at = take(&slot);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    give_back(at);
    if (threadIdx.x == 0) atomicAdd(count, 1ull);
}

extern "C" int launch_neighbour(int is_behind, int ctas, unsigned long long* count, void* stream) {
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(32);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = &at;
    cfg.numAttrs = is_behind ? 1 : 0;
    return (int)cudaLaunchKernelEx(&cfg, is_behind ? behind : ahead, count);
}
