// Programmatic launch in a stream: a kernel launched through launch_pdl() may start while its
// predecessor in the stream still runs, and waits in pdl_wait() until all of the predecessor's
// writes are visible. Every kernel launched this way calls pdl_wait() in all its threads before it
// touches global memory, so a kernel that ends has everything before it in the stream done. Saves
// about 2 us between two short kernels.
// Such a kernel has no non-coherent loads (__ldg, or a __restrict__ pointer that lets the compiler make them): they are taken
// to be of memory that nothing writes while the kernel runs, so they may be moved above the wait.
#pragma once

#include <cuda_runtime.h>

namespace bl {

__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
// Let the successor's blocks be scheduled once all blocks of this kernel have come this far.
__device__ __forceinline__ void pdl_release() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

// `cluster`: blocks per cluster (of consecutive blocks).
template <typename... P, typename... A>
cudaError_t launch_pdl_cluster(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, unsigned cluster, cudaStream_t s,
                               A &&...args) {
    cudaLaunchConfig_t c{};
    c.gridDim = dim3(grid);
    c.blockDim = dim3(threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    cudaLaunchAttribute at[2]{};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
}
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t s, A &&...args) {
    return launch_pdl_cluster(kernel, grid, threads, smem, 1, s, static_cast<A &&>(args)...);
}

}  // namespace bl
