// pdl.cuh -- launches with programmatic stream serialisation.
//
// A kernel launched so may have its blocks scheduled while the kernel before it
// in the stream drains; every thread of it starts with grid_wait(), which returns
// once that kernel is complete and its writes are visible, so nothing is read or
// written early.  grid_launch_next() lets the next kernel launched so be scheduled
// once all blocks have called it.  (A kernel launched without the attribute waits
// for the one before it as a whole, and grid_wait() in it returns at once.)
#pragma once

#include <cuda_runtime.h>

#include <utility>

namespace attn {

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// clusters: CTAs of a cluster (1: none).
template <typename... Params, typename... Args>
cudaError_t launch_serial_clusters(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, int clusters,
                                   cudaStream_t stream, Args&&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = clusters;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = clusters > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

template <typename... Params, typename... Args>
cudaError_t launch_serial(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                          Args&&... args) {
    return launch_serial_clusters(kernel, grid, threads, smem, 1, stream, std::forward<Args>(args)...);
}

}  // namespace attn
