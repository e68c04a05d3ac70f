// Programmatic dependent launch: a kernel launched with launch_after may be set
// up while the kernel before it in the stream still runs. It calls
// wait_previous() in every thread before it touches global memory (which waits
// until that kernel, and so all before it, has finished), and allow_next() once
// its own CTAs have started. What the kernel before may have written is not read
// with __ldg: its non-coherent loads are for data that no one writes while the
// kernel runs, and this one does run, though it waits, while the one before writes.
#pragma once

#include <cuda_runtime.h>

namespace pa {

__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// kern<<<grid, block, smem, stream>>>(args...) with that attribute, as a cluster of `cluster` CTAs if that is above 1.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kern)(P...), dim3 grid, unsigned block, size_t smem, unsigned cluster,
                         cudaStream_t stream, A &&...args) {
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<A &&>(args)...);
}

}  // namespace pa
