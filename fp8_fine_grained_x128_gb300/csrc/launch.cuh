// launch.cuh -- programmatic dependent launch.
//
// A kernel launched with launch_dependent lets the next kernel of the stream be
// set up while it runs, and waits, before it touches memory, for the one before
// it to be complete (about 1 us less between two short calls).  Every thread of
// such a kernel calls dependency_wait(), so that its completion implies that of
// everything before it.  A long kernel calls dependents_launch() late or not at
// all (its end does the same): CTAs of the next kernel that sit and wait take
// registers and threads from its own (the norm's backward at 8192 x 4096: 53 us a
// call with the early launch, 42 without).
#pragma once

#include <cuda_runtime.h>

#include "../../include/fp8fg.h"

namespace fp8fg {

__device__ __forceinline__ void dependents_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// cluster: CTAs of a cluster (0: as the kernel is compiled).
template <typename... P, typename... A>
inline int launch_dependent_cluster(void (*kernel)(P...), dim3 grid, unsigned cluster, unsigned block, size_t smem, cudaStream_t st, A... args)
{
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

template <typename... P, typename... A>
inline int launch_dependent(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t st, A... args)
{
    return launch_dependent_cluster(kernel, grid, 0, block, smem, st, args...);
}

}  // namespace fp8fg
