// launch.cuh -- programmatic dependent launch.
//
// A kernel launched with launch_dependent lets the next kernel of the stream be
// set up while it runs, and waits, before it touches memory, for the one before
// it to be complete (about 1 us less between two short calls).  Every thread of
// such a kernel calls dependency_wait(), so that its completion implies that of
// everything before it.
#pragma once

#include <cuda_runtime.h>

#include "../../include/fp8fg.h"

namespace fp8fg {

__device__ __forceinline__ void dependents_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
inline int launch_dependent(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t st, A... args)
{
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
}

}  // namespace fp8fg
