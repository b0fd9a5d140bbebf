// tq_launch.cuh -- kernels of one call that follow one another without a gap.
//
// A kernel launched by launch_after may start while the one before it in the stream still runs (its
// CTAs come in as those of the other have all started and leave room).  It waits with grid_wait
// before it touches anything that a kernel of the call writes, or writes anything that one reads;
// every kernel that such a launch follows says grid_go when that may happen.  The wait is for the
// kernel before, and for the others through it, since each of them has waited as well; that a kernel
// has been let start says nothing of what it may read.  Before its wait a kernel reads only what was
// there before the call (the parameter set, records): a call's first launch is an ordinary one,
// behind all earlier work.
#pragma once

#include <cuda_runtime.h>

namespace tq {

__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_go() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), unsigned grid, unsigned block, size_t smem, cudaStream_t s, A... args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace tq
