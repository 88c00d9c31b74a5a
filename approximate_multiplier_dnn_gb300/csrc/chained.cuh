// Launches that overlap the end of the kernel before them on the stream: the
// next kernel's blocks start, set up their barriers and tensor memory, and wait
// for the kernels before to be complete only when they first touch global
// memory.  Every kernel launched this way calls chain_wait() before that; one
// that has others chained to it calls chain_start() early.  For calls of a few
// kernels of a few microseconds each, most of a launch's latency is hidden.
#pragma once

#include <cuda_runtime.h>

namespace amsim {

__device__ __forceinline__ void chain_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// `chained` false: an ordinary launch (the first of a call: what runs before
// it on the stream is not the library's).
template <typename... P, typename... A>
cudaError_t chain_launch(bool chained, void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                         const A &...args)
{
    cudaLaunchConfig_t c{};
    c.gridDim = grid;
    c.blockDim = block;
    c.dynamicSmemBytes = smem;
    c.stream = st;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a[0].val.programmaticStreamSerializationAllowed = 1;
    c.attrs = a;
    c.numAttrs = chained ? 1 : 0;
    return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

}  // namespace amsim
