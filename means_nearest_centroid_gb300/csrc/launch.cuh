// launch.cuh -- chains of launches: a kernel launched with launch_after may
// start its set-up while the kernel before it in the stream still runs, and
// calls wait_for_previous() before it touches anything that kernel wrote (or
// reads).  A kernel that lets its successor do so calls let_next_start().
//
// A kernel so launched may be running while its inputs are still written.  It
// reads them with plain loads: __ldg (and const __restrict__) would promise that
// they do not change while it runs, which lets the compiler move the loads.
#pragma once

#include <cuda_runtime.h>

namespace kma {

__device__ __forceinline__ void let_next_start()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void wait_for_previous()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem,
                         cudaStream_t stream, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace kma
