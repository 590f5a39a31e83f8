// gdn_launch.cuh -- launches that overlap the end of the kernel before them on the stream.
//
// A kernel started by launch_after() may have its CTAs on the SMs while the stream's previous kernel
// still runs; its first instruction of weight is begin_after(), which waits until that kernel is complete
// and its writes are visible, and then lets the next kernel's CTAs come as these leave.  Nothing is read or
// written before it.  What is saved is the launch itself, 1 to 3 us between kernels of a few us.
#pragma once

#include "gdn_tc.cuh"

namespace gdn {

#if defined(__CUDACC__)
__device__ __forceinline__ void begin_after()
{
    tc::grid_dep_wait();
    tc::grid_dep_launch();
}

template <typename... P>
inline int launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, P... args)
{
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return (int)cudaLaunchKernelEx(&cfg, kernel, args...);
}
#endif

}  // namespace gdn
