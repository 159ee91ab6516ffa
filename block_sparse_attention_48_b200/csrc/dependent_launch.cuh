// Launch of a kernel whose CTAs may start before the stream's previous kernel has ended
// (programmatic dependent launch).  The kernel itself waits for that end before it reads or
// writes anything (wait_prerequisites, by every thread); what is gained is the launch's
// latency, and the start of CTAs on SMs that the previous kernel has left.
//
// What the previous kernel writes is then written while this one is already running.  So
// such a kernel loads with ordinary loads, which are coherent and stay behind the wait: the
// read-only path (__ldg, ld.global.nc) is for memory that nothing writes in a kernel's whole
// lifetime, and the compiler may move such loads, and those of the other __ld functions, over
// the wait.
#pragma once

#include <cuda_runtime.h>

namespace fa {

// The stream's next kernel may start its CTAs once every CTA of this one has called this.
__device__ __forceinline__ void launch_dependents()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// The previous kernel has ended, and what it wrote can be read.
__device__ __forceinline__ void wait_prerequisites()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <class... P>
inline cudaError_t launch_after(void (*kern)(P...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                                const P&... p)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p...);
}

} // namespace fa
