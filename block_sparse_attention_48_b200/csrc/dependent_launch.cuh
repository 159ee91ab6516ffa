// Launch of a kernel whose CTAs may start before the stream's previous kernel has ended
// (programmatic dependent launch).  The kernel itself waits for that end before it reads or
// writes anything (wait_prerequisites, by every thread); what is gained is the launch's
// latency, and the start of CTAs on SMs that the previous kernel has left.
//
// What the previous kernel writes is then written while this one is already running.  So
// such a kernel loads with ordinary loads, or ld_cg: the read-only path (__ldg, ld.global.nc)
// is for memory that nothing writes in a kernel's whole lifetime, and the compiler may move
// such loads, and the other __ld functions, over the wait.
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

// Loads from L2, issued where they stand: of what other CTAs of this kernel, or the kernel
// before, have written.
__device__ __forceinline__ int ld_cg(const int* p)
{
    int x;
    asm volatile("ld.global.cg.s32 %0, [%1];" : "=r"(x) : "l"(p) : "memory");
    return x;
}

__device__ __forceinline__ float2 ld_cg(const float2* p)
{
    float2 x;
    asm volatile("ld.global.cg.v2.f32 {%0, %1}, [%2];" : "=f"(x.x), "=f"(x.y) : "l"(p) : "memory");
    return x;
}

__device__ __forceinline__ float4 ld_cg(const float4* p)
{
    float4 x;
    asm volatile("ld.global.cg.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                 : "l"(p)
                 : "memory");
    return x;
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
