// launch.cuh -- kernels that start while the one before them ends.
//
// A kernel launched by launch_early may be set up (its CTAs resident, barriers
// and tensor memory ready) before the kernel ahead of it in the stream has
// finished; it calls wait_for_stream() in every thread before it reads or
// writes any memory that another kernel may use.  From there on the kernel
// behind it may be set up in turn, once all its own CTAs have come that far: a
// waiting CTA never keeps one out that it waits for.  A kernel ends after the
// one it waited for, so the order of the stream holds along a chain, and in a
// captured graph as well.  Chains of small kernels gain 2 to 4 us a step.
//
// Such a kernel reads global memory with ordinary loads alone.  The read-only
// path (__ldg, ld.global.nc, const __restrict__) wants memory that nobody
// writes as long as the kernel lives, and here the kernel ahead may be writing
// it still; the compiler may also move such a load ahead of the wait.
#pragma once

#include <cuda_runtime.h>

namespace nvfp4 {

__device__ __forceinline__ void wait_for_stream() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... P, typename... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, int cluster, const A&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace nvfp4
