// fa_pdl.cuh -- programmatic dependent launch for the rotation, the paged cache and its decode:
// short kernels that follow one another in a serving step.
#pragma once

#include <atomic>

#include <cuda_runtime.h>

#include "fa_internal.h"

namespace fa {

// pdl_launch(): the next kernel of the stream may be launched once every CTA of this one has said
// so (or ended); it runs its prologue and stops at its pdl_wait().  pdl_wait(): returns when the
// kernels before this one have ended and their writes are visible.  Every CTA of such a kernel
// calls it before its first access to device memory, so that the end of a kernel still means the
// end of all before it.  One exception: the kernels that join states read a length in front of it, past the L1
// (__ldcg).  The kernel before each of them says pdl_launch() only behind its own pdl_wait(), on every path, and
// so whatever wrote the lengths has ended.
__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Allows a kernel its dynamic shared memory (more than 48 KB), once on each device: 0.2 us a call otherwise.
template <auto Kernel>
int allow_smem(size_t bytes)
{
    static std::atomic<unsigned long long> done{0};   // a bit a device
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess)
        return ERR_CUDA;
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit)
        return OK;
    if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != cudaSuccess)
        return ERR_CUDA;
    done.fetch_or(bit, std::memory_order_relaxed);
    return OK;
}

// Launches a kernel; with overlap, one that calls pdl_wait() and may start while the one before it
// still runs, so that the launch latency is hidden.  cluster > 0: CTAs of a cluster.
template <typename... P, typename... A>
int launch_overlapped(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster, bool overlap, cudaStream_t s,
                      const A &...args)
{
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = overlap ? 1 : 0;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 0 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? OK : ERR_CUDA;
}

}  // namespace fa
