// launch_util.h -- host helpers shared by the kernel launchers (internal).
#pragma once

#include <cuda_runtime.h>

#include <mutex>

namespace ss2d {

constexpr int kMaxDevices = 128;

// Serialises the raising of shared-memory limits across host threads.
inline std::mutex g_configure_smem_mutex;

// Raises a kernel's dynamic shared-memory limit to `bytes` and asks for the largest
// shared-memory carveout, once per device and size (configured[] is per kernel and holds
// the limit set so far on each device).  Safe to call from several host threads: the
// limit only grows, so a call never lowers it under another thread's larger launch.
template <class K>
cudaError_t configure_smem(K kernel, int bytes, int *configured)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 0 || dev >= kMaxDevices)
        return cudaErrorInvalidDevice;
    if (bytes <= __atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE))
        return cudaSuccess;
    std::lock_guard<std::mutex> lock(g_configure_smem_mutex);
    if (bytes <= __atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE))
        return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess)
        return e;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             (int)cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess)
        return e;
    __atomic_store_n(&configured[dev], bytes, __ATOMIC_RELEASE);
    return cudaSuccess;
}

// Launches a kernel that may be scheduled before the work ahead of it in its stream is done
// (programmatic dependent launch), in clusters of `cluster` CTAs.  Such a kernel calls
// grid_wait() in every thread before it reads or writes global memory (it waits for the work ahead, and only what stands
// behind it is promised to see that work's writes), and grid_next() when all that it holds of its SM is taken, so that
// its own successor can be scheduled behind it.  While it is scheduled early the work ahead still writes, so it
// reads nothing through the read-only path (__ldg), which may only be given what no one writes during the kernel.
template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), unsigned grid, int threads, size_t smem, cudaStream_t s, int cluster,
                         const A &...args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attrs[2]{};
    attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[0].val.programmaticStreamSerializationAllowed = 1;
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = (unsigned)cluster;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

#ifdef __CUDACC__
// Waits until the work ahead in the stream is done and its writes are visible.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
// Lets the work behind in the stream be scheduled, once every CTA of this grid has called it or ended.
__device__ __forceinline__ void grid_next() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }
#endif

}  // namespace ss2d
