// Launches with programmatic stream serialisation: a kernel's CTAs may be
// scheduled while the last CTAs of the kernel before it in the stream still
// run, so that its launch and its set-up overlap their tail.  Every kernel
// launched this way calls grid_wait() before its first access to global memory
// (reads and writes): the call returns once the kernels before it have ended
// and their writes are visible.
#pragma once
#include <cuda_runtime.h>

#include <utility>

namespace mxa2a {

// (Data that an earlier kernel may have written is read after this call with
// plain or volatile loads: a load that the compiler takes for invariant could
// be moved above it.)
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// the next kernel may be scheduled once every CTA has got here
__device__ __forceinline__ void grid_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// cluster: CTAs per cluster, 1 for none
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, unsigned threads, size_t smem, int cluster, cudaStream_t stream,
                   Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim = {(unsigned)cluster, 1, 1};
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Opt in to `bytes` of dynamic shared memory, once per device and kernel (the
// call costs more than a launch).  `done`: a static bit set of the caller.
template <typename K>
cudaError_t allow_smem(K kernel, size_t bytes, unsigned long long& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && (__atomic_load_n(&done, __ATOMIC_ACQUIRE) >> dev & 1)) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && dev < 64) __atomic_fetch_or(&done, 1ull << dev, __ATOMIC_RELEASE);
    return e;
}

}  // namespace mxa2a
