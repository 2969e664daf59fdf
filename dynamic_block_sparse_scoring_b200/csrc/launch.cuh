// What the launchers of the window and paged kernels ask of the device, asked once per device.
#pragma once

#include <atomic>

#include "common.cuh"

namespace nsa {

constexpr int MAX_DEVICES = 64;

// SM count of the current device.
inline cudaError_t sm_count(int* n, int* device) {
    static std::atomic<int> known[MAX_DEVICES];
    cudaError_t e = cudaGetDevice(device);
    if (e != cudaSuccess) return e;
    const bool keep = *device >= 0 && *device < MAX_DEVICES;
    if (keep && (*n = known[*device].load(std::memory_order_relaxed)) > 0) return cudaSuccess;
    e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, *device);
    if (e == cudaSuccess && keep) known[*device].store(*n, std::memory_order_relaxed);
    return e;
}

// Allows `bytes` of dynamic shared memory for a kernel on `device`, once; one
// `done` array per kernel.
inline cudaError_t allow_smem(const void* kernel, int bytes, int device, std::atomic<bool>* done) {
    const bool keep = device >= 0 && device < MAX_DEVICES;
    if (keep && done[device].load(std::memory_order_relaxed)) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && keep) done[device].store(true, std::memory_order_relaxed);
    return e;
}

// Launches a kernel that may start while the one before it in the stream still
// runs; it waits for that one's results itself (griddepcontrol.wait).
template <class... Params, class... Args>
cudaError_t launch_dependent(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                             const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

__device__ __forceinline__ void pdl_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace nsa
