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

}  // namespace nsa
