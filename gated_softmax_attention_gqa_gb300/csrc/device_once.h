// device_once.h -- what is asked of or set on a device once and then remembered (host side).
// Calls come from several threads, none of which holds a lock: the tables are atomic, and
// two threads that find an entry missing both fill it in, alike.
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>

namespace gattn {

// Raise a kernel's dynamic shared-memory limit once per device.
// `func` identifies the kernel; up to 64 kernels per device are remembered
// (beyond that the attribute is simply set again on every call).
inline cudaError_t set_smem_once(const void* func, int bytes) {
    constexpr int kDevices = 64, kKernels = 64;
    static std::atomic<const void*> seen[kDevices][kKernels] = {};  // filled from the front
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < kDevices;
    for (int i = 0; known && i < kKernels; ++i) {
        const void* f = seen[dev][i].load(std::memory_order_acquire);
        if (f == func) return cudaSuccess;
        if (!f) break;
    }
    e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    for (int i = 0; known && i < kKernels; ++i) {
        const void* f = nullptr;
        if (seen[dev][i].compare_exchange_strong(f, func, std::memory_order_acq_rel) || f == func) break;
    }
    return cudaSuccess;
}

// SMs of the current device, 0 on failure.
inline int sm_count() {
    static std::atomic<int> cached[64] = {};
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const bool known = dev >= 0 && dev < 64;
    if (known && (n = cached[dev].load(std::memory_order_relaxed)) > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (known) cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace gattn
