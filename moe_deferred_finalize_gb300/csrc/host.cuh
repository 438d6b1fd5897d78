// Host helpers shared by the C-ABI translation units: alignment checks, the
// device's multiprocessor count, and the status of runtime calls.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "moe_finalize.h"

namespace moef {

constexpr int kMaxDevices = 64;

inline bool aligned(const void *p, uintptr_t a) {
    return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}

// Multiprocessor count of the current device, cached per device (host
// threads may race to fill an entry; they all store the same value).
inline cudaError_t current_sms(int *sms) {
    static std::atomic<int> cache[kMaxDevices];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev >= 0 && dev < kMaxDevices) {
        const int cached = cache[dev].load(std::memory_order_relaxed);
        if (cached > 0) {
            *sms = cached;
            return cudaSuccess;
        }
    }
    int n = 0;
    err = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (err != cudaSuccess) return err;
    if (dev >= 0 && dev < kMaxDevices) cache[dev].store(n, std::memory_order_relaxed);
    *sms = n;
    return cudaSuccess;
}

// Status of a runtime call.  A refused call also leaves its error in the
// thread's last-error slot, where the caller's next unrelated launch check
// would find it; the error is reported here, so it is taken out of the slot.
inline moef_status cuda_status(cudaError_t err) {
    if (err == cudaSuccess) return MOEF_OK;
    (void)cudaGetLastError();
    return MOEF_ERR_CUDA;
}

}  // namespace moef
