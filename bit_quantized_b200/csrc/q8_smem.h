// The dynamic shared-memory limit of a kernel (host code only).
#pragma once

#include <cuda_runtime_api.h>

#include <mutex>
#include <new>
#include <unordered_map>

namespace q8 {

// Lets `kernel` launch with `bytes` of dynamic shared memory on the current
// device.  The limit is a per-kernel, per-device attribute: it is set once (to
// the largest size asked for) instead of on every launch, which keeps the host
// side of a call short.  Setting it replaces it, so a size is looked up, set and
// recorded under one lock: two threads that ask for different sizes at once
// would otherwise leave the smaller limit in place under the larger record.
inline cudaError_t raise_smem_limit(const void* kernel, int bytes) {
    static std::mutex mu;
    static std::unordered_map<const void*, int> limits[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
        cudaGetLastError();
        return cudaErrorInvalidDevice;
    }
    std::lock_guard<std::mutex> lk(mu);
    int* limit;
    try {
        limit = &limits[dev][kernel];
    } catch (const std::bad_alloc&) {   // no exception leaves through the C interface
        return cudaErrorMemoryAllocation;
    }
    if (*limit >= bytes) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) *limit = bytes;
    else cudaGetLastError();
    return e;
}

template <typename K>
cudaError_t set_smem(K kernel, int bytes) {
    return raise_smem_limit(reinterpret_cast<const void*>(kernel), bytes);
}

}  // namespace q8
