// dyn_smem.h -- a kernel's dynamic shared memory limit, raised as its launches need it.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <mutex>
#include <stddef.h>

namespace moe {

// The largest size set for a kernel, per device (one static object a kernel).
struct SmemSet {
    std::atomic<int> bytes[64];
};

// cudaFuncSetAttribute(MaxDynamicSharedMemorySize), when a launch needs more than was set
// before. Calls may come from several threads: one at a time compares and sets, or a
// smaller size set last would take a larger one back before its launch.
template <typename K>
inline cudaError_t ensure_dyn_smem(K kern, size_t bytes, SmemSet &set) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::atomic<int> *was = dev >= 0 && dev < 64 ? &set.bytes[dev] : nullptr;
    if (was && was->load(std::memory_order_acquire) >= (int)bytes) return cudaSuccess;
    static std::mutex one;
    std::lock_guard<std::mutex> lock(one);
    if (was && was->load(std::memory_order_relaxed) >= (int)bytes) return cudaSuccess;
    e = cudaFuncSetAttribute((const void *)kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && was) was->store((int)bytes, std::memory_order_release);
    return e;
}

}  // namespace moe
