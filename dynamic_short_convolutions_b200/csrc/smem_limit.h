// smem_limit.h -- raises a kernel's dynamic shared-memory limit, once per device.
#pragma once

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

namespace dynconv {

// The attribute belongs to the kernel on a device and stays; setting it costs a launch of a few microseconds a
// good part of its host time, so it is set on the first launch there (`done`: a bit per device, one word per
// kernel; devices from 64 on set it every time).
inline cudaError_t smem_limit(std::atomic<uint64_t>& done, const void* kernel, size_t bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && bit) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

}  // namespace dynconv

// One word per expansion: expand it once per kernel instantiation (inside the templated launcher).
#define DC_SMEM_LIMIT(kernel, bytes)                                                  \
    ([&]() {                                                                          \
        static std::atomic<uint64_t> done{0};                                         \
        return ::dynconv::smem_limit(done, reinterpret_cast<const void*>(kernel), bytes); \
    }())
