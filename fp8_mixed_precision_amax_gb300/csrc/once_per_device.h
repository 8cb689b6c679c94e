// once_per_device.h -- set-up that CUDA keeps for each device by itself: a kernel's
// shared-memory limit (cudaFuncSetAttribute acts on the current device), how many
// clusters fit.
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>
#include <cstddef>

namespace fp8k {

constexpr int kDeviceSlots = 64;   // devices a process may use

// Runs a set-up at the first use on each device.  One that fails is tried again by the next
// call.  Threads that come at the same time may both run it, which these set-ups allow: so
// there is no lock, and no exception on the way to a C entry point.
class OncePerDevice {
    std::atomic<bool> done_[kDeviceSlots] = {};

   public:
    // set_up(device) -> cudaError_t; *device: the current device
    template <typename F>
    cudaError_t run(F set_up, int *device = nullptr) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        if (dev < 0 || dev >= kDeviceSlots) return cudaErrorInvalidDevice;
        if (device != nullptr) *device = dev;
        if (done_[dev].load(std::memory_order_acquire)) return cudaSuccess;
        e = set_up(dev);
        if (e == cudaSuccess) done_[dev].store(true, std::memory_order_release);
        return e;
    }
};

// A kernel's limit of dynamic shared memory, raised on each device that launches it.  One
// (static) object for each kernel.
class SmemLimit {
    OncePerDevice once_;

   public:
    template <typename K>
    cudaError_t allow(K *kernel, size_t bytes) {
        return once_.run([kernel, bytes](int) {
            return cudaFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(bytes));
        });
    }
};

}  // namespace fp8k
