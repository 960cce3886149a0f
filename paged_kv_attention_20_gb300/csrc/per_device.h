// Values that hold for one CUDA device and stay as they are for the process: a
// kernel's attributes set (they hold for the device that was current), its
// resident CTAs, the device's SMs.
#pragma once

#include <atomic>

#include <cuda_runtime.h>

namespace pa {

class PerDevice {
public:
    // The current device's value (> 0): the one kept for it, or what setup(dev, value)
    // works out.  Errors are not kept.  Threads whose first calls meet may each run
    // setup, which has the same effect as running it once.
    template <typename F> cudaError_t get(int &value, F &&setup) {
        int dev = 0;
        const cudaError_t e = cudaGetDevice(&dev);
        return e == cudaSuccess ? get_on(dev, value, setup) : e;
    }
    template <typename F> cudaError_t get_on(int dev, int &value, F &&setup) {
        const bool kept = dev >= 0 && dev < kDevices;
        if (kept) {
            value = known_[dev].load(std::memory_order_acquire);
            if (value) return cudaSuccess;
        }
        const cudaError_t e = setup(dev, value);
        if (e == cudaSuccess && kept) known_[dev].store(value, std::memory_order_release);
        return e;
    }

private:
    static constexpr int kDevices = 64;
    std::atomic<int> known_[kDevices] = {};
};

// Lets `kernel` use `smem` bytes of dynamic shared memory on the current device, once a device.
template <typename K> cudaError_t allow_smem(PerDevice &done, K kernel, size_t smem) {
    int value = 0;
    return done.get(value, [&](int, int &v) {
        v = 1;
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    });
}

// SMs of the current device.
inline cudaError_t device_sms(int &sms) {
    static PerDevice known;
    return known.get(sms, [](int dev, int &v) { return cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev); });
}

// allow_smem for a persistent kernel; ctas: how many of its CTAs the device holds at once.
template <typename K>
cudaError_t resident_ctas(PerDevice &done, K kernel, int threads, size_t smem, int &ctas) {
    return done.get(ctas, [&](int dev, int &v) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        int per_sm = 0, sms = 0;
        if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        v = per_sm * sms > 0 ? per_sm * sms : 1;
        return e;
    });
}

}  // namespace pa
