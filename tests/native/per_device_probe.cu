// Host build of the library's per-device values (pa::PerDevice), so a CPU test
// can drive them with device numbers of its own.  Test infrastructure only:
// nothing in the library uses it.
#include <thread>
#include <vector>

#include "per_device.h"

static pa::PerDevice g_values;

// Value kept for `dev`; a first call works out `fresh` (and fails when it is 0).  -1: failed.
extern "C" int probe_per_device(int dev, int fresh, int *setups) {
    int value = 0;
    const cudaError_t e = g_values.get_on(dev, value, [&](int d, int &v) {
        ++*setups;
        v = fresh;
        return d == dev && fresh ? cudaSuccess : cudaErrorInvalidValue;
    });
    return e == cudaSuccess ? value : -1;
}

// First calls of `threads` threads on each of devices 0..15, all at once: the
// number of calls that saw another value than their device's.
extern "C" int probe_per_device_threads(int threads) {
    pa::PerDevice values;
    std::atomic<int> wrong{0};
    std::vector<std::thread> all;
    for (int t = 0; t < threads; ++t)
        all.emplace_back([&] {
            for (int dev = 0; dev < 16; ++dev) {
                int value = 0;
                const cudaError_t e = values.get_on(dev, value, [](int d, int &v) {
                    v = 100 + d;
                    return cudaSuccess;
                });
                if (e != cudaSuccess || value != 100 + dev) ++wrong;
            }
        });
    for (auto &t : all) t.join();
    return wrong.load();
}
