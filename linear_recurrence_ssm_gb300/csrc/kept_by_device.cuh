// kept_by_device.cuh -- an answer about a kernel, asked of the driver once for
// each device (host side; several threads may ask at once).
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>

namespace ssm {

// `N` answers a device, above 0.  A failure is not kept, and beyond the devices
// that have a place every call asks.
template <int N>
struct KeptByDevice {
    static constexpr int kDevices = 64;
    std::atomic<int> of[kDevices][N];

    // ask(device, &answer)
    template <typename Ask>
    cudaError_t get(int place, int *answer, Ask ask) {
        int device = 0;
        if (cudaError_t e = cudaGetDevice(&device)) return e;
        std::atomic<int> *kept = device < kDevices ? &of[device][place] : nullptr;
        if (kept && (*answer = kept->load(std::memory_order_relaxed)) > 0) return cudaSuccess;
        if (cudaError_t e = ask(device, answer)) return e;
        if (kept) kept->store(*answer, std::memory_order_relaxed);
        return cudaSuccess;
    }
};

}  // namespace ssm
