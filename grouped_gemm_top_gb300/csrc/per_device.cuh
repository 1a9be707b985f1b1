// What moe_init finds out about a device, kept for each.
#pragma once

#include <cuda_runtime_api.h>

namespace moe {

constexpr int kMaxDevices = 64;

// A T for every device; here() is the current one's (all zeros where there is
// none).  moe_init writes it before its device counts as initialised, so a call
// never plans by another device's numbers, nor reads them while they are written.
template <typename T>
class PerDevice {
public:
    T& here() {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return none_ = T{};
        return of_[dev];
    }

private:
    T of_[kMaxDevices] = {};
    T none_ = {};
};

}  // namespace moe
