// Fake devices for a test without a GPU: the guard that makes a device current
// until it is destroyed.
#pragma once

#include <c10/cuda/CUDAStream.h>

namespace c10 {
namespace cuda {
struct OptionalCUDAGuard {
    int before = -1;
    OptionalCUDAGuard() = default;
    OptionalCUDAGuard(const OptionalCUDAGuard&) = delete;
    void set_index(DeviceIndex device) {
        if (before < 0) before = fake::current;
        fake::current = device;
    }
    ~OptionalCUDAGuard() {
        if (before >= 0) fake::current = before;
    }
};
}  // namespace cuda
}  // namespace c10
