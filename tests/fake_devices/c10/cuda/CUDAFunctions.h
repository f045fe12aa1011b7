// Fake devices for a test without a GPU: the current one.
#pragma once

#include <c10/cuda/CUDAStream.h>

namespace c10 {
namespace cuda {
inline DeviceIndex current_device() { return static_cast<DeviceIndex>(fake::current); }
}  // namespace cuda
}  // namespace c10
