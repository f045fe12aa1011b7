// Fake devices for a test without a GPU: the streams.  Device d's current
// stream has the handle 0x1000 + d.
#pragma once

#include <c10/core/Device.h>
#include <cuda_runtime_api.h>

namespace fake {
inline int current = 0;          // the current device
}

namespace c10 {
namespace cuda {
struct CUDAStream {
    DeviceIndex device;
    cudaStream_t stream() const { return reinterpret_cast<cudaStream_t>(0x1000 + static_cast<size_t>(device)); }
};
inline CUDAStream getCurrentCUDAStream(DeviceIndex device = -1) {
    return {device < 0 ? static_cast<DeviceIndex>(fake::current) : device};
}
}  // namespace cuda
}  // namespace c10
