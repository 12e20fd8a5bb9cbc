// See HIPFunctions.h beside it.
#pragma once
#include <c10/hip/HIPFunctions.h>
#include <hip/hip_runtime_api.h>

namespace c10::hip {
struct HIPStream {
  hipStream_t stream() const { return nullptr; }
};
inline HIPStream getCurrentHIPStream(c10::DeviceIndex) { return {}; }
}  // namespace c10::hip
