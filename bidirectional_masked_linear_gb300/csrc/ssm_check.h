// ssm_check.h -- which memory the state space block's calls take (no device code).
#pragma once

#include <cuda_runtime_api.h>

namespace lion {

// Memory that kernels of `device` can use.  Another device's own is not taken:
// its address faults unless peer access is on, and its streams order nothing here.
inline bool usable_on(const cudaPointerAttributes& at, int device) {
  if (at.type == cudaMemoryTypeDevice) return at.device == device;
  if (at.type == cudaMemoryTypeManaged) return true;
  return at.type == cudaMemoryTypeHost && at.devicePointer != nullptr;
}

}  // namespace lion
