// esa_host.h -- host-side checks shared by the units that define C ABI
// entry points.  Internal to the library.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace esa {

// ESA_OK when the current device is compute capability 10.0, else ESA_ERR_DEVICE.
int check_current_device();

inline bool aligned_to(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// 0, or ESA_ERR_LAUNCH with the runtime's sticky error cleared.
inline int runtime_status(cudaError_t e) {
  if (e == cudaSuccess) return 0;
  cudaGetLastError();
  return -5;
}

// SM count of the current device (148 when it cannot be read).
int sm_count();

}  // namespace esa
