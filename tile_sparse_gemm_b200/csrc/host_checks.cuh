// Argument checks shared by the C ABI's source files.
#pragma once

#include <cuda_runtime.h>

#include "patch.h"

namespace patch {

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// SM count of the current device; PATCH_ERR_DEVICE unless it is compute capability 10.x
inline patch_status_t device_sms(int* sms) {
  int dev = 0, major = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PATCH_ERR_CUDA;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess)
    return PATCH_ERR_CUDA;
  if (major != 10) return PATCH_ERR_DEVICE;
  if (cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return PATCH_ERR_CUDA;
  return PATCH_OK;
}

}  // namespace patch
