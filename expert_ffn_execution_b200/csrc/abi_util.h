// abi_util.h -- what the C entry points share: device facts, argument checks.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "strata_moe.h"

namespace strata {

constexpr int kMaxDevices = 64;

inline int num_sms_of_current_device() {
  static int cache[kMaxDevices] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
  if (cache[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
      n = 148;
    cache[dev] = n;
  }
  return cache[dev];
}

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline int32_t from_cuda(cudaError_t e) { return e == cudaSuccess ? STRATA_OK : STRATA_ECUDA; }

// Bytes of an element, 0 for an unknown dtype.
inline int dtype_bytes(int32_t dt) {
  return dt == STRATA_DTYPE_F32 ? 4 : (dt == STRATA_DTYPE_F16 || dt == STRATA_DTYPE_BF16) ? 2 : 0;
}

}  // namespace strata
