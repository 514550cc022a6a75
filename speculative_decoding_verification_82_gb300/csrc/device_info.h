// device_info.h -- the current device's number of multiprocessors, looked up once per device.
//
// Any host thread may call it at any time, so the kept values are atomic; a value found twice is the same value.
#pragma once

#include <cuda_runtime_api.h>

#include <atomic>

namespace specv {

// The multiprocessors of the current device, or -1 where the runtime gives none; *device receives the device.
inline int sm_count(int* device = nullptr) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return -1;
  if (device) *device = dev;
  static std::atomic<int> cache[64];
  if (dev < 64) {
    const int known = cache[dev].load(std::memory_order_relaxed);
    if (known > 0) return known;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
  if (dev < 64) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace specv
