// Compute units of the current device, asked for once per device.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>

namespace fpx {

inline int current_cus() {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices] = {};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return 256;
  if (dev >= 0 && dev < kDevices) {
    const int n = known[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
  }
  int cus = 0;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) return 256;
  if (dev >= 0 && dev < kDevices) known[dev].store(cus, std::memory_order_relaxed);
  return cus;
}

}  // namespace fpx
