// device_guard.h - the device switch around each C-ABI call.
#pragma once

#include <cuda_runtime.h>

namespace rnn {

// Makes the handle's device current for one call and puts the caller's
// current device back afterwards (nothing to do when it already is current).
struct DeviceGuard {
  int prev = -1;
  bool ok = true;
  explicit DeviceGuard(int dev) {
    int cur = 0;
    if (cudaGetDevice(&cur) != cudaSuccess) { ok = false; return; }
    if (cur == dev) return;
    if (cudaSetDevice(dev) != cudaSuccess) { ok = false; return; }
    prev = cur;
  }
  ~DeviceGuard() {
    if (prev >= 0) cudaSetDevice(prev);
  }
  DeviceGuard(const DeviceGuard&) = delete;
  DeviceGuard& operator=(const DeviceGuard&) = delete;
};

}  // namespace rnn
