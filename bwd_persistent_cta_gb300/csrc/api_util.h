// api_util.h - what the entry points of the operators beside the recurrent layers
// share: argument checks, buffer layout, and a call's place among its handle's.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "call_order.h"
#include "device_guard.h"
#include "rnn.h"

namespace rnn {

inline size_t al(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline bool flag(int v) { return v == 0 || v == 1; }

// The current device, when it is one the kernels run on.
inline rnn_status_t pick_device(int* dev, int* sms) {
  if (cudaGetDevice(dev) != cudaSuccess) return RNN_CUDA_ERROR;
  int major = 0, minor = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *dev) != cudaSuccess ||
      cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess)
    return RNN_CUDA_ERROR;
  return major == 10 && minor == 3 ? RNN_OK : RNN_NOT_SUPPORTED;
}

struct Bump {
  size_t off = 0;
  size_t take(size_t bytes) {
    const size_t o = off;
    off = al(off + bytes);
    return o;
  }
};

// A row stride in elements: 0 = dense; otherwise at least a row, and a
// multiple of ``unit`` elements.
inline bool row_ok(int64_t row, int64_t dense, int64_t unit, int64_t* out) {
  *out = row ? row : dense;
  return *out >= dense && *out % unit == 0;
}

// A call's place among the handle's calls that share something on the device:
// lengths, workspace or reserve.
struct Ordered {
  CallOrder& order;
  cudaStream_t s;
  bool on;
  rnn_status_t rc = RNN_OK;
  Ordered(CallOrder& order_, bool shares, cudaStream_t s_) : order(order_), s(s_), on(shares) {
    if (on) rc = order.enter(s);
  }
  // The call's status; what was launched before a failure counts as well.
  rnn_status_t done(int e) {
    const rnn_status_t l = on ? order.leave(s) : RNN_OK;
    return e ? static_cast<rnn_status_t>(e) : l;
  }
};

// New lengths of a handle's sequences: a host array of B ints in [0, T], or null
// for full length.
inline rnn_status_t set_lengths(CallOrder& order, const int* lengths, int B, int T, int** d_len, int* has_len) {
  if (!lengths) {
    *has_len = 0;
    return RNN_OK;
  }
  for (int b = 0; b < B; ++b)
    if (lengths[b] < 0 || lengths[b] > T) return RNN_BAD_PARAM;
  if (!*d_len && cudaMalloc(d_len, sizeof(int) * B) != cudaSuccess) {
    *d_len = nullptr;
    return RNN_CUDA_ERROR;
  }
  // no call may still read the old lengths, and none may start before the new
  // ones have landed: a copy from pageable memory can return earlier, and streams
  // that do not wait for the legacy stream would not wait for it either
  if (order.wait() != RNN_OK ||
      cudaMemcpy(*d_len, lengths, sizeof(int) * B, cudaMemcpyHostToDevice) != cudaSuccess ||
      cudaStreamSynchronize(cudaStreamLegacy) != cudaSuccess)
    return RNN_CUDA_ERROR;
  *has_len = 1;
  return RNN_OK;
}

template <typename T>
T* at(const void* base, size_t off) {
  return reinterpret_cast<T*>(const_cast<char*>(static_cast<const char*>(base)) + off);
}

}  // namespace rnn
