// clip.h - launch interface of gradient clipping.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "rnn.h"

namespace rnn {

// The tensors of a launch come as kernel arguments, which a graph keeps with the
// node: up to this many.
constexpr int kClipGroup = 1000;

struct ClipArgs {
  int num;                     // tensors
  const int64_t* start;        // device [num + 1]: elements before each tensor
  const int* dtype;            // device [num]
  const int64_t* host_start;   // host, the same
  const void* const* grads;    // host
  void* const* out;            // host, or null = in place
  float max_norm, eps;
  float* norm;
  double* partial;             // [launch][CTA]
  int scale;                   // 0: the norm alone
  int split;                   // tensors scaled in place go last: others read their memory
  int num_sms;
};
size_t clip_workspace_bytes(int num, int num_sms);
int launch_clip(const ClipArgs& c, cudaStream_t s, int* launches);

}  // namespace rnn
