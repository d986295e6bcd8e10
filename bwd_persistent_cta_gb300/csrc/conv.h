// conv.h - launch interface of the causal convolution.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "rnn.h"

namespace rnn {

struct ConvArgs {
  int B, T, D, W;
  int bfirst, silu;
  const int* len;              // [B] valid tokens, or null = T
  const void *x, *w, *bias;
  int64_t x_row;
  int num_sms;

  __host__ __device__ int64_t row(int b, int t) const {
    return bfirst ? static_cast<int64_t>(b) * T + t : static_cast<int64_t>(t) * B + b;
  }
};

struct ConvFwdArgs {
  ConvArgs a;
  const void* s0;              // [B][W - 1][D] or null
  void *y, *sT;                // sT or null
};
int launch_conv_forward(const ConvFwdArgs& f, int is_bf16, cudaStream_t s);

size_t conv_workspace_bytes(const ConvArgs& a);

struct ConvBwdArgs {
  ConvArgs a;
  const void *s0, *dy, *dsT;
  void *dx, *ds0;
  float *dw, *dbias;
  float* partial;              // [CTA][W + 1][D], or null
};
int launch_conv_backward(const ConvBwdArgs& b, int is_bf16, cudaStream_t s, int* launches);

struct ConvStepArgs {
  ConvArgs a;
  void* state;                 // [slot][W - 1][D]
  const int* slots;            // [B] or null = b
  int num_slots;
  void* y;
};
int launch_conv_step(const ConvStepArgs& p, int is_bf16, cudaStream_t s);

}  // namespace rnn
