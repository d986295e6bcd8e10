// norm.h - launch interface of the block norm.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "rnn.h"

namespace rnn {

struct NormArgs {
  int rows, groups, cols;
  int norm_in, gate, residual, norm_out;
  float eps;
  const void *y, *z, *x, *w_in, *scale, *w_out;
  int64_t y_row, z_row, x_row;
  // forward
  void *x_out, *n_out;
  // backward
  const void *dx_out, *dn_out;
  void *dy, *dz, *dx;
  float *dw_in, *dscale, *dw_out;
  float* partial;              // [3][CTAs][cols]
  int num_sms;
};

size_t norm_workspace_bytes(const NormArgs& a);
int launch_norm_forward(const NormArgs& a, int is_bf16, cudaStream_t s);
// *launches receives the number of kernels.
int launch_norm_backward(const NormArgs& a, int is_bf16, cudaStream_t s, int* launches);

}  // namespace rnn
