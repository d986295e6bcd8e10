// scan.h - launch interface of the selective scan.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "rnn.h"

namespace rnn {

// Tokens between the states that a training forward keeps.
constexpr int kScanKeep = 4;

struct ScanArgs {
  int B, T, D, N, G;
  int bfirst, softplus;
  const int* len;              // [B] valid tokens, or null = T
  const void *x, *dt, *z, *Bm, *Cm;
  const float *A, *skip, *bias;
  int64_t x_row, dt_row, z_row, B_row, C_row;
  int num_sms;

  __host__ __device__ int64_t row(int b, int t) const {
    return bfirst ? static_cast<int64_t>(b) * T + t : static_cast<int64_t>(t) * B + b;
  }
  __host__ __device__ int keeps() const { return (T + kScanKeep - 1) / kScanKeep; }
};

// A long sequence runs as several segments side by side: what each leaves by itself
// (the state forward, its gradient backward, and the sum of its steps) is computed
// first.  Byte offsets in the scratch of a call.
struct ScanSplit {
  int nseg, len;               // segments, tokens of each
  size_t ends;                 // [B][nseg][D][N]
  size_t sums;                 // [B][nseg][D]
  size_t first;                // [B][D][N]: the initial state where the final one overwrites it
  size_t bytes;
};
ScanSplit scan_split_forward(const ScanArgs& a, int is_bf16);
ScanSplit scan_split_backward(const ScanArgs& a);

struct ScanSegs {
  int nseg, len;
  float *ends, *sums;
};

// The reserve: what a training forward keeps.
struct ScanReserve {
  size_t kept, ungated, bytes;
};
ScanReserve scan_reserve(const ScanArgs& a);

struct ScanFwdArgs {
  ScanArgs a;
  const float* h0;             // or null
  float* hT;                   // or null
  void* y;
  float* kept;                 // [B][keep][D][N] the state before every kScanKeep tokens, or null
  float* ungated;              // [rows][D] y before its gate, or null
  ScanSegs g;
  float* first;                // where the first segment copies h0 to, or null
};
int launch_scan_forward(const ScanFwdArgs& f, void* work, int is_bf16, cudaStream_t s, int* launches);

// Byte offsets of the backward's scratch behind its segments': partial sums over channels
// (of dB and dC), over tokens and sequences (of dA, dD and the bias).
struct ScanBwdLayout {
  size_t bc, dA, dD, dbias, bytes;
};
ScanBwdLayout scan_bwd_layout(const ScanArgs& a);

struct ScanBwdArgs {
  ScanArgs a;
  const void* dy;
  const float* dhT;            // or null
  const float *kept, *ungated;
  rnn_scan_grad_t grad;
  char* work;
  ScanSegs g;
  float *bc, *pA, *pD, *pbias; // partial sums, or null
};
int launch_scan_backward(const ScanBwdArgs& b, int is_bf16, cudaStream_t s, int* launches);

struct ScanStepArgs {
  ScanArgs a;
  float* state;                // [slot][D][N]
  const int* slots;            // [B] or null = b
  int num_slots;
  void* y;
};
int launch_scan_step(const ScanStepArgs& p, int is_bf16, cudaStream_t s);

}  // namespace rnn
