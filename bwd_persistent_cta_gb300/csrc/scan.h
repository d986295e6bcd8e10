// scan.h - launch interface of the selective scan.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "rnn.h"

namespace rnn {

// Tokens a tile: what a CTA stages at once, and the distance of the states that a
// training forward keeps.
constexpr int kScanTile = 16;

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
  __host__ __device__ int tiles() const { return (T + kScanTile - 1) / kScanTile; }
};

// A long sequence runs as several segments side by side.  ends: byte offset of [B][nseg]
// [D][N], the state that each segment alone leaves; sums: of [B][nseg][D], the sum of its
// steps; first: of [B][D][N], the initial state where the final one overwrites it.
struct ScanSplit {
  int nseg, len;               // segments, tokens of each (a multiple of the tile)
  size_t ends, sums, first, bytes;
};
ScanSplit scan_split(const ScanArgs& a, int is_bf16);

struct ScanFwdArgs {
  ScanArgs a;
  const float* h0;             // or null
  float* hT;                   // or null
  void* y;
  float* kept;                 // [B][tile][D][N] the state before each tile, or null
  int nseg, seg;               // segments, tokens of each
  float *ends, *sums;
  float* first;                // where the first segment copies h0 to, or null
};
int launch_scan_forward(const ScanFwdArgs& f, void* work, int is_bf16, cudaStream_t s, int* launches);

// Byte offsets of the backward's scratch: partial sums over channels (of dB and dC),
// over tokens and sequences (of dA, dD and the bias).
struct ScanBwdLayout {
  size_t bc, dA, dD, dbias, bytes;
};
ScanBwdLayout scan_bwd_layout(const ScanArgs& a);

struct ScanBwdArgs {
  ScanArgs a;
  const void* dy;
  const float* dhT;            // or null
  const float* kept;
  rnn_scan_grad_t grad;
  char* work;
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
