// delta.h - internal layouts and launch interfaces of the gated delta rule.
//
// Per (sequence b, value head h) = bh = b * Hv + h, with chunks of C tokens
// counted from the start of the sequence (nc = ceil(T / C)):
//   S0  [bh][chunk][Dv][Dk]   the state before each chunk
//   E   [bh][t][Dv] fp32      e_t = v_t - a_t S_{t-1} k_t
//   dS1 [bh][chunk][Dv][Dk]   the gradient of the state after each chunk
//   Y   [bh][t][Dv] fp32      y_t, the gradient of u_t = beta_t e_t
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "rnn.h"

namespace rnn {

struct DeltaArgs {
  int B, T, Hk, Hv, Dk, Dv;
  int bfirst;
  float scale;
  const int* len;              // [B] valid tokens, or null = T
  const void *q, *k, *v, *g, *beta;
  int64_t q_row, k_row, v_row, g_row, beta_row;

  __host__ __device__ int64_t row(int b, int t) const {
    return bfirst ? static_cast<int64_t>(b) * T + t : static_cast<int64_t>(t) * B + b;
  }
};

// exp(kDecayFloor) is below the smallest fp32 subnormal, so a decay that is
// not representable (g = -inf included) acts as a reset: the floor keeps
// differences of cumulative decays free of inf - inf.
constexpr float kDecayFloor = -110.f;

// Cumulative decays are unevaluated sums of two floats: the difference of two of
// them stays exact to fp32 however many resets lie before both.
struct TwoF {
  float h, l;
};
__device__ __forceinline__ TwoF two_add(TwoF a, TwoF b) {
  const float s = a.h + b.h, bb = s - a.h;
  const float err = (a.h - (s - bb)) + (b.h - bb);
  const float l = err + (a.l + b.l);
  const float h = s + l;
  return {h, l - (h - s)};
}

// --- fp32 kernels: every type and size --------------------------------------
constexpr int kSimtChunk = 32;

struct DeltaRecurArgs {
  DeltaArgs a;
  const float* s_in;           // [slot][Hv][Dv][Dk] or null = zero
  float* s_out;                // same layout, or null
  const int* slots;            // [B] or null = b
  int num_slots;
  void* o;
  float* ckpt;                 // S0 of every chunk, or null
  float* e;                    // E, or null
  unsigned int* status;        // the serving step: where a bounded wait reports
  int num_sms;
};
int launch_delta_recur(const DeltaRecurArgs& r, int is_bf16, cudaStream_t s);

// The serving step's pipeline.  Turn n of a CTA's walk fills stage n % kUnits; the
// phase of that fill has the parity of n / kUnits.  At turn n the fills of turns
// n .. n + kUnits - 1 are under way, as far as the walk has that many.
constexpr int kUnits = 4;
struct StepFill {
  int stage;
  unsigned int parity;
};
__host__ __device__ constexpr StepFill step_fill(int turn) {
  return {turn % kUnits, static_cast<unsigned int>(turn / kUnits) & 1u};
}
// The last turn whose fill is under way at turn ``turn`` of a walk of ``turns``.
__host__ __device__ constexpr int step_last_fill(int turn, int turns) {
  return turn + kUnits < turns ? turn + kUnits - 1 : turns - 1;
}

struct DeltaRecurBwdArgs {
  DeltaArgs a;
  const void* dout;
  const float* dsT;            // or null
  float* ds0;                  // or null
  float* ckpt;                 // dS1 of every chunk
  float* y;
  int num_sms;
};
int launch_delta_recur_bwd(const DeltaRecurBwdArgs& r, int is_bf16, cudaStream_t s);

struct DeltaChunkBwdArgs {
  DeltaArgs a;
  const void* dout;
  const float *s0, *ds1, *e, *y;
  void *dq, *dk, *dv, *dg, *dbeta;
};
int launch_delta_chunk_bwd(const DeltaChunkBwdArgs& r, int is_bf16, cudaStream_t s);

}  // namespace rnn
