// delta_tc.h - the gated delta rule on tensor cores (bf16 storage): buffers and
// launches.  Chunks of 64 tokens; everything a matrix instruction reads is fp16
// scaled by a power of two (see delta_tc.cu).
//
// Per key head (bk = b * Hk + hk) and value head (bh = b * Hv + h), tiles of one
// chunk, each row's 16-byte pieces exchanged by (row & 7) so that the tile is
// copied to shared memory as it is and read there without bank conflicts:
//   K16, Q16 [bk][chunk][64][Dk]  k and q, columns in the order of the MMA
//            fragments (position 32 m + 8 i + 2 c + w holds column
//            32 m + 8 c + 2 i + w), so that a thread's state columns are
//            eight neighbours
//   TH       [bh][chunk] packed tile (tri_line) of (I + A diag(beta))^-1 - I
//   TB       [bh][chunk] packed tile of (I + diag(beta) A)^-1 - I   (training)
//   P        [bh][chunk] packed tile of scale D * Q K^T; the low part in training
//   SC       [bh][chunk][kSc]        per-token factors and tile scales
// Training, kept for the backward:
//   S0       [bh][chunk][Dv][Dk] fp16, one scale per 16 value columns
//   E        [bh][chunk][64][Dv] fp16, likewise (e_t)
// and by the backward's first kernel for its second:
//   dS1, Y   as S0 and E
#pragma once

#include "delta.h"

namespace rnn {

constexpr int kTc = 64;              // tokens a chunk
constexpr int kTri = 80 * 128;       // bytes of a packed triangular tile
// SC: [0,64) e^G, [64,128) e^{G_C - G}, [128,192) beta, [192,256) and from kScGl the
// two parts of G, and the scales between.  The scans read the first kScScan.
enum { kScG = 192, kScK = 256, kScQ, kScTH, kScTB, kScP, kScEnd, kScBu, kScBy, kScBo, kScScan = 268, kScGl = 268, kSc = 332 };

struct DeltaTcBufs {
  void *k16, *q16, *th, *tb, *p;
  float* sc;
  void *s0, *e;                      // training
  float *s0_scale, *e_scale;         // [bh][chunk][Dv/16]
};

struct DeltaTcArgs {
  DeltaArgs a;
  DeltaTcBufs w;
  const float* s_in;
  float* s_out;
  void* o;
  unsigned int* status;              // first rnn_status_t a kernel reports
  int train, num_sms;
};
// Once per device and handle: the kernels' shared memory limits.
int delta_tc_init(int Dk);
bool delta_tc_supported(int Dk, int Dv, int is_bf16);
int launch_delta_tc_forward(const DeltaTcArgs& t, cudaStream_t s, int* launches);

struct DeltaTcBwdArgs {
  DeltaArgs a;
  DeltaTcBufs w;
  const void* dout;
  const float* dsT;
  float* ds0;
  void *ds1, *y;
  float *ds1_scale, *y_scale, *do_scale;   // do_scale: of the fp16 copy of do, made where it is used
  void *dq, *dk, *dv, *dg, *dbeta;
  unsigned int* status;
  int num_sms;
};
int launch_delta_tc_backward(const DeltaTcBwdArgs& t, cudaStream_t s, int* launches);

}  // namespace rnn
