// delta_tc.cu - the gated delta rule by chunks of 64 tokens on tensor cores.
//
// With G the cumulative decay of a chunk (a token's own included),
// D_ij = exp(G_i - G_j) for j <= i, A the strictly lower part of D * K K^T and
// P = scale D * Q K^T (lower part with the diagonal):
//   r = v - e^G S0 k                     e = (I + A diag(beta))^-1 r
//   o = scale e^G S0 q + P (beta e)      S1 = e^{G_C} S0 + sum_j e^{G_C - G_j} beta_j e_j k_j^T
// so one kernel (prep) computes what does not depend on the state, all chunks
// at once, and one (scan) walks the chunks of a head.  Value columns are
// independent: a warp of the scan owns 16 of them and keeps its part of the
// state, S [16][Dk], in the accumulator fragments of mma.m16n8k16.  The
// accumulator fragment of one product is the A operand of the next,
//   S K^T [16][64] -> r -> r T^T [16][64] -> u -> u K [16][Dk] -> S,
// so nothing passes through shared memory or another warp inside a chunk, which
// is what the length of the chain (T / 64 chunks) asks for.
//
// Operands are fp16 scaled by a power of two that brings the largest element of
// the tile (of a warp's 16 rows) to [2^13, 2^14); the scale leaves the product
// in fp32.  bf16 inputs are exact that way (8 of 11 bits; what lies more than
// 2^-29 below the tile's largest element loses bits).  Values computed here are
// split into a high and a low fp16 part, 22 bits, where they reach the state:
// S, r, u and the inverse; the output takes the high part alone, 11 bits where
// its own rounding keeps 8.
#include <cuda_fp16.h>

#include "common.cuh"
#include "delta_tc.h"
#include "pair.cuh"

namespace rnn {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr uint64_t kScanTimeoutNs = 2000000000ull;     // of a wait for a chunk's copies

// --- scales and fragments -----------------------------------------------------
// The power of two that brings m to [2^13, 2^14), and its inverse.  NaN when m is
// an infinity or NaN: the whole tile then shows it, instead of its other values
// losing their bits to a scale of no use.
__device__ __forceinline__ float up_scale(float m) {
  const int e = (__float_as_int(m) >> 23) & 255;
  int f = 267 - e;
  f = f < 1 ? 1 : f > 253 ? 253 : f;
  return __int_as_float(e == 255 ? 0x7fc00000 : f << 23);
}
__device__ __forceinline__ float inv_scale(float f) { return __int_as_float((254 << 23) - __float_as_int(f)); }

// A power of two, at most one, that keeps products with a factor of at most m
// below twice their other factor.
__device__ __forceinline__ float below_inverse(float m) {
  int f = 254 - ((__float_as_int(m) >> 23) & 255);
  f = f < 27 ? 27 : f > 127 ? 127 : f;
  return __int_as_float(f << 23);
}

__device__ __forceinline__ uint32_t pack_h(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack_b(float x, float y) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 unpack_h(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
__device__ __forceinline__ float2 unpack_b(uint32_t v) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}

// Largest of non-negative values over the warp: their bits order as integers.
__device__ __forceinline__ float warp_max(float m) {
  return __uint_as_float(__reduce_max_sync(kFull, __float_as_uint(m)));
}

__device__ __forceinline__ float2 lo2(const float (&x)[4]) { return make_float2(x[0], x[1]); }
__device__ __forceinline__ float2 hi2(const float (&x)[4]) { return make_float2(x[2], x[3]); }
__device__ __forceinline__ void set4(float (&x)[4], float2 lo, float2 hi) {
  x[0] = lo.x; x[1] = lo.y; x[2] = hi.x; x[3] = hi.y;
}

// x = hi + lo to 22 bits.
__device__ __forceinline__ void split(float2 x, uint32_t& hi, uint32_t& lo) {
  hi = pack_h(x.x, x.y);
  const float2 l = fma2(unpack_h(hi), both(-1.f), x);
  lo = pack_h(l.x, l.y);
}
__device__ __forceinline__ uint32_t pack_h(float2 x) { return pack_h(x.x, x.y); }

// D = A B: the first product of a sum.
__device__ __forceinline__ void mma_h0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_h(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_b(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_t(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
__device__ __forceinline__ void ldsm_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr));
}
// Transpose of an 8 x 8 matrix of 16-bit elements held as fragments.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Sixteen bytes, or zeros.
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void* src, bool ok) {
  const int n = ok ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}

// Byte offset of 16-byte piece ``p`` of row ``r`` in a tile of PITCH-byte rows.
template <int PITCH>
__device__ __forceinline__ uint32_t swz(int r, int p) {
  return static_cast<uint32_t>(r * PITCH + ((p ^ (r & 7)) << 4));
}

// B operand of two neighbouring n-tiles (n0, n0 + 8) and one k-step of 16, from
// a tile whose rows are n (k along the row): b[0..1] and b[2..3].
template <int PITCH>
__device__ __forceinline__ void load_b_rows_n(uint32_t (&b)[4], uint32_t tile, int n0, int kk, int lane) {
  ldsm(b, tile + swz<PITCH>(n0 + (lane & 7) + ((lane >> 4) << 3), 2 * kk + ((lane >> 3) & 1)));
}
// The same from a tile whose rows are k (n along the row).
template <int PITCH>
__device__ __forceinline__ void load_b_rows_k(uint32_t (&b)[4], uint32_t tile, int n0, int kk, int lane) {
  ldsm_t(b, tile + swz<PITCH>(16 * kk + (lane & 7) + (((lane >> 3) & 1) << 3), (n0 >> 3) + (lane >> 4)));
}

// The same operands of the scans, which read many of a chunk's tiles: the
// lane's part of the address is computed once, and the rest are constants.  A
// piece index 2 kk + b exchanged by x = lane & 7 is ((2 kk & 7) + b ^ x) with the
// higher bits untouched, so four offsets serve a row of any length.
struct LaneOffsets {
  uint32_t n[2][4], k[2][4];     // of packed tiles, of rows of Dk columns
  // ``first``: the first of the warp's pieces in the rows of Dk columns, 0 or 4 of 8
  __device__ __forceinline__ void init(int dk_pitch, int lane, int first = 0) {
    const int x = lane & 7;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int an = 2 * i + ((lane >> 3) & 1), ak = 2 * i + (lane >> 4);
      const int rn = x + ((lane >> 4) << 3), rk = x + (((lane >> 3) & 1) << 3);
      n[0][i] = rn * 128 + ((an ^ x) << 4);
      n[1][i] = rn * dk_pitch + (((an ^ first) ^ x) << 4);
      k[0][i] = rk * 128 + ((ak ^ x) << 4);
      k[1][i] = rk * dk_pitch + (((ak ^ first) ^ x) << 4);
    }
  }
};
// A lower triangular 64 x 64 tile in two fp16 parts, its ten 16 x 16 blocks (b, kb),
// kb <= b, packed into 80 lines of 128 bytes: block row 1 in lines 16..31 (high |
// low), block row 3 in 48..63 and 64..79, block row 2 in 32..47 with what does
// not fit beside block row 0 in lines 0..15.  A block's rows are 16 lines from
// tri_line, two pieces from tri_piece; pieces are exchanged by (line & 7).  10 KB
// instead of 16 let two scan CTAs of four warps share an SM where Dk is 64.
__host__ __device__ constexpr int tri_line(int b, int kb, int part) {
  return b < 2 ? 16 * b : b == 2 ? (part && kb ? 0 : 32) : 48 + 16 * part;
}
__host__ __device__ constexpr int tri_piece(int b, int kb, int part) {
  return b == 0 ? 2 * part : b == 1 ? 2 * kb + 4 * part : b == 2 ? (part ? (kb ? 2 + 2 * kb : 6) : 2 * kb) : 2 * kb;
}
// rows n: tiles n0, n0 + 8 and k-step kk; rows k likewise (n0 a multiple of 16)
template <int PITCH>
__device__ __forceinline__ void scan_b_n(uint32_t (&b)[4], uint32_t tile, const LaneOffsets& o, int n0, int kk) {
  ldsm(b, tile + o.n[1][kk & 3] + n0 * PITCH + (kk >> 2) * 128);
}
template <int PITCH>
__device__ __forceinline__ void scan_b_k(uint32_t (&b)[4], uint32_t tile, const LaneOffsets& o, int n0, int kk) {
  ldsm_t(b, tile + o.k[1][(n0 >> 4) & 3] + 16 * kk * PITCH + (n0 >> 6) * 128);
}

// The same of a packed triangular tile: block row n0 / 16, k-step kk = its column (rows n), or the reverse (rows k).
__device__ __forceinline__ void scan_tri_n(uint32_t (&b)[4], uint32_t tile, const LaneOffsets& o, int n0, int kk, int part) {
  ldsm(b, tile + o.n[0][tri_piece(n0 >> 4, kk, part) >> 1] + tri_line(n0 >> 4, kk, part) * 128);
}
__device__ __forceinline__ void scan_tri_k(uint32_t (&b)[4], uint32_t tile, const LaneOffsets& o, int n0, int kk, int part) {
  ldsm_t(b, tile + o.k[0][tri_piece(kk, n0 >> 4, part) >> 1] + tri_line(kk, n0 >> 4, part) * 128);
}

// Value column (of a warp's 16) behind row r of its fragments; row r + 8 is two
// further.  A transposed fragment pair then holds four neighbouring columns.
__device__ __forceinline__ int dv_of_row(int r) { return 4 * (r >> 1) + (r & 1); }

// ---------------------------------------------------------------------------
// prep: everything of a chunk that does not depend on the state
// ---------------------------------------------------------------------------
constexpr int kXP = 68;              // pitch of the fp32 64 x 64 matrices: fragment rows on different banks
// C[16][8 NB] = sign cw (A (yw B)) by one warp, on fp32 matrices in shared memory
// (pitch kXP): A [16][8 KB], row k of B weighted by yw[k] and row i of the result
// by cw[i] where given.  Each factor is split into two tf32 parts (11 + 10 bits)
// and the product of the low parts dropped: 2^-21 of the product, whatever the
// scale of the factors.
template <int KB, int NB>
__device__ __forceinline__ void warp_mul(float* C, const float* A, const float* B, const float* yw, const float* cw,
                                         float sign, int lane) {
  const int r = lane >> 2, c = lane & 3;
  float acc[NB][4];
#pragma unroll
  for (int n = 0; n < NB; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[n][e] = 0.f;
#pragma unroll
  for (int k = 0; k < KB; ++k) {
    float x[4];
    x[0] = A[r * kXP + 8 * k + c];
    x[1] = A[(r + 8) * kXP + 8 * k + c];
    x[2] = A[r * kXP + 8 * k + c + 4];
    x[3] = A[(r + 8) * kXP + 8 * k + c + 4];
    uint32_t ah[4], al[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ah[i] = __float_as_uint(x[i]) & 0xffffe000u;
      al[i] = __float_as_uint(x[i] - __uint_as_float(ah[i]));
    }
    const float w0 = yw ? yw[8 * k + c] : 1.f, w1 = yw ? yw[8 * k + c + 4] : 1.f;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const float y0 = w0 * B[(8 * k + c) * kXP + 8 * n + r], y1 = w1 * B[(8 * k + c + 4) * kXP + 8 * n + r];
      const uint32_t b0 = __float_as_uint(y0) & 0xffffe000u, b1 = __float_as_uint(y1) & 0xffffe000u;
      const uint32_t l0 = __float_as_uint(y0 - __uint_as_float(b0)), l1 = __float_as_uint(y1 - __uint_as_float(b1));
      mma_t(acc[n], al, b0, b1);
      mma_t(acc[n], ah, l0, l1);
      mma_t(acc[n], ah, b0, b1);
    }
  }
  const float s0 = sign * (cw ? cw[r] : 1.f), s1 = sign * (cw ? cw[r + 8] : 1.f);
#pragma unroll
  for (int n = 0; n < NB; ++n) {
    *reinterpret_cast<float2*>(C + r * kXP + 8 * n + 2 * c) = make_float2(s0 * acc[n][0], s0 * acc[n][1]);
    *reinterpret_cast<float2*>(C + (r + 8) * kXP + 8 * n + 2 * c) = make_float2(s1 * acc[n][2], s1 * acc[n][3]);
  }
}

template <int DK, bool TRAIN>
struct PrepSmem {
  union {
    struct {
      unsigned char K[kTc * DK * 2], Q[kTc * DK * 2];
    } in;
    struct {                         // once K and Q are multiplied
      float A[kTc * kXP];
      float X[TRAIN ? 2 : 1][kTc * kXP];   // the inverses
    };
  };
  float Gh[kTc], Gl[kTc], beta[kTc];
  float red[4][4];
};

// Largest |X_ij| over the block's threads (each gives its own), for channel ch.
__device__ __forceinline__ float block_max4(float (*red)[4], int ch, float m) {
  m = warp_max(m);
  if ((threadIdx.x & 31) == 0) red[ch][threadIdx.x >> 5] = m;
  __syncthreads();
  return fmaxf(fmaxf(red[ch][0], red[ch][1]), fmaxf(red[ch][2], red[ch][3]));
}

// One CTA of 128 threads per chunk and value head.  K K^T and Q K^T run on the
// tensor cores from the exact bf16 inputs (warp w: rows 16 w .. 16 w + 15, the
// blocks at or below the diagonal).  The unit triangular inverses start from
// 16 x 16 diagonal blocks by substitution in fp32, a thread a column; then blocks
// are joined twice, [[X, 0], [-Y L X, Y]], on the tensor cores.  No power of L
// appears, so keys that are all alike (L with entries near one) cost no accuracy.
// With training, warps 0 and 1 work on (I + A beta)^-1 and 2 and 3 on
// (I + beta A)^-1, else the second half idles in the inverse.
// Bound by latency: short phases between barriers, four to six CTAs an SM.  Chunks
// of D = 128: 4096 in 123 us (training), 8192 in 170 us (inference); joining the
// inverses in fp32 on the CUDA cores took 157 and 245.
template <int DK, bool TRAIN>
__global__ void __launch_bounds__(128, TRAIN ? 4 : 6) delta_prep_kernel(const DeltaTcArgs p) {
  constexpr int PK = DK * 2;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  PrepSmem<DK, TRAIN>& sm = *reinterpret_cast<PrepSmem<DK, TRAIN>*>(smem_raw);
  const DeltaArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nc = (a.T + kTc - 1) / kTc;
  const int64_t bid = blockIdx.x;
  const int c = static_cast<int>(bid % nc), h = static_cast<int>(bid / nc % a.Hv), b = static_cast<int>(bid / nc / a.Hv);
  const int len = a.len ? a.len[b] : a.T;
  const int t0 = c * kTc, nt = len - t0;
  if (nt <= 0) return;
  const int per = a.Hv / a.Hk, hk = h / per;
  const int64_t bhc = (static_cast<int64_t>(b) * a.Hv + h) * nc + c, bkc = (static_cast<int64_t>(b) * a.Hk + hk) * nc + c;
  const uint32_t ks = smem_u32(sm.in.K), qs = smem_u32(sm.in.Q);

  constexpr int PR = DK / 8, STEP = 128 / PR;         // pieces of a row; rows between a thread's pieces
  const int pt = tid / PR, pch = tid % PR;
  {
    const int64_t row0 = a.row(b, t0), tstep = a.bfirst ? 1 : a.B;
    const __nv_bfloat16 *kp = static_cast<const __nv_bfloat16*>(a.k) + row0 * a.k_row + hk * DK + pch * 8,
                        *qp = static_cast<const __nv_bfloat16*>(a.q) + row0 * a.q_row + hk * DK + pch * 8;
#pragma unroll
    for (int i = 0; i < kTc / STEP; ++i) {
      const int t = pt + i * STEP;
      const bool ok = t < nt;
      const int64_t dt = ok ? t * tstep : 0;
      cp16_or_zero(ks + swz<PK>(t, pch), kp + dt * a.k_row, ok);
      cp16_or_zero(qs + swz<PK>(t, pch), qp + dt * a.q_row, ok);
    }
  }
  cp_commit();
  // cumulative decay in two floats: D_ij stays exact to fp32 however large G
  float* sc = p.w.sc + bhc * kSc;
  if (warp == 0) {
    TwoF g2[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      const bool ok = t < nt;
      const int64_t row = a.row(b, t0 + (ok ? t : 0));
      float g = ok ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.g)[row * a.g_row + h]) : 0.f;
      g2[i] = {g < kDecayFloor ? kDecayFloor : g, 0.f};
      const float be = ok ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.beta)[row * a.beta_row + h]) : 0.f;
      sm.beta[t] = be;
      sc[128 + t] = be;
    }
    TwoF pair = two_add(g2[0], g2[1]);
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
      const TwoF up = {__shfl_up_sync(kFull, pair.h, w), __shfl_up_sync(kFull, pair.l, w)};
      if (lane >= w) pair = two_add(up, pair);
    }
    TwoF before = {__shfl_up_sync(kFull, pair.h, 1), __shfl_up_sync(kFull, pair.l, 1)};
    if (lane == 0) before = {0.f, 0.f};
    const TwoF end = {__shfl_sync(kFull, pair.h, 31), __shfl_sync(kFull, pair.l, 31)};
    g2[0] = two_add(before, g2[0]);
    g2[1] = pair;
    float bu = 0.f, by = 0.f, bo = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t = 2 * lane + i;
      sm.Gh[t] = g2[i].h;
      sm.Gl[t] = g2[i].l;
      const float eg = expf(g2[i].h + g2[i].l), ee = expf((end.h - g2[i].h) + (end.l - g2[i].l));
      const float be = fabsf(sm.beta[t]);
      sc[t] = eg;
      sc[64 + t] = ee;
      sc[kScG + t] = g2[i].h;
      sc[kScGl + t] = g2[i].l;
      bu = fmaxf(bu, be * fmaxf(1.f, ee));
      by = fmaxf(by, be * eg);
      bo = fmaxf(bo, fabsf(a.scale) * eg);
    }
    bu = warp_max(bu);
    by = warp_max(by);
    bo = warp_max(bo);
    if (lane == 0) {
      sc[kScEnd] = expf(end.h + end.l);
      sc[kScBu] = below_inverse(bu);
      sc[kScBy] = below_inverse(by);
      sc[kScBo] = below_inverse(bo);
    }
  }
  cp_wait<0>();
  __syncthreads();

  // scales of the key and query tiles, and their fp16 copies (one head of a group writes)
  float km, qm;
  {
    // bf16 magnitudes order as 16-bit integers, two at a time
    uint32_t kx = 0, qx = 0;
#pragma unroll
    for (int i = 0; i < kTc / STEP; ++i) {
      const uint4 u = *reinterpret_cast<const uint4*>(sm.in.K + (tid + i * 128) * 16), w = *reinterpret_cast<const uint4*>(sm.in.Q + (tid + i * 128) * 16);
      kx = __vmaxu2(__vmaxu2(kx, __vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu)), __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
      qx = __vmaxu2(__vmaxu2(qx, __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu)), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
    }
    km = warp_max(__uint_as_float(max(kx >> 16, kx & 0xffffu) << 16));
    qm = warp_max(__uint_as_float(max(qx >> 16, qx & 0xffffu) << 16));
  }
  if (lane == 0) {
    sm.red[0][warp] = km;
    sm.red[1][warp] = qm;
  }
  __syncthreads();
  const float kf = up_scale(fmaxf(fmaxf(sm.red[0][0], sm.red[0][1]), fmaxf(sm.red[0][2], sm.red[0][3])));
  const float qf = up_scale(fmaxf(fmaxf(sm.red[1][0], sm.red[1][1]), fmaxf(sm.red[1][2], sm.red[1][3])));
  if (tid == 0) {
    sc[kScK] = inv_scale(kf);
    sc[kScQ] = inv_scale(qf);
  }
  if (h % per == 0) {
    unsigned char* ko = static_cast<unsigned char*>(p.w.k16) + bkc * kTc * PK;
    unsigned char* qo = static_cast<unsigned char*>(p.w.q16) + bkc * kTc * PK;
    // piece 4 m + i of the permuted row holds words i of pieces 4 m .. 4 m + 3
    auto permute = [&](const unsigned char* in, unsigned char* out, float f, int t, int m) {
      uint4 w[4];
#pragma unroll
      for (int c4 = 0; c4 < 4; ++c4) w[c4] = *reinterpret_cast<const uint4*>(in + swz<PK>(t, 4 * m + c4));
      auto half2_of = [&](uint32_t v) { return pack_h(mul2(unpack_b(v), both(f))); };
      *reinterpret_cast<uint4*>(out + swz<PK>(t, 4 * m)) = make_uint4(half2_of(w[0].x), half2_of(w[1].x), half2_of(w[2].x), half2_of(w[3].x));
      *reinterpret_cast<uint4*>(out + swz<PK>(t, 4 * m + 1)) = make_uint4(half2_of(w[0].y), half2_of(w[1].y), half2_of(w[2].y), half2_of(w[3].y));
      *reinterpret_cast<uint4*>(out + swz<PK>(t, 4 * m + 2)) = make_uint4(half2_of(w[0].z), half2_of(w[1].z), half2_of(w[2].z), half2_of(w[3].z));
      *reinterpret_cast<uint4*>(out + swz<PK>(t, 4 * m + 3)) = make_uint4(half2_of(w[0].w), half2_of(w[1].w), half2_of(w[2].w), half2_of(w[3].w));
    };
    constexpr int MR = DK / 32;
#pragma unroll
    for (int i = 0; i < kTc * MR / 128; ++i) {
      const int t = (tid + i * 128) / MR, m = (tid + i * 128) % MR;
      permute(sm.in.K, ko, kf, t, m);
      permute(sm.in.Q, qo, qf, t, m);
    }
  }

  // K K^T and Q K^T
  float kk[8][4], qk[8][4];
#pragma unroll
  for (int n = 0; n < 8; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) kk[n][i] = qk[n][i] = 0.f;
#pragma unroll
  for (int s = 0; s < DK / 16; ++s) {
    uint32_t ak[4], aq[4];
    const uint32_t at = swz<PK>(16 * warp + (lane & 15), 2 * s + (lane >> 4));
    ldsm(ak, ks + at);
    ldsm(aq, qs + at);
#pragma unroll
    for (int n = 0; n < 8; n += 2) {
      if (n > 2 * warp) continue;
      uint32_t bb[4];
      load_b_rows_n<PK>(bb, ks, 8 * n, s, lane);
      mma_b(kk[n], ak, bb[0], bb[1]);
      mma_b(kk[n + 1], ak, bb[2], bb[3]);
      mma_b(qk[n], aq, bb[0], bb[1]);
      mma_b(qk[n + 1], aq, bb[2], bb[3]);
    }
  }
  __syncthreads();                    // K and Q are read: X may take their place
  float pm = 0.f;
  const int r = lane >> 2, cc = 2 * (lane & 3);
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    if (n > 2 * warp + 1) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 16 * warp + r + (e >> 1) * 8, j = 8 * n + cc + (e & 1);
      const float d = j <= i ? __expf((sm.Gh[i] - sm.Gh[j]) + (sm.Gl[i] - sm.Gl[j])) : 0.f;
      sm.A[i * kXP + j] = j < i ? d * kk[n][e] : 0.f;
      qk[n][e] = j <= i ? a.scale * d * qk[n][e] : 0.f;
      pm = fmaxf(pm, fabsf(qk[n][e]));
    }
  }
  const float pf = up_scale(block_max4(sm.red, 2, pm));
  if (tid == 0) sc[kScP] = inv_scale(pf);
  unsigned char* po = static_cast<unsigned char*>(p.w.p) + bhc * kTri;
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    if (n > 2 * warp + 1) continue;
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const int i = 16 * warp + r + (e >> 1) * 8;
      uint32_t hi, lo;
      split(make_float2(qk[n][e] * pf, qk[n][e + 1] * pf), hi, lo);
      auto at = [&](int part) {
        return swz<128>(tri_line(warp, n >> 1, part) + (i & 15), tri_piece(warp, n >> 1, part) + (n & 1)) + 2 * cc;
      };
      *reinterpret_cast<uint32_t*>(po + at(0)) = hi;
      if (TRAIN) *reinterpret_cast<uint32_t*>(po + at(1)) = lo;
    }
  }

  // the inverses: which = 0: L_ij = A_ij beta_j, which = 1: L_ij = beta_i A_ij
  const int which = tid >> 6, col = tid & 63;
  const bool mine = TRAIN || which == 0;
  float* X = sm.X[TRAIN ? which : 0];
  if (mine) {
    const int b0 = col & ~15, jc = col & 15;
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int j = 0; j < i; ++j) {
        // which = 0: y_j = beta_j x_j is kept; which = 1: the row's beta after the sum
        s0 = j & 1 ? s0 : fmaf(-sm.A[(b0 + i) * kXP + b0 + j], x[j], s0);
        s1 = j & 1 ? fmaf(-sm.A[(b0 + i) * kXP + b0 + j], x[j], s1) : s1;
      }
      const float bi = sm.beta[b0 + i];
      const float one = i == jc ? 1.f : 0.f;
      const float v = i < jc ? 0.f : which ? fmaf(bi, s0 + s1, one) : s0 + s1 + one;
      x[i] = which ? v : bi * v;
      X[(b0 + i) * kXP + col] = v;
    }
  }
  __syncthreads();
  // Two of 16 make one of 32: a warp a pair.  The product L X waits in the block
  // above the diagonal, which is zeroed again for the next join.
  const int t64 = tid & 63, half = warp & 1;
  if (mine) {
    const int o = 32 * half;
    float* above = X + o * kXP + o + 16;
    warp_mul<2, 2>(above, sm.A + (o + 16) * kXP + o, X + o * kXP + o, which ? nullptr : sm.beta + o,
                   which ? sm.beta + o + 16 : nullptr, 1.f, lane);
    __syncwarp();
    warp_mul<2, 2>(X + (o + 16) * kXP + o, X + (o + 16) * kXP + o + 16, above, nullptr, nullptr, -1.f, lane);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 2; ++i)
      *reinterpret_cast<float4*>(above + (lane >> 2) * kXP + 8 * i * kXP + 4 * (lane & 3)) = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __syncthreads();
  // two of 32 make the whole: a warp 16 rows
  if (mine)
    warp_mul<4, 4>(X + 16 * half * kXP + 32, sm.A + (32 + 16 * half) * kXP, X, which ? nullptr : sm.beta,
                   which ? sm.beta + 32 + 16 * half : nullptr, 1.f, lane);
  __syncthreads();
  if (mine)
    warp_mul<4, 4>(X + (32 + 16 * half) * kXP, X + (32 + 16 * half) * kXP + 32, X + 32, nullptr, nullptr, -1.f, lane);
  __syncthreads();
  // strictly lower part, high and low: the diagonal goes, the blocks above it are not read
  if (mine) X[t64 * (kXP + 1)] = 0.f;
  __syncthreads();
  // piece ch of rows i, i + 8, ..: rows of 16-block i / 16 have 2 (i / 16) + 2 pieces
  const int wi = t64 >> 3, wch = t64 & 7;
  float xm = 0.f;
  if (mine) {
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      if (wch > (n | 1)) continue;
      const float4 u = *reinterpret_cast<const float4*>(X + (wi + 8 * n) * kXP + 8 * wch), w = *reinterpret_cast<const float4*>(X + (wi + 8 * n) * kXP + 8 * wch + 4);
      xm = fmaxf(xm, fmaxf(fmaxf(fmaxf(fabsf(u.x), fabsf(u.y)), fmaxf(fabsf(u.z), fabsf(u.w))),
                           fmaxf(fmaxf(fabsf(w.x), fabsf(w.y)), fmaxf(fabsf(w.z), fabsf(w.w)))));
    }
  }
  xm = warp_max(xm);
  if (lane == 0) sm.red[3][warp] = xm;
  __syncthreads();
  if (!mine) return;
  const float xf = up_scale(fmaxf(sm.red[3][2 * which], sm.red[3][2 * which + 1]));
  if (t64 == 0) sc[which ? kScTB : kScTH] = inv_scale(xf);
  unsigned char* xo = static_cast<unsigned char*>(which ? p.w.tb : p.w.th) + bhc * kTri;
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    if (wch > (n | 1)) continue;
    const float4 u = *reinterpret_cast<const float4*>(X + (wi + 8 * n) * kXP + 8 * wch), w = *reinterpret_cast<const float4*>(X + (wi + 8 * n) * kXP + 8 * wch + 4);
    uint4 hi, lo;
    split(mul2(make_float2(u.x, u.y), both(xf)), hi.x, lo.x);
    split(mul2(make_float2(u.z, u.w), both(xf)), hi.y, lo.y);
    split(mul2(make_float2(w.x, w.y), both(xf)), hi.z, lo.z);
    split(mul2(make_float2(w.z, w.w), both(xf)), hi.w, lo.w);
    auto at = [&](int part) {
      return swz<128>(tri_line(n >> 1, wch >> 1, part) + wi + 8 * (n & 1), tri_piece(n >> 1, wch >> 1, part) + (wch & 1));
    };
    *reinterpret_cast<uint4*>(xo + at(0)) = hi;
    *reinterpret_cast<uint4*>(xo + at(1)) = lo;
  }
}

// ---------------------------------------------------------------------------
// pieces of the scans
// ---------------------------------------------------------------------------
// A thread's part of a state: tile j holds, for rows r and r + 8 of the warp's
// 16 value columns, the state columns behind positions 8 j + 2 (lane & 3).
template <int DK>
struct State {
  float v[DK / 8][4];
};

// fp32 state rows <-> fragments: 8 neighbouring columns a thread, row and m.
template <int DKW>
__device__ __forceinline__ void state_load(State<DKW>& S, const float* base, int pitch, int lane) {
  const int r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const float* p = base + (dv_of_row(r) + 2 * half) * pitch + 8 * c;
#pragma unroll
    for (int m = 0; m < DKW / 32; ++m) {
      const float4 x = *reinterpret_cast<const float4*>(p + 32 * m), y = *reinterpret_cast<const float4*>(p + 32 * m + 4);
      S.v[4 * m][2 * half] = x.x; S.v[4 * m][2 * half + 1] = x.y;
      S.v[4 * m + 1][2 * half] = x.z; S.v[4 * m + 1][2 * half + 1] = x.w;
      S.v[4 * m + 2][2 * half] = y.x; S.v[4 * m + 2][2 * half + 1] = y.y;
      S.v[4 * m + 3][2 * half] = y.z; S.v[4 * m + 3][2 * half + 1] = y.w;
    }
  }
}
template <int DKW>
__device__ __forceinline__ void state_store(const State<DKW>& S, float* base, int pitch, int lane) {
  const int r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float* p = base + (dv_of_row(r) + 2 * half) * pitch + 8 * c;
#pragma unroll
    for (int m = 0; m < DKW / 32; ++m) {
      *reinterpret_cast<float4*>(p + 32 * m) = make_float4(S.v[4 * m][2 * half], S.v[4 * m][2 * half + 1],
                                                           S.v[4 * m + 1][2 * half], S.v[4 * m + 1][2 * half + 1]);
      *reinterpret_cast<float4*>(p + 32 * m + 4) = make_float4(S.v[4 * m + 2][2 * half], S.v[4 * m + 2][2 * half + 1],
                                                               S.v[4 * m + 3][2 * half], S.v[4 * m + 3][2 * half + 1]);
    }
  }
}
template <int DK>
__device__ __forceinline__ float state_max(const State<DK>& S) {      // over the warp
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < DK / 8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(S.v[j][i]));
  return warp_max(m);
}
// fp16 copy of the state, scaled by f.
template <int DKW>
__device__ __forceinline__ void state_store_half(const State<DKW>& S, float f, __half* base, int pitch, int lane) {
  const int r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    __half* p = base + (dv_of_row(r) + 2 * half) * pitch + 8 * c;
#pragma unroll
    for (int m = 0; m < DKW / 32; ++m) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = pack_h(mul2(half ? hi2(S.v[4 * m + i]) : lo2(S.v[4 * m + i]), both(f)));
      *reinterpret_cast<uint4*>(p + 32 * m) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// X[8][4] is [16 value columns][64 tokens] as accumulator tiles over tokens.
using Frag = float[8][4];
__device__ __forceinline__ float frag_max(const Frag& x) {
  float m = 0.f;
#pragma unroll
  for (int n = 0; n < 8; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, fabsf(x[n][i]));
  return warp_max(m);
}
// x[.][t] *= w[t] for per-token factors in shared memory, times f.
__device__ __forceinline__ float2 pair_of(const float* p, int n, int lane) {
  return *reinterpret_cast<const float2*>(p + 8 * n + 2 * (lane & 3));
}
__device__ __forceinline__ void frag_scale(Frag& x, const float* w, int lane) {
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    const float2 f = pair_of(w, n, lane);
    set4(x[n], mul2(lo2(x[n]), f), mul2(hi2(x[n]), f));
  }
}
// x += f y
__device__ __forceinline__ void frag_add(Frag& x, const Frag& y, float f) {
#pragma unroll
  for (int n = 0; n < 8; ++n) set4(x[n], fma2(lo2(y[n]), both(f), lo2(x[n])), fma2(hi2(y[n]), both(f), hi2(x[n])));
}
// A operand (k = tokens 16 kk ..) of a fragment scaled by f, high and low part.
__device__ __forceinline__ void frag_a(const Frag& x, int kk, float f, uint32_t (&hi)[4], uint32_t (&lo)[4]) {
  split(mul2(lo2(x[2 * kk]), both(f)), hi[0], lo[0]);
  split(mul2(hi2(x[2 * kk]), both(f)), hi[1], lo[1]);
  split(mul2(lo2(x[2 * kk + 1]), both(f)), hi[2], lo[2]);
  split(mul2(hi2(x[2 * kk + 1]), both(f)), hi[3], lo[3]);
}
__device__ __forceinline__ void frag_a_hi(const Frag& x, int kk, float f, uint32_t (&hi)[4]) {
  hi[0] = pack_h(mul2(lo2(x[2 * kk]), both(f)));
  hi[1] = pack_h(mul2(hi2(x[2 * kk]), both(f)));
  hi[2] = pack_h(mul2(lo2(x[2 * kk + 1]), both(f)));
  hi[3] = pack_h(mul2(hi2(x[2 * kk + 1]), both(f)));
}

// A warp's [64 tokens][16 columns] slice of a chunk of a bf16 sequence: thread
// (lane / 4, lane % 4) of tile n holds token 8 n + lane / 4, columns 4 (lane % 4)
// .. + 3 (the columns of fragment rows 2 c, 2 c + 1 and 8 + 2 c, 9 + 2 c).
struct Slice {
  uint2 v[8];
};
// Rows of W slices in shared memory, 32 bytes further apart than they are long:
// the four rows that half a warp reads at a time fall on different banks.
template <int W>
struct SeqTile {
  static constexpr int PITCH = 32 * W + 32;
  unsigned char row[kTc][PITCH];
};
template <int W>
__device__ __forceinline__ void slice_load(Slice& s, const SeqTile<W>& t, int warp, int lane) {
  const unsigned char* p = t.row[lane >> 2] + 32 * warp + 8 * (lane & 3);
#pragma unroll
  for (int n = 0; n < 8; ++n) s.v[n] = *reinterpret_cast<const uint2*>(p + 8 * n * SeqTile<W>::PITCH);
}
// Fragment tile n (fp32) of a slice.
__device__ __forceinline__ void slice_frag(const Slice& s, int n, float2& lo, float2& hi) {
  lo = unpack_b(transpose8(s.v[n].x));
  hi = unpack_b(transpose8(s.v[n].y));
}

// A chunk's tiles arrive by bulk copies that one thread issues and an mbarrier
// counts, its rows of a sequence by one 16-byte copy in four a thread: loads into
// registers, with the few scoreboards a warp has, would hold up the shared memory
// reads issued after them.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :: "r"(dst), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}
// What one chunk of a scan reads: the tiles of prep and W slices of a sequence.
template <int DK, int W>
struct ScanStage {
  unsigned char K[kTc * DK * 2], Q[kTc * DK * 2], T[kTri], P[kTri];
  float sc[kScScan];
  SeqTile<W> x;
};
template <int DK, int W>
struct alignas(128) ScanSmem {
  ScanStage<DK, W> st[2];
  uint64_t full[2];
  float smax[2][W];                  // of the warps' states, by turn
};
struct ScanSource {
  const char *k, *q, *t, *p, *sc;        // of chunk 0
  const __nv_bfloat16* x;                // this thread's piece of the first 16 tokens
  int64_t x_step;                        // elements 16 tokens further
};
// By every thread, once all have left the stage.  ``left`` tokens of the sequence
// start here; rows beyond them are zeros.
template <int DK, int W>
__device__ __forceinline__ void scan_fetch(ScanStage<DK, W>& st, uint64_t* bar, const ScanSource& src, int c, int left) {
  if (threadIdx.x == 0) {
    fence_proxy_async_smem();
    mbar_arrive_expect_tx(bar, 2 * kTc * DK * 2 + 2 * kTri + kScScan * 4);
    bulk_copy(smem_u32(st.K), src.k + static_cast<int64_t>(c) * kTc * DK * 2, kTc * DK * 2, bar);
    bulk_copy(smem_u32(st.Q), src.q + static_cast<int64_t>(c) * kTc * DK * 2, kTc * DK * 2, bar);
    bulk_copy(smem_u32(st.T), src.t + static_cast<int64_t>(c) * kTri, kTri, bar);
    bulk_copy(smem_u32(st.P), src.p + static_cast<int64_t>(c) * kTri, kTri, bar);
    bulk_copy(smem_u32(st.sc), src.sc + static_cast<int64_t>(c) * kSc * 4, kScScan * 4, bar);
  }
  const int t = threadIdx.x / (2 * W), ch = threadIdx.x % (2 * W);
  const __nv_bfloat16* x = src.x + 4 * c * src.x_step;
  const uint32_t dst = smem_u32(st.x.row[t]) + 16 * ch;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool ok = t + 16 * i < left;
    cp16_or_zero(dst + i * 16 * SeqTile<W>::PITCH, x + (ok ? i * src.x_step : 0), ok);
  }
  cp_commit();
}
// Waits for turn ``it`` of a scan; true when it did not come in time, for every
// thread of the CTA.  Nobody reads the other stage any more then.
__device__ __forceinline__ bool scan_arrive(uint64_t* full, int it, unsigned int* status) {
  cp_wait<0>();
  const bool late = !mbar_wait(&full[it & 1], (it >> 1) & 1, kScanTimeoutNs);
  if (!__syncthreads_or(late)) return false;
  // a copy that is still under way keeps the CTA for as long again
  if (threadIdx.x == 0) {
    atomicCAS(status, 0u, static_cast<unsigned int>(RNN_TIMEOUT));
    mbar_wait(&full[it & 1], (it >> 1) & 1, kScanTimeoutNs);
  }
  return true;
}

// Z = S X^T over the key columns, X = K16 ([16][64 tokens]), from both parts of
// S; with BOTH also Z2 = S X2^T, X2 = Q16, from the high part.
template <int DK, bool BOTH, int DKW>
__device__ __forceinline__ void state_times(const State<DKW>& S, float f, uint32_t x, uint32_t x2, Frag& z, Frag& z2,
                                            const LaneOffsets& lo_) {
#pragma unroll
  for (int kk = 0; kk < DKW / 16; ++kk) {
    uint32_t hi[4], lo[4];
    split(mul2(lo2(S.v[2 * kk]), both(f)), hi[0], lo[0]);
    split(mul2(hi2(S.v[2 * kk]), both(f)), hi[1], lo[1]);
    split(mul2(lo2(S.v[2 * kk + 1]), both(f)), hi[2], lo[2]);
    split(mul2(hi2(S.v[2 * kk + 1]), both(f)), hi[3], lo[3]);
#pragma unroll
    for (int n = 0; n < 8; n += 2) {
      uint32_t bb[4];
      scan_b_n<DK * 2>(bb, x, lo_, 8 * n, kk);
      if (kk == 0) {
        mma_h0(z[n], hi, bb[0], bb[1]);
        mma_h0(z[n + 1], hi, bb[2], bb[3]);
      } else {
        mma_h(z[n], hi, bb[0], bb[1]);
        mma_h(z[n + 1], hi, bb[2], bb[3]);
      }
      mma_h(z[n], lo, bb[0], bb[1]);
      mma_h(z[n + 1], lo, bb[2], bb[3]);
      if (BOTH) {
        scan_b_n<DK * 2>(bb, x2, lo_, 8 * n, kk);
        if (kk == 0) {
          mma_h0(z2[n], hi, bb[0], bb[1]);
          mma_h0(z2[n + 1], hi, bb[2], bb[3]);
        } else {
          mma_h(z2[n], hi, bb[0], bb[1]);
          mma_h(z2[n + 1], hi, bb[2], bb[3]);
        }
      }
    }
  }
}

// S = decay S + sum_t X[.][t] B[t][.], with X scaled by f and B a tile of 64
// tokens; ``g`` undoes the scales.
template <int DK, int DKW>
__device__ __forceinline__ void state_update(State<DKW>& S, float decay, const Frag& x, float f, uint32_t tile, float g,
                                             const LaneOffsets& lo_) {
  uint32_t hi[4][4], lo[4][4];
#pragma unroll
  for (int kk = 0; kk < 4; ++kk) frag_a(x, kk, f, hi[kk], lo[kk]);
#pragma unroll
  for (int j = 0; j < DKW / 8; j += 4) {
    float acc[4][4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        uint32_t bb[4];
        scan_b_k<DK * 2>(bb, tile, lo_, 8 * (j + i), kk);
        if (kk == 0) {
          mma_h0(acc[i], hi[kk], bb[0], bb[1]);
          mma_h0(acc[i + 1], hi[kk], bb[2], bb[3]);
        } else {
          mma_h(acc[i], hi[kk], bb[0], bb[1]);
          mma_h(acc[i + 1], hi[kk], bb[2], bb[3]);
        }
        mma_h(acc[i], lo[kk], bb[0], bb[1]);
        mma_h(acc[i + 1], lo[kk], bb[2], bb[3]);
      }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      set4(S.v[j + i], fma2(lo2(acc[i]), both(g), mul2(lo2(S.v[j + i]), both(decay))),
           fma2(hi2(acc[i]), both(g), mul2(hi2(S.v[j + i]), both(decay))));
  }
}

// Writes a fragment as fp16 rows [64][Dv] scaled by f (a warp's 16 columns).
__device__ __forceinline__ void frag_store_half(const Frag& x, float f, __half* base, int pitch, int lane) {
  __half* p = base + (lane >> 2) * pitch + 4 * (lane & 3);
#pragma unroll
  for (int n = 0; n < 8; ++n)
    *reinterpret_cast<uint2*>(p + 8 * n * pitch) =
        make_uint2(transpose8(pack_h(mul2(lo2(x[n]), both(f)))), transpose8(pack_h(mul2(hi2(x[n]), both(f)))));
}
// Writes a fragment to a dense bf16 sequence: ``p`` points at the thread's columns
// of the chunk's token lane / 4, ``step`` elements lead 8 tokens further, and
// ``left`` tokens of the sequence start here.
__device__ __forceinline__ void frag_store_seq(const Frag& x, __nv_bfloat16* p, int64_t step, int left, int lane) {
  const int t = lane >> 2;
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    const uint32_t lo = transpose8(pack_b(x[n][0], x[n][1])), hi = transpose8(pack_b(x[n][2], x[n][3]));
    if (t + 8 * n < left) *reinterpret_cast<uint2*>(p + n * step) = make_uint2(lo, hi);
  }
}
// Zero rows len .. T-1 of a warp's columns.  The last chunk has written its own
// masked rows already, but not always zeros: a NaN in a token, or an infinity in
// the state, reaches them as a product with zero.  The thread that wrote an
// element there (of a warp that owns whole chunks) writes it again.
__device__ __forceinline__ void zero_rows(__nv_bfloat16* base, const DeltaArgs& a, int64_t stride, int b, int len, int lane) {
  for (int t = (len & ~7) + (lane >> 2); t < a.T; t += 8)
    if (t >= len) *reinterpret_cast<uint2*>(base + a.row(b, t) * stride + 4 * (lane & 3)) = make_uint2(0u, 0u);
}

// ---------------------------------------------------------------------------
// the forward scan
// ---------------------------------------------------------------------------
// W warps of one value head, 16 value columns each.  A chunk of D = 128 is 400
// products m16n8k16 a warp, 8.2 cycles each on a scheduler: 1.7 us of the 3.25
// (W = 4, inference); with two warps a scheduler (W = 8) 3.5 of 5.4.  The rest is
// the chain of scaling and splitting between dependent products.
template <int DK, bool TRAIN, int W>
__global__ void __launch_bounds__(32 * W) delta_scan_fwd_kernel(const DeltaTcArgs p) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  ScanSmem<DK, W>& sm = *reinterpret_cast<ScanSmem<DK, W>*>(smem_raw);
  const DeltaArgs& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = a.Dv / (16 * W);
  const int64_t bid = blockIdx.x;
  const int grp = static_cast<int>(bid % groups), h = static_cast<int>(bid / groups % a.Hv),
            b = static_cast<int>(bid / groups / a.Hv);
  const int slice = grp * W + warp, dv0 = slice * 16;
  const int hk = h / (a.Hv / a.Hk);
  const int len = a.len ? a.len[b] : a.T;
  const int nc = (a.T + kTc - 1) / kTc, ncb = (len + kTc - 1) / kTc;
  const int64_t bh = static_cast<int64_t>(b) * a.Hv + h, bk = static_cast<int64_t>(b) * a.Hk + hk;
  const int64_t o_row = static_cast<int64_t>(a.Hv) * a.Dv;
  const int64_t s_off = (bh * a.Dv + dv0) * DK;
  const int64_t ts_ = a.bfirst ? 1 : a.B;           // rows from token to token
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + static_cast<int64_t>(h) * a.Dv + dv0;
  const int64_t o_step = 8 * ts_ * o_row;
  __nv_bfloat16* ow = o + a.row(b, lane >> 2) * o_row + 4 * (lane & 3);
  LaneOffsets off;
  off.init(DK * 2, lane);
  ScanSource src;
  src.k = static_cast<const char*>(p.w.k16) + bk * nc * kTc * DK * 2;
  src.q = static_cast<const char*>(p.w.q16) + bk * nc * kTc * DK * 2;
  src.t = static_cast<const char*>(p.w.th) + bh * nc * kTri;
  src.p = static_cast<const char*>(p.w.p) + bh * nc * kTri;
  src.sc = reinterpret_cast<const char*>(p.w.sc) + bh * nc * kSc * 4;
  src.x = static_cast<const __nv_bfloat16*>(a.v) + a.row(b, threadIdx.x / (2 * W)) * a.v_row + static_cast<int64_t>(h) * a.Dv +
          grp * 16 * W + 8 * (threadIdx.x % (2 * W));
  src.x_step = 16 * ts_ * a.v_row;

  if (threadIdx.x == 0) {
    mbar_init(&sm.full[0], 1);
    mbar_init(&sm.full[1], 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (ncb > 0) scan_fetch<DK, W>(sm.st[0], &sm.full[0], src, 0, len);
  State<DK> S;
  if (p.s_in) {
    state_load<DK>(S, p.s_in + s_off, DK, lane);
  } else {
#pragma unroll
    for (int j = 0; j < DK / 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) S.v[j][i] = 0.f;
  }
  for (int c = 0; c < ncb; ++c) {
    // one scale for the states of the CTA: their copies then need none of their own in the gradients
    const float own_max = state_max<DK>(S);
    if (lane == 0) sm.smax[c & 1][warp] = own_max;
    if (scan_arrive(sm.full, c, p.status)) return;
    float smax = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) smax = fmaxf(smax, sm.smax[c & 1][w]);
    if (c + 1 < ncb) scan_fetch<DK, W>(sm.st[(c + 1) & 1], &sm.full[(c + 1) & 1], src, c + 1, len - (c + 1) * kTc);
    const ScanStage<DK, W>& s = sm.st[c & 1];
    const uint32_t ks = smem_u32(s.K), qs = smem_u32(s.Q), ts = smem_u32(s.T), ps = smem_u32(s.P);

    const float sf = up_scale(smax), si = inv_scale(sf);
    if (TRAIN) {
      state_store_half<DK>(S, sf, static_cast<__half*>(p.w.s0) + ((bh * nc + c) * a.Dv + dv0) * DK, DK, lane);
      if (lane == 0) p.w.s0_scale[(bh * nc + c) * (a.Dv / 16) + slice] = si;
    }
    Frag z, oq, acc;
    state_times<DK, true>(S, sf, ks, qs, z, oq, off);
    // r = v - e^G S0 k
    const float zk = -si * s.sc[kScK], zq = si * s.sc[kScQ] * a.scale;
    Slice vs;
    slice_load<W>(vs, s.x, warp, lane);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const float2 eg = pair_of(s.sc, n, lane), ek = mul2(eg, both(zk)), eq = mul2(eg, both(zq));
      float2 lo, hi;
      slice_frag(vs, n, lo, hi);
      set4(z[n], fma2(lo2(z[n]), ek, lo), fma2(hi2(z[n]), ek, hi));
      set4(oq[n], mul2(lo2(oq[n]), eq), mul2(hi2(oq[n]), eq));
    }
    // e = r + (T - I) r: the identity stays in fp32
    const float rf = up_scale(frag_max(z));
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      uint32_t hi[4], lo[4];
      frag_a(z, kk, rf, hi, lo);
#pragma unroll
      for (int n = 2 * kk; n < 8; n += 2) {     // j <= i
        uint32_t bh_[4], bl_[4];
        scan_tri_n(bh_, ts, off, 8 * n, kk, 0);
        scan_tri_n(bl_, ts, off, 8 * n, kk, 1);
        if (kk == 0) {
          mma_h0(acc[n], hi, bh_[0], bh_[1]);
          mma_h0(acc[n + 1], hi, bh_[2], bh_[3]);
        } else {
          mma_h(acc[n], hi, bh_[0], bh_[1]);
          mma_h(acc[n + 1], hi, bh_[2], bh_[3]);
        }
        mma_h(acc[n], lo, bh_[0], bh_[1]);
        mma_h(acc[n + 1], lo, bh_[2], bh_[3]);
        mma_h(acc[n], hi, bl_[0], bl_[1]);
        mma_h(acc[n + 1], hi, bl_[2], bl_[3]);
      }
    }
    frag_add(z, acc, inv_scale(rf) * s.sc[kScTH]);
    const float ef = up_scale(frag_max(z));
    if (TRAIN) {
      frag_store_half(z, ef, static_cast<__half*>(p.w.e) + (bh * nc + c) * kTc * a.Dv + dv0, a.Dv, lane);
      if (lane == 0) p.w.e_scale[(bh * nc + c) * (a.Dv / 16) + slice] = inv_scale(ef);
    }
    // u = beta e; o = scale e^G S0 q + P u.  The scale of e times a bound on the
    // weights (kScBu) serves u and e^{G_C - G} u.
    const float uf = ef * s.sc[kScBu], ui = inv_scale(uf);
    frag_scale(z, s.sc + 128, lane);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      uint32_t hi[4];
      frag_a_hi(z, kk, uf, hi);
#pragma unroll
      for (int n = 2 * kk; n < 8; n += 2) {
        uint32_t bb[4];
        scan_tri_n(bb, ps, off, 8 * n, kk, 0);
        if (kk == 0) {
          mma_h0(acc[n], hi, bb[0], bb[1]);
          mma_h0(acc[n + 1], hi, bb[2], bb[3]);
        } else {
          mma_h(acc[n], hi, bb[0], bb[1]);
          mma_h(acc[n + 1], hi, bb[2], bb[3]);
        }
      }
    }
    frag_add(oq, acc, ui * s.sc[kScP]);
    frag_store_seq(oq, ow, o_step, a.T - c * kTc, lane);
    ow += 8 * o_step;
    // S1 = e^{G_C} S0 + (e^{G_C - G} u) k
    frag_scale(z, s.sc + 64, lane);
    state_update<DK>(S, s.sc[kScEnd], z, uf, ks, ui * s.sc[kScK], off);
  }
  zero_rows(o, a, o_row, b, len, lane);
  if (p.s_out) state_store<DK>(S, p.s_out + s_off, DK, lane);
}

// ---------------------------------------------------------------------------
// the scans with two warps to 16 value columns
// ---------------------------------------------------------------------------
// Where there are too few heads to fill the GPU, a chunk's time is one warp's
// chain.  Two warps then share 16 value columns: each keeps half of the state's
// key columns (half the products with the state, and half of its update) and
// finishes half of the token blocks, 0 and 3 or 1 and 2 (the same number of
// triangular products).  A chunk of D = 128 takes 2.4 us instead of 3.0 for a lone
// warp (16384 tokens, 32 heads: 623 against 772 us), not half: both warps split
// the whole of r and u.  Partial sums and finished blocks cross through shared
// memory, two exchanges a chunk forward and three backward, on a barrier of the
// two warps.
template <int DK>
struct alignas(128) PairSmem {
  static constexpr int W = 2;
  ScanStage<DK, W> st[2];
  uint64_t full[2];
  float smax[2][2 * W];
  float4 a[W][2][12][32], b[W][2][4][32];
};
template <int N>
struct Blk {
  static constexpr int v = N;
};
__device__ __forceinline__ void pair_sync(int pair) { asm volatile("bar.sync %0, 64;" :: "r"(pair + 1) : "memory"); }
__device__ __forceinline__ float4 as4(const float (&x)[4]) { return make_float4(x[0], x[1], x[2], x[3]); }
__device__ __forceinline__ void from4(float (&x)[4], float4 v) { x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w; }
__device__ __forceinline__ void add4(float (&x)[4], float4 v) { x[0] += v.x; x[1] += v.y; x[2] += v.z; x[3] += v.w; }
// Calls f with this warp's token blocks and its partner's.
template <typename F>
__device__ __forceinline__ void with_blocks(int half, F f) {
  if (half) f(Blk<1>(), Blk<2>(), Blk<0>(), Blk<3>());
  else f(Blk<0>(), Blk<3>(), Blk<1>(), Blk<2>());
}
// Sends this warp's two blocks of x and takes the partner's.
template <typename B0, typename B1, typename P0, typename P1>
__device__ __forceinline__ void swap_blocks(Frag& x, float4 (*mine)[32], float4 (*theirs)[32], int pair, int lane, B0, B1, P0, P1) {
  mine[0][lane] = as4(x[2 * B0::v]); mine[1][lane] = as4(x[2 * B0::v + 1]);
  mine[2][lane] = as4(x[2 * B1::v]); mine[3][lane] = as4(x[2 * B1::v + 1]);
  pair_sync(pair);
  from4(x[2 * P0::v], theirs[0][lane]); from4(x[2 * P0::v + 1], theirs[1][lane]);
  from4(x[2 * P1::v], theirs[2][lane]); from4(x[2 * P1::v + 1], theirs[3][lane]);
}
// acc of block b = the triangular product of a split fragment: rows n (kk <= b) or rows k (kk >= b)
template <bool ROWS_N, bool LOW_A, typename BB>
__device__ __forceinline__ void tri_block(Frag& acc, const uint32_t (&hi)[4][4], const uint32_t (&lo)[4][4], uint32_t tile,
                                          const LaneOffsets& off, bool low_b, BB) {
  constexpr int b = BB::v, n = 2 * b;
#pragma unroll
  for (int i = 0; i <= (ROWS_N ? b : 3 - b); ++i) {
    const int kk = ROWS_N ? i : b + i;
    uint32_t t[4];
    if (ROWS_N) scan_tri_n(t, tile, off, 8 * n, kk, 0);
    else scan_tri_k(t, tile, off, 8 * n, kk, 0);
    if (i == 0) {
      mma_h0(acc[n], hi[kk], t[0], t[1]);
      mma_h0(acc[n + 1], hi[kk], t[2], t[3]);
    } else {
      mma_h(acc[n], hi[kk], t[0], t[1]);
      mma_h(acc[n + 1], hi[kk], t[2], t[3]);
    }
    if (LOW_A) {
      mma_h(acc[n], lo[kk], t[0], t[1]);
      mma_h(acc[n + 1], lo[kk], t[2], t[3]);
    }
    if (low_b) {
      if (ROWS_N) scan_tri_n(t, tile, off, 8 * n, kk, 1);
      else scan_tri_k(t, tile, off, 8 * n, kk, 1);
      mma_h(acc[n], hi[kk], t[0], t[1]);
      mma_h(acc[n + 1], hi[kk], t[2], t[3]);
    }
  }
}
// Stores of one 16-token block.
template <typename BB>
__device__ __forceinline__ void block_store_half(const Frag& x, float f, __half* base, int pitch, int lane, BB) {
  __half* p = base + (lane >> 2) * pitch + 4 * (lane & 3);
#pragma unroll
  for (int n = 2 * BB::v; n < 2 * BB::v + 2; ++n)
    *reinterpret_cast<uint2*>(p + 8 * n * pitch) =
        make_uint2(transpose8(pack_h(mul2(lo2(x[n]), both(f)))), transpose8(pack_h(mul2(hi2(x[n]), both(f)))));
}
template <typename BB>
__device__ __forceinline__ void block_store_seq(const Frag& x, __nv_bfloat16* p, int64_t step, int left, int lane, BB) {
#pragma unroll
  for (int n = 2 * BB::v; n < 2 * BB::v + 2; ++n) {
    const uint32_t lo = transpose8(pack_b(x[n][0], x[n][1])), hi = transpose8(pack_b(x[n][2], x[n][3]));
    if ((lane >> 2) + 8 * n < left) *reinterpret_cast<uint2*>(p + n * step) = make_uint2(lo, hi);
  }
}

template <int DK, bool TRAIN>
__global__ void __launch_bounds__(128) delta_pair_fwd_kernel(const DeltaTcArgs p) {
  constexpr int W = 2, DKW = DK / 2;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  PairSmem<DK>& sm = *reinterpret_cast<PairSmem<DK>*>(smem_raw);
  const DeltaArgs& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, pair = warp >> 1, half = warp & 1;
  const int groups = a.Dv / (16 * W);
  const int64_t bid = blockIdx.x;
  const int grp = static_cast<int>(bid % groups), h = static_cast<int>(bid / groups % a.Hv),
            b = static_cast<int>(bid / groups / a.Hv);
  const int slice = grp * W + pair, dv0 = slice * 16;
  const int hk = h / (a.Hv / a.Hk);
  const int len = a.len ? a.len[b] : a.T;
  const int nc = (a.T + kTc - 1) / kTc, ncb = (len + kTc - 1) / kTc;
  const int64_t bh = static_cast<int64_t>(b) * a.Hv + h, bk = static_cast<int64_t>(b) * a.Hk + hk;
  const int64_t o_row = static_cast<int64_t>(a.Hv) * a.Dv;
  const int64_t s_off = (bh * a.Dv + dv0) * DK + DKW * half;
  const int64_t ts_ = a.bfirst ? 1 : a.B;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + static_cast<int64_t>(h) * a.Dv + dv0;
  const int64_t o_step = 8 * ts_ * o_row;
  __nv_bfloat16* ow = o + a.row(b, lane >> 2) * o_row + 4 * (lane & 3);
  // this warp's half of the key columns: 128 bytes further, or the other four pieces of a 128-byte row
  LaneOffsets off;
  off.init(DK * 2, lane, DK == 64 ? 4 * half : 0);
  const uint32_t koff = DK == 128 ? 128 * half : 0;
  ScanSource src;
  src.k = static_cast<const char*>(p.w.k16) + bk * nc * kTc * DK * 2;
  src.q = static_cast<const char*>(p.w.q16) + bk * nc * kTc * DK * 2;
  src.t = static_cast<const char*>(p.w.th) + bh * nc * kTri;
  src.p = static_cast<const char*>(p.w.p) + bh * nc * kTri;
  src.sc = reinterpret_cast<const char*>(p.w.sc) + bh * nc * kSc * 4;
  const int piece = threadIdx.x & 63;              // the first 64 threads fetch
  src.x = static_cast<const __nv_bfloat16*>(a.v) + a.row(b, piece / (2 * W)) * a.v_row + static_cast<int64_t>(h) * a.Dv +
          grp * 16 * W + 8 * (piece % (2 * W));
  src.x_step = 16 * ts_ * a.v_row;

  if (threadIdx.x == 0) {
    mbar_init(&sm.full[0], 1);
    mbar_init(&sm.full[1], 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (ncb > 0 && threadIdx.x < 64) scan_fetch<DK, W>(sm.st[0], &sm.full[0], src, 0, len);
  State<DKW> S;
  if (p.s_in) {
    state_load<DKW>(S, p.s_in + s_off, DK, lane);
  } else {
#pragma unroll
    for (int j = 0; j < DKW / 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) S.v[j][i] = 0.f;
  }
  for (int c = 0; c < ncb; ++c) {
    const float own_max = state_max<DKW>(S);
    if (lane == 0) sm.smax[c & 1][warp] = own_max;
    if (scan_arrive(sm.full, c, p.status)) return;
    if (c + 1 < ncb && threadIdx.x < 64)
      scan_fetch<DK, W>(sm.st[(c + 1) & 1], &sm.full[(c + 1) & 1], src, c + 1, len - (c + 1) * kTc);
    float smax = 0.f;
#pragma unroll
    for (int w = 0; w < 2 * W; ++w) smax = fmaxf(smax, sm.smax[c & 1][w]);
    const ScanStage<DK, W>& s = sm.st[c & 1];
    const uint32_t ks = smem_u32(s.K) + koff, qs = smem_u32(s.Q) + koff, ts = smem_u32(s.T), ps = smem_u32(s.P);
    float4 (*xa)[32] = sm.a[pair][half], (*ya)[32] = sm.a[pair][half ^ 1], (*xb)[32] = sm.b[pair][half],
           (*yb)[32] = sm.b[pair][half ^ 1];

    const float sf = up_scale(smax), si = inv_scale(sf);
    if (TRAIN) {
      state_store_half<DKW>(S, sf, static_cast<__half*>(p.w.s0) + ((bh * nc + c) * a.Dv + dv0) * DK + DKW * half, DK, lane);
      if (lane == 0 && half == 0) p.w.s0_scale[(bh * nc + c) * (a.Dv / 16) + slice] = si;
    }
    Frag z, oq, acc;
    state_times<DK, true>(S, sf, ks, qs, z, oq, off);
    with_blocks(half, [&](auto, auto, auto p0, auto p1) {
#pragma unroll
      for (int n = 0; n < 8; ++n) xa[n][lane] = as4(z[n]);
      xa[8][lane] = as4(oq[2 * decltype(p0)::v]); xa[9][lane] = as4(oq[2 * decltype(p0)::v + 1]);
      xa[10][lane] = as4(oq[2 * decltype(p1)::v]); xa[11][lane] = as4(oq[2 * decltype(p1)::v + 1]);
    });
    pair_sync(pair);
    const float zk = -si * s.sc[kScK], zq = si * s.sc[kScQ] * a.scale;
    Slice vs;
    slice_load<W>(vs, s.x, pair, lane);
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      add4(z[n], ya[n][lane]);
      const float2 ek = mul2(pair_of(s.sc, n, lane), both(zk));
      float2 lo, hi;
      slice_frag(vs, n, lo, hi);
      set4(z[n], fma2(lo2(z[n]), ek, lo), fma2(hi2(z[n]), ek, hi));
    }
    const float rf = up_scale(frag_max(z));
    uint32_t hi[4][4], lo[4][4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) frag_a(z, kk, rf, hi[kk], lo[kk]);
    const float ti = inv_scale(rf) * s.sc[kScTH];
    with_blocks(half, [&](auto b0, auto b1, auto p0, auto p1) {
      constexpr int n0 = 2 * decltype(b0)::v, n1 = 2 * decltype(b1)::v;
      add4(oq[n0], ya[8][lane]); add4(oq[n0 + 1], ya[9][lane]);
      add4(oq[n1], ya[10][lane]); add4(oq[n1 + 1], ya[11][lane]);
      tri_block<true, true>(acc, hi, lo, ts, off, true, b0);
      tri_block<true, true>(acc, hi, lo, ts, off, true, b1);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        set4(z[n0 + i], fma2(lo2(acc[n0 + i]), both(ti), lo2(z[n0 + i])), fma2(hi2(acc[n0 + i]), both(ti), hi2(z[n0 + i])));
        set4(z[n1 + i], fma2(lo2(acc[n1 + i]), both(ti), lo2(z[n1 + i])), fma2(hi2(acc[n1 + i]), both(ti), hi2(z[n1 + i])));
      }
      swap_blocks(z, xb, yb, pair, lane, b0, b1, p0, p1);
    });
    const float ef = up_scale(frag_max(z));
    if (TRAIN) {
      __half* e = static_cast<__half*>(p.w.e) + (bh * nc + c) * kTc * a.Dv + dv0;
      with_blocks(half, [&](auto b0, auto b1, auto, auto) {
        block_store_half(z, ef, e, a.Dv, lane, b0);
        block_store_half(z, ef, e, a.Dv, lane, b1);
      });
      if (lane == 0 && half == 0) p.w.e_scale[(bh * nc + c) * (a.Dv / 16) + slice] = inv_scale(ef);
    }
    const float uf = ef * s.sc[kScBu], ui = inv_scale(uf);
    frag_scale(z, s.sc + 128, lane);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) frag_a_hi(z, kk, uf, hi[kk]);
    const float pi = ui * s.sc[kScP];
    with_blocks(half, [&](auto b0, auto b1, auto, auto) {
      tri_block<true, false>(acc, hi, lo, ps, off, false, b0);
      tri_block<true, false>(acc, hi, lo, ps, off, false, b1);
      auto finish = [&](auto bb) {
#pragma unroll
        for (int n = 2 * decltype(bb)::v; n < 2 * decltype(bb)::v + 2; ++n) {
          const float2 eq = mul2(pair_of(s.sc, n, lane), both(zq));
          set4(oq[n], fma2(lo2(acc[n]), both(pi), mul2(lo2(oq[n]), eq)), fma2(hi2(acc[n]), both(pi), mul2(hi2(oq[n]), eq)));
        }
        block_store_seq(oq, ow, o_step, a.T - c * kTc, lane, bb);
      };
      finish(b0);
      finish(b1);
    });
    ow += 8 * o_step;
    frag_scale(z, s.sc + 64, lane);
    state_update<DK>(S, s.sc[kScEnd], z, uf, ks, ui * s.sc[kScK], off);
  }
  pair_sync(pair);                  // both warps have written rows of the last chunk
  if (half == 0) zero_rows(o, a, o_row, b, len, lane);
  if (p.s_out) state_store<DKW>(S, p.s_out + s_off, DK, lane);
}

int check_launch() { return cudaGetLastError() == cudaSuccess ? 0 : RNN_CUDA_ERROR; }

// 16-column slices a scan CTA takes: 8 or 4, a warp each, or 2 with two warps each;
// 8 for Dk 128 only.  What counts is the number of turns times a chunk's time,
// measured with 152 CTAs of 16 chunks, us:
//            Dk 128: 8     4     2      Dk 64: 8     4     2
//   inference       5.8   3.5   2.75          3.9   2.3   2.25
//   training        6.9   4.3   3.0           4.5   2.7   2.6
//   reverse         8.3   5.3   3.45          5.5   3.35  2.75
// One CTA is resident on an SM, but two of 4 slices with Dk 64, which take 3.7, 4.4
// and 5.1 together: never longer than one of 8, which is therefore not built.
enum { kScanInfer, kScanTrain, kScanReverse };
int scan_slices(const DeltaArgs& a, int num_sms, int kind) {
  struct Choice {
    int take, two;               // slices; whether two CTAs share an SM
    double us[3], us2[3];
  };
  static const Choice c128[] = {{8, 0, {5.8, 6.9, 8.3}, {}}, {4, 0, {3.5, 4.3, 5.3}, {}}, {2, 0, {2.75, 3.0, 3.45}, {}}};
  static const Choice c64[] = {{4, 1, {2.3, 2.7, 3.35}, {3.7, 4.4, 5.1}}, {2, 0, {2.25, 2.6, 2.75}, {}}};
  const int n = a.Dv / 16;
  int best = 2;
  double least = 1e30;
  auto weigh = [&](const Choice& c) {
    if (n % c.take) return;
    const int64_t ctas = static_cast<int64_t>(a.B) * a.Hv * (n / c.take), turns = (ctas + num_sms - 1) / num_sms;
    const double cost = c.two ? static_cast<double>(turns / 2) * c.us2[kind] + static_cast<double>(turns % 2) * c.us[kind]
                              : static_cast<double>(turns) * c.us[kind];
    if (cost < least) {
      least = cost;
      best = c.take;
    }
  };
  if (a.Dk == 64)
    for (const Choice& c : c64) weigh(c);
  else
    for (const Choice& c : c128) weigh(c);
  return best;
}

template <typename F>
int set_smem(F* f, int bytes) {
  return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess ? 0 : RNN_CUDA_ERROR;
}

template <int DK, bool TRAIN>
int forward(const DeltaTcArgs& t, cudaStream_t s, int* launches) {
  const int nc = (t.a.T + kTc - 1) / kTc;
  const int psm = sizeof(PrepSmem<DK, TRAIN>);
  delta_prep_kernel<DK, TRAIN><<<static_cast<unsigned>(static_cast<int64_t>(nc) * t.a.Hv * t.a.B), 128, psm, s>>>(t);
  int rc = check_launch();
  if (rc) return rc;
  ++*launches;
  const int w = scan_slices(t.a, t.num_sms, TRAIN ? kScanTrain : kScanInfer);
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(t.a.B) * t.a.Hv * (t.a.Dv / (16 * w)));
  if constexpr (DK == 128)
    if (w == 8) delta_scan_fwd_kernel<DK, TRAIN, 8><<<grid, 256, sizeof(ScanSmem<DK, 8>), s>>>(t);
  if (w == 4) delta_scan_fwd_kernel<DK, TRAIN, 4><<<grid, 128, sizeof(ScanSmem<DK, 4>), s>>>(t);
  if (w == 2) delta_pair_fwd_kernel<DK, TRAIN><<<grid, 128, sizeof(PairSmem<DK>), s>>>(t);
  rc = check_launch();
  if (!rc) ++*launches;
  return rc;
}

// ---------------------------------------------------------------------------
// the reverse scan
// ---------------------------------------------------------------------------
// The same ownership for the state gradient, chunks in reverse:
//   du = P^T do + e^{G_C - G} dS1 k          y = (I + beta A)^-T du
//   dS0 = e^{G_C} dS1 + (scale e^G do) q^T - (e^G beta y) k^T,   dv = beta y
template <int DK, int W>
__global__ void __launch_bounds__(32 * W) delta_scan_bwd_kernel(const DeltaTcBwdArgs p) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  ScanSmem<DK, W>& sm = *reinterpret_cast<ScanSmem<DK, W>*>(smem_raw);
  const DeltaArgs& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = a.Dv / (16 * W);
  const int64_t bid = blockIdx.x;
  const int grp = static_cast<int>(bid % groups), h = static_cast<int>(bid / groups % a.Hv),
            b = static_cast<int>(bid / groups / a.Hv);
  const int slice = grp * W + warp, dv0 = slice * 16;
  const int hk = h / (a.Hv / a.Hk);
  const int len = a.len ? a.len[b] : a.T;
  const int nc = (a.T + kTc - 1) / kTc, ncb = (len + kTc - 1) / kTc;
  const int64_t bh = static_cast<int64_t>(b) * a.Hv + h, bk = static_cast<int64_t>(b) * a.Hk + hk;
  const int64_t o_row = static_cast<int64_t>(a.Hv) * a.Dv;
  const int64_t s_off = (bh * a.Dv + dv0) * DK;
  const int64_t ts_ = a.bfirst ? 1 : a.B, o_step = 8 * ts_ * o_row;
  __nv_bfloat16* dv = static_cast<__nv_bfloat16*>(p.dv) + static_cast<int64_t>(h) * a.Dv + dv0 + 4 * (lane & 3) +
                      a.row(b, (lane >> 2) + (ncb > 0 ? ncb - 1 : 0) * kTc) * o_row;
  LaneOffsets off;
  off.init(DK * 2, lane);
  ScanSource src;
  src.k = static_cast<const char*>(p.w.k16) + bk * nc * kTc * DK * 2;
  src.q = static_cast<const char*>(p.w.q16) + bk * nc * kTc * DK * 2;
  src.t = static_cast<const char*>(p.w.tb) + bh * nc * kTri;
  src.p = static_cast<const char*>(p.w.p) + bh * nc * kTri;
  src.sc = reinterpret_cast<const char*>(p.w.sc) + bh * nc * kSc * 4;
  src.x = static_cast<const __nv_bfloat16*>(p.dout) + a.row(b, threadIdx.x / (2 * W)) * o_row + static_cast<int64_t>(h) * a.Dv +
          grp * 16 * W + 8 * (threadIdx.x % (2 * W));
  src.x_step = 16 * ts_ * o_row;

  if (threadIdx.x == 0) {
    mbar_init(&sm.full[0], 1);
    mbar_init(&sm.full[1], 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (ncb > 0) scan_fetch<DK, W>(sm.st[0], &sm.full[0], src, ncb - 1, len - (ncb - 1) * kTc);
  State<DK> S;
  if (p.dsT) {
    state_load<DK>(S, p.dsT + s_off, DK, lane);
  } else {
#pragma unroll
    for (int j = 0; j < DK / 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) S.v[j][i] = 0.f;
  }
  for (int it = 0; it < ncb; ++it) {
    const int c = ncb - 1 - it;
    const float own_max = state_max<DK>(S);
    if (lane == 0) sm.smax[it & 1][warp] = own_max;
    if (scan_arrive(sm.full, it, p.status)) return;
    float smax = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) smax = fmaxf(smax, sm.smax[it & 1][w]);
    if (c > 0) scan_fetch<DK, W>(sm.st[(it + 1) & 1], &sm.full[(it + 1) & 1], src, c - 1, kTc);
    const ScanStage<DK, W>& s = sm.st[it & 1];
    const uint32_t ks = smem_u32(s.K), qs = smem_u32(s.Q), ts = smem_u32(s.T), ps = smem_u32(s.P);

    const float sf = up_scale(smax), si = inv_scale(sf);
    state_store_half<DK>(S, sf, static_cast<__half*>(p.ds1) + ((bh * nc + c) * a.Dv + dv0) * DK, DK, lane);
    if (lane == 0) p.ds1_scale[(bh * nc + c) * (a.Dv / 16) + slice] = si;
    Frag z, acc;
    state_times<DK, false>(S, sf, ks, ks, z, z, off);
    // P^T do: do is exact in fp16 once scaled
    Slice ds;
    slice_load<W>(ds, s.x, warp, lane);
    float dm = 0.f;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const float2 x = unpack_b(ds.v[n].x), y = unpack_b(ds.v[n].y);
      dm = fmaxf(fmaxf(dm, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(y.x), fabsf(y.y)));
    }
    const float df = up_scale(warp_max(dm));
    if (lane == 0) p.do_scale[(bh * nc + c) * (a.Dv / 16) + slice] = inv_scale(df);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      float2 x0, x1, y0, y1;
      slice_frag(ds, 2 * kk, x0, x1);
      slice_frag(ds, 2 * kk + 1, y0, y1);
      const uint32_t ad[4] = {pack_h(mul2(x0, both(df))), pack_h(mul2(x1, both(df))), pack_h(mul2(y0, both(df))),
                              pack_h(mul2(y1, both(df)))};
#pragma unroll
      for (int n = 0; n <= 2 * kk; n += 2) {      // j <= i
        uint32_t bh_[4], bl_[4];
        scan_tri_k(bh_, ps, off, 8 * n, kk, 0);
        scan_tri_k(bl_, ps, off, 8 * n, kk, 1);
        if (n == 2 * kk) {
          mma_h0(acc[n], ad, bh_[0], bh_[1]);
          mma_h0(acc[n + 1], ad, bh_[2], bh_[3]);
        } else {
          mma_h(acc[n], ad, bh_[0], bh_[1]);
          mma_h(acc[n + 1], ad, bh_[2], bh_[3]);
        }
        mma_h(acc[n], ad, bl_[0], bl_[1]);
        mma_h(acc[n + 1], ad, bl_[2], bl_[3]);
      }
    }
    const float zk = si * s.sc[kScK], pi = inv_scale(df) * s.sc[kScP];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const float2 ee = mul2(pair_of(s.sc + 64, n, lane), both(zk));
      set4(z[n], fma2(lo2(acc[n]), both(pi), mul2(lo2(z[n]), ee)), fma2(hi2(acc[n]), both(pi), mul2(hi2(z[n]), ee)));
    }
    // y = du + (T - I)^T du
    const float uf = up_scale(frag_max(z));
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      uint32_t hi[4], lo[4];
      frag_a(z, kk, uf, hi, lo);
#pragma unroll
      for (int n = 0; n <= 2 * kk; n += 2) {
        uint32_t bh_[4], bl_[4];
        scan_tri_k(bh_, ts, off, 8 * n, kk, 0);
        scan_tri_k(bl_, ts, off, 8 * n, kk, 1);
        if (n == 2 * kk) {
          mma_h0(acc[n], hi, bh_[0], bh_[1]);
          mma_h0(acc[n + 1], hi, bh_[2], bh_[3]);
        } else {
          mma_h(acc[n], hi, bh_[0], bh_[1]);
          mma_h(acc[n + 1], hi, bh_[2], bh_[3]);
        }
        mma_h(acc[n], lo, bh_[0], bh_[1]);
        mma_h(acc[n + 1], lo, bh_[2], bh_[3]);
        mma_h(acc[n], hi, bl_[0], bl_[1]);
        mma_h(acc[n + 1], hi, bl_[2], bl_[3]);
      }
    }
    frag_add(z, acc, inv_scale(uf) * s.sc[kScTB]);
    const float yf = up_scale(frag_max(z));
    frag_store_half(z, yf, static_cast<__half*>(p.y) + (bh * nc + c) * kTc * a.Dv + dv0, a.Dv, lane);
    if (lane == 0) p.y_scale[(bh * nc + c) * (a.Dv / 16) + slice] = inv_scale(yf);
    frag_scale(z, s.sc + 128, lane);
    frag_store_seq(z, dv, o_step, a.T - c * kTc, lane);
    dv -= 8 * o_step;
    // -e^G beta y and scale e^G do; their scales follow from those of y and do
    // and bounds on the weights (kScBy, kScBo)
    const float xf = yf * s.sc[kScBy], af = df * s.sc[kScBo];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const float2 eg = pair_of(s.sc, n, lane), es = mul2(eg, both(a.scale)), em = mul2(eg, both(-1.f));
      float2 lo, hi;
      slice_frag(ds, n, lo, hi);
      set4(acc[n], mul2(lo, es), mul2(hi, es));
      set4(z[n], mul2(lo2(z[n]), em), mul2(hi2(z[n]), em));
    }
    state_update<DK>(S, s.sc[kScEnd], acc, af, qs, inv_scale(af) * s.sc[kScQ], off);
    state_update<DK>(S, 1.f, z, xf, ks, inv_scale(xf) * s.sc[kScK], off);
  }
  zero_rows(static_cast<__nv_bfloat16*>(p.dv) + static_cast<int64_t>(h) * a.Dv + dv0, a, o_row, b, len, lane);
  if (p.ds0) state_store<DK>(S, p.ds0 + s_off, DK, lane);
}

template <int DK>
__global__ void __launch_bounds__(128) delta_pair_bwd_kernel(const DeltaTcBwdArgs p) {
  constexpr int W = 2, DKW = DK / 2;
  extern __shared__ __align__(128) unsigned char smem_raw[];
  PairSmem<DK>& sm = *reinterpret_cast<PairSmem<DK>*>(smem_raw);
  const DeltaArgs& a = p.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, pair = warp >> 1, half = warp & 1;
  const int groups = a.Dv / (16 * W);
  const int64_t bid = blockIdx.x;
  const int grp = static_cast<int>(bid % groups), h = static_cast<int>(bid / groups % a.Hv),
            b = static_cast<int>(bid / groups / a.Hv);
  const int slice = grp * W + pair, dv0 = slice * 16;
  const int hk = h / (a.Hv / a.Hk);
  const int len = a.len ? a.len[b] : a.T;
  const int nc = (a.T + kTc - 1) / kTc, ncb = (len + kTc - 1) / kTc;
  const int64_t bh = static_cast<int64_t>(b) * a.Hv + h, bk = static_cast<int64_t>(b) * a.Hk + hk;
  const int64_t o_row = static_cast<int64_t>(a.Hv) * a.Dv;
  const int64_t s_off = (bh * a.Dv + dv0) * DK + DKW * half;
  const int64_t ts_ = a.bfirst ? 1 : a.B, o_step = 8 * ts_ * o_row;
  __nv_bfloat16* dv = static_cast<__nv_bfloat16*>(p.dv) + static_cast<int64_t>(h) * a.Dv + dv0 + 4 * (lane & 3) +
                      a.row(b, (lane >> 2) + (ncb > 0 ? ncb - 1 : 0) * kTc) * o_row;
  LaneOffsets off;
  off.init(DK * 2, lane, DK == 64 ? 4 * half : 0);
  const uint32_t koff = DK == 128 ? 128 * half : 0;
  ScanSource src;
  src.k = static_cast<const char*>(p.w.k16) + bk * nc * kTc * DK * 2;
  src.q = static_cast<const char*>(p.w.q16) + bk * nc * kTc * DK * 2;
  src.t = static_cast<const char*>(p.w.tb) + bh * nc * kTri;
  src.p = static_cast<const char*>(p.w.p) + bh * nc * kTri;
  src.sc = reinterpret_cast<const char*>(p.w.sc) + bh * nc * kSc * 4;
  const int piece = threadIdx.x & 63;
  src.x = static_cast<const __nv_bfloat16*>(p.dout) + a.row(b, piece / (2 * W)) * o_row + static_cast<int64_t>(h) * a.Dv +
          grp * 16 * W + 8 * (piece % (2 * W));
  src.x_step = 16 * ts_ * o_row;

  if (threadIdx.x == 0) {
    mbar_init(&sm.full[0], 1);
    mbar_init(&sm.full[1], 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (ncb > 0 && threadIdx.x < 64) scan_fetch<DK, W>(sm.st[0], &sm.full[0], src, ncb - 1, len - (ncb - 1) * kTc);
  State<DKW> S;
  if (p.dsT) {
    state_load<DKW>(S, p.dsT + s_off, DK, lane);
  } else {
#pragma unroll
    for (int j = 0; j < DKW / 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) S.v[j][i] = 0.f;
  }
  for (int it = 0; it < ncb; ++it) {
    const int c = ncb - 1 - it;
    const float own_max = state_max<DKW>(S);
    if (lane == 0) sm.smax[it & 1][warp] = own_max;
    if (scan_arrive(sm.full, it, p.status)) return;
    if (c > 0 && threadIdx.x < 64) scan_fetch<DK, W>(sm.st[(it + 1) & 1], &sm.full[(it + 1) & 1], src, c - 1, kTc);
    float smax = 0.f;
#pragma unroll
    for (int w = 0; w < 2 * W; ++w) smax = fmaxf(smax, sm.smax[it & 1][w]);
    const ScanStage<DK, W>& s = sm.st[it & 1];
    const uint32_t ks = smem_u32(s.K) + koff, qs = smem_u32(s.Q) + koff, ts = smem_u32(s.T), ps = smem_u32(s.P);
    float4 (*xa)[32] = sm.a[pair][half], (*ya)[32] = sm.a[pair][half ^ 1], (*xb)[32] = sm.b[pair][half],
           (*yb)[32] = sm.b[pair][half ^ 1];

    const float sf = up_scale(smax), si = inv_scale(sf);
    state_store_half<DKW>(S, sf, static_cast<__half*>(p.ds1) + ((bh * nc + c) * a.Dv + dv0) * DK + DKW * half, DK, lane);
    if (lane == 0 && half == 0) p.ds1_scale[(bh * nc + c) * (a.Dv / 16) + slice] = si;
    Frag z, acc;
    state_times<DK, false>(S, sf, ks, ks, z, z, off);
    // the partner's blocks of this half's sum
    with_blocks(half, [&](auto, auto, auto p0, auto p1) {
      constexpr int n0 = 2 * decltype(p0)::v, n1 = 2 * decltype(p1)::v;
      xa[0][lane] = as4(z[n0]); xa[1][lane] = as4(z[n0 + 1]);
      xa[2][lane] = as4(z[n1]); xa[3][lane] = as4(z[n1 + 1]);
    });
    Slice ds;
    slice_load<W>(ds, s.x, pair, lane);
    float dm = 0.f;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const float2 x = unpack_b(ds.v[n].x), y = unpack_b(ds.v[n].y);
      dm = fmaxf(fmaxf(dm, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(y.x), fabsf(y.y)));
    }
    const float df = up_scale(warp_max(dm));
    if (lane == 0 && half == 0) p.do_scale[(bh * nc + c) * (a.Dv / 16) + slice] = inv_scale(df);
    Frag x;                                   // do, for the operand here and the update below
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      float2 lo, hi;
      slice_frag(ds, n, lo, hi);
      set4(x[n], lo, hi);
    }
    uint32_t hi[4][4], lo[4][4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) frag_a_hi(x, kk, df, hi[kk]);
    const float zk = si * s.sc[kScK], pi = inv_scale(df) * s.sc[kScP];
    with_blocks(half, [&](auto b0, auto b1, auto p0, auto p1) {
      tri_block<false, false>(acc, hi, lo, ps, off, true, b0);
      tri_block<false, false>(acc, hi, lo, ps, off, true, b1);
      pair_sync(pair);
      auto join = [&](auto bb, int at) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int n = 2 * decltype(bb)::v + i;
          add4(z[n], ya[at + i][lane]);
          const float2 ee = mul2(pair_of(s.sc + 64, n, lane), both(zk));
          set4(z[n], fma2(lo2(acc[n]), both(pi), mul2(lo2(z[n]), ee)), fma2(hi2(acc[n]), both(pi), mul2(hi2(z[n]), ee)));
        }
      };
      join(b0, 0);
      join(b1, 2);
      swap_blocks(z, xb, yb, pair, lane, b0, b1, p0, p1);
    });
    // y = du + (T - I)^T du
    const float uf = up_scale(frag_max(z)), ti = inv_scale(uf) * s.sc[kScTB];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) frag_a(z, kk, uf, hi[kk], lo[kk]);
    with_blocks(half, [&](auto b0, auto b1, auto p0, auto p1) {
      tri_block<false, true>(acc, hi, lo, ts, off, true, b0);
      tri_block<false, true>(acc, hi, lo, ts, off, true, b1);
      constexpr int n0 = 2 * decltype(b0)::v, n1 = 2 * decltype(b1)::v;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        set4(z[n0 + i], fma2(lo2(acc[n0 + i]), both(ti), lo2(z[n0 + i])), fma2(hi2(acc[n0 + i]), both(ti), hi2(z[n0 + i])));
        set4(z[n1 + i], fma2(lo2(acc[n1 + i]), both(ti), lo2(z[n1 + i])), fma2(hi2(acc[n1 + i]), both(ti), hi2(z[n1 + i])));
      }
      swap_blocks(z, xa + 4, ya + 4, pair, lane, b0, b1, p0, p1);
    });
    const float yf = up_scale(frag_max(z));
    {
      __half* y = static_cast<__half*>(p.y) + (bh * nc + c) * kTc * a.Dv + dv0;
      with_blocks(half, [&](auto b0, auto b1, auto, auto) {
        block_store_half(z, yf, y, a.Dv, lane, b0);
        block_store_half(z, yf, y, a.Dv, lane, b1);
      });
      if (lane == 0 && half == 0) p.y_scale[(bh * nc + c) * (a.Dv / 16) + slice] = inv_scale(yf);
    }
    frag_scale(z, s.sc + 128, lane);
    with_blocks(half, [&](auto b0, auto b1, auto, auto) {
      block_store_seq(z, dv, o_step, a.T - c * kTc, lane, b0);
      block_store_seq(z, dv, o_step, a.T - c * kTc, lane, b1);
    });
    dv -= 8 * o_step;
    const float xf = yf * s.sc[kScBy], af = df * s.sc[kScBo];
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const float2 eg = pair_of(s.sc, n, lane), es = mul2(eg, both(a.scale)), em = mul2(eg, both(-1.f));
      set4(x[n], mul2(lo2(x[n]), es), mul2(hi2(x[n]), es));
      set4(z[n], mul2(lo2(z[n]), em), mul2(hi2(z[n]), em));
    }
    state_update<DK>(S, s.sc[kScEnd], x, af, qs, inv_scale(af) * s.sc[kScQ], off);
    state_update<DK>(S, 1.f, z, xf, ks, inv_scale(xf) * s.sc[kScK], off);
  }
  pair_sync(pair);
  if (half == 0) zero_rows(static_cast<__nv_bfloat16*>(p.dv) + static_cast<int64_t>(h) * a.Dv + dv0, a, o_row, b, len, lane);
  if (p.ds0) state_store<DKW>(S, p.ds0 + s_off, DK, lane);
}

// ---------------------------------------------------------------------------
// the gradients of q, k, g and beta, all chunks at once
// ---------------------------------------------------------------------------
// Bound by what surrounds the products, not by them (24 % of the tensor pipe) nor
// by memory (1.6 of 6.8 TB/s): ldmatrix and its waits, scaling, sums across warps.
// 4096 chunks of D = 128 in 362 us.  Eight warps with tiles of 32 x 32 took 428;
// rescaling A operands in the products instead of pieces on arrival 407.
// The sums of delta_chunk_bwd_kernel (delta_simt.cu) on the tensor cores, with
// single fp16 operands: every output is rounded to bf16, 8 times coarser.  A CTA
// walks chunks of a key head with a stride; per value head the value columns
// pass in slices of 64 through two stages, the next one (and the next chunk's
// keys and queries) arriving while this one is multiplied.  Warp (rg, cq) of
// 2 x Dk / 16 owns rows 32 rg .. + 31 and 16 of the key columns of every product.
// The fp16 copies of S0, dS1, e, y and do carry one scale per 16 value columns;
// each piece is brought to the head's largest as it arrives, exactly (a power of
// two), so that one accumulator takes the sum over all value columns.
template <int DK>
struct GradSmem {
  static constexpr int NW = DK / 8, NT = 32 * NW;                // warps, threads
  struct Stage {
    unsigned char dO[kTc * 128], E[kTc * 128], Y[kTc * 128];     // [64 tokens][64 columns]
    unsigned char S0[64 * DK * 2], dS[64 * DK * 2];              // [64 value columns][Dk]
  } st[2];
  unsigned char K[2][kTc * DK * 2], Q[2][kTc * DK * 2];
  unsigned char mP[kTc * 128], mA[kTc * 128];
  float eG[kTc], eE[kTc], beta[kTc], Gh[kTc], Gl[kTc];
  // per 16 value columns: the fp16 pair that brings S0, dS1, e, y to the head's
  // scale, the fp32 factor that does so from bf16 for do; and the head's inverse scales
  uint32_t ratio[5][16];
  float inv[5];
  float own[NW / 2][kTc], thru[NW / 2][kTc], row[NW / 2][kTc], col[2][kTc];
  float red[NW], mx[2][NW];
  alignas(16) float dG[kTc];     // read in pairs
  float w[kTc];
};
enum { kRs = 0, kRd, kRe, kRy, kRo };

// A place in a CTA's walk: chunk c of (batch b, key head hk), value head hh of
// the group, slice sl; t0 and nt its first token and valid tokens.
struct GradPos {
  int item, b, hk, c, nt, hh, sl;
};

template <int DK>
__global__ void __launch_bounds__(GradSmem<DK>::NT) delta_grad_kernel(const DeltaTcBwdArgs p) {
  using SM = GradSmem<DK>;
  constexpr int PK = DK * 2, NT = SM::NT, NW = SM::NW, CQ = NW / 2;
  constexpr int NJ = 8 / CQ;                   // n-tiles of a warp in the pair matrices
  extern __shared__ __align__(128) unsigned char smem_raw[];
  SM& sm = *reinterpret_cast<SM*>(smem_raw);
  const DeltaArgs& a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rg = warp / CQ, cq = warp % CQ;
  const int r = lane >> 2, cc = 2 * (lane & 3);
  const int nc = (a.T + kTc - 1) / kTc, per = a.Hv / a.Hk, ns = (a.Dv + 63) / 64, n16 = a.Dv / 16;
  const int items = a.B * a.Hk * nc;           // below 2^31: checked when the handle is made
  const int64_t qk_row = static_cast<int64_t>(a.Hk) * DK, v_row = static_cast<int64_t>(a.Hv) * a.Dv;

  auto at_item = [&](GradPos& g, int item) {
    g.item = item;
    const int bk = item / nc;
    g.c = item - bk * nc;
    g.b = bk / a.Hk;
    g.hk = bk - g.b * a.Hk;
    g.nt = item < items ? (a.len ? a.len[g.b] : a.T) - g.c * kTc : 1;
    g.hh = g.sl = 0;
  };
  auto next_item = [&](GradPos& g, int item) {
    at_item(g, item);
    while (g.nt <= 0) at_item(g, item += gridDim.x);
  };
  // this CTA's chunks without tokens: zeros
  if (a.len) {
    for (int item = blockIdx.x; item < items; item += gridDim.x) {
      GradPos g;
      at_item(g, item);
      if (g.nt > 0) continue;
      const int t0 = g.c * kTc, span = min(kTc, a.T - t0);
      for (int x = tid; x < span * DK / 8; x += NT) {
        const int64_t at = a.row(g.b, t0 + x / (DK / 8)) * qk_row + g.hk * DK + x % (DK / 8) * 8;
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dq) + at) = make_uint4(0u, 0u, 0u, 0u);
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.dk) + at) = make_uint4(0u, 0u, 0u, 0u);
      }
      for (int x = tid; x < span * per; x += NT) {
        const int64_t at = a.row(g.b, t0 + x / per) * a.Hv + g.hk * per + x % per;
        static_cast<__nv_bfloat16*>(p.dg)[at] = __float2bfloat16_rn(0.f);
        static_cast<__nv_bfloat16*>(p.dbeta)[at] = __float2bfloat16_rn(0.f);
      }
    }
  }

  auto head_chunk = [&](const GradPos& g) {
    return (static_cast<int64_t>(g.b) * a.Hv + g.hk * per + g.hh) * nc + g.c;
  };
  const int64_t tstep = a.bfirst ? 1 : a.B;
  auto fetch = [&](const GradPos& g, int stage, int kq) {
    const int64_t bhc = head_chunk(g), row0 = a.row(g.b, g.c * kTc);
    typename SM::Stage& s = sm.st[stage];
    const uint32_t dO = smem_u32(s.dO), E = smem_u32(s.E), Y = smem_u32(s.Y), S0 = smem_u32(s.S0), dS = smem_u32(s.dS);
    const int v0 = g.sl * 64;
    {
      // piece ch of tokens t, t + NT / 8, ...
      const int ch = tid & 7;
      const bool in = v0 + ch * 8 < a.Dv;
      const int col = in ? v0 + ch * 8 : 0;
      const __nv_bfloat16* dop = static_cast<const __nv_bfloat16*>(p.dout) + row0 * v_row +
                                 static_cast<int64_t>(g.hk * per + g.hh) * a.Dv + col;
      const __half *ep = static_cast<const __half*>(p.w.e) + bhc * kTc * a.Dv + col,
                   *yp = static_cast<const __half*>(p.y) + bhc * kTc * a.Dv + col;
#pragma unroll
      for (int i = 0; i < kTc * 8 / NT; ++i) {
        const int t = (tid >> 3) + i * (NT / 8);
        const uint32_t at = swz<128>(t, ch);
        const bool ok = in && t < g.nt;
        cp16_or_zero(dO + at, dop + (ok ? t * tstep * v_row : 0), ok);
        cp16_or_zero(E + at, ep + t * a.Dv, in);
        cp16_or_zero(Y + at, yp + t * a.Dv, in);
      }
    }
    {
      constexpr int PR = DK / 8;
      const int ch = tid % PR;
      const int64_t base = (bhc * a.Dv + v0) * DK + ch * 8;
#pragma unroll
      for (int i = 0; i < 64 * PR / NT; ++i) {
        const int d = tid / PR + i * (NT / PR);
        const bool in = v0 + d < a.Dv;
        const int64_t at = in ? base + d * DK : 0;
        cp16_or_zero(S0 + swz<PK>(d, ch), static_cast<const __half*>(p.w.s0) + at, in);
        cp16_or_zero(dS + swz<PK>(d, ch), static_cast<const __half*>(p.ds1) + at, in);
      }
      if (g.hh == 0 && g.sl == 0) {
        const uint32_t ks = smem_u32(sm.K[kq]), qs = smem_u32(sm.Q[kq]);
        const __nv_bfloat16 *kp = static_cast<const __nv_bfloat16*>(a.k) + row0 * a.k_row + g.hk * DK + ch * 8,
                            *qp = static_cast<const __nv_bfloat16*>(a.q) + row0 * a.q_row + g.hk * DK + ch * 8;
#pragma unroll
        for (int i = 0; i < kTc * PR / NT; ++i) {
          const int t = tid / PR + i * (NT / PR);
          const bool ok = t < g.nt;
          const int64_t dt = ok ? t * tstep : 0;
          cp16_or_zero(ks + swz<PK>(t, ch), kp + dt * a.k_row, ok);
          cp16_or_zero(qs + swz<PK>(t, ch), qp + dt * a.q_row, ok);
        }
      }
    }
    cp_commit();
  };
  // bf16 -> fp16 times f, in place (each thread the pieces it copied itself)
  auto to_half = [&](unsigned char* at, float f) {
    const uint4 v = *reinterpret_cast<uint4*>(at);
    *reinterpret_cast<uint4*>(at) = make_uint4(pack_h(mul2(unpack_b(v.x), both(f))), pack_h(mul2(unpack_b(v.y), both(f))),
                                               pack_h(mul2(unpack_b(v.z), both(f))), pack_h(mul2(unpack_b(v.w), both(f))));
  };

  GradPos cur;
  next_item(cur, blockIdx.x);
  int stage = 0, kq = 0;
  if (cur.item < items) fetch(cur, 0, 0);
  float dq[2][2][4], dk[2][2][4];
  float N[2][NJ][4], Pm[2][NJ][4];
  float t_[3][2][2][4];            // do S0, y S0, e dS1 of the head
  float2 frob2 = both(0.f);
  while (cur.item < items) {
    const int t0 = cur.c * kTc, nt = cur.nt, h = cur.hk * per + cur.hh;
    const int64_t bhc = head_chunk(cur);
    const float* sc = p.w.sc + bhc * kSc;
    typename SM::Stage& s = sm.st[stage];
    const uint32_t ks = smem_u32(sm.K[kq]), qs = smem_u32(sm.Q[kq]);
    const bool new_head = cur.sl == 0, new_item = new_head && cur.hh == 0;
    if (new_item) {
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) dq[mt][n][e] = dk[mt][n][e] = 0.f;
    }
    if (new_head) {
      if (tid < kTc) {
        sm.eG[tid] = sc[tid];
        sm.eE[tid] = sc[64 + tid];
        sm.beta[tid] = sc[128 + tid];
        sm.Gh[tid] = sc[kScG + tid];
        sm.Gl[tid] = sc[kScGl + tid];
      }
      if (warp >= 3 && warp < 8) {
        const int w = warp - 3;
        const float* x = w == kRs ? p.w.s0_scale : w == kRd ? p.ds1_scale : w == kRe ? p.w.e_scale : w == kRy ? p.y_scale : p.do_scale;
        const int e = lane < n16 ? __float_as_int(x[bhc * n16 + lane]) >> 23 : 0;       // of the inverse scales
        const int m = __reduce_max_sync(kFull, e);
        if (lane < 16) {
          const int d = e - m;                          // 2^d as fp16: zero below 2^-24
          const float f = d < -24 ? 0.f : __int_as_float((127 + d) << 23);
          sm.ratio[w][lane] = w == kRo ? __float_as_uint(__int_as_float((254 - m) << 23)) : pack_h(f, f);
        }
        if (lane == 0) sm.inv[w] = __int_as_float(m << 23);
      }
      // the stage's pieces are scaled with these below
      __syncthreads();
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
        for (int n = 0; n < NJ; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) N[mt][n][e] = Pm[mt][n][e] = 0.f;
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) t_[i][mt][n][e] = 0.f;
      }
      frob2 = both(0.f);
    }
    cp_wait<0>();
    // this thread's own pieces: do to fp16, the others to the head's scale, <S0, dS1>, and a new chunk's keys and
    // queries to fp16
    auto rescale = [&](unsigned char* at, uint32_t ratio) {
      uint4 v = *reinterpret_cast<uint4*>(at);
      if (ratio == 0x3c003c00u) return v;               // ones
      const __half2 m = *reinterpret_cast<const __half2*>(&ratio);
      auto mul = [&](uint32_t x) {
        const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&x), m);
        return *reinterpret_cast<const uint32_t*>(&y);
      };
      v = make_uint4(mul(v.x), mul(v.y), mul(v.z), mul(v.w));
      *reinterpret_cast<uint4*>(at) = v;
      return v;
    };
    {
      const int ch = tid & 7, s16 = cur.sl * 4 + (ch >> 1);
      if (s16 < n16) {
        const float f = __uint_as_float(sm.ratio[kRo][s16]);
        const uint32_t re = sm.ratio[kRe][s16], ry = sm.ratio[kRy][s16];
#pragma unroll
        for (int i = 0; i < kTc * 8 / NT; ++i) {
          const uint32_t at = swz<128>((tid >> 3) + i * (NT / 8), ch);
          to_half(s.dO + at, f);
          rescale(s.E + at, re);
          rescale(s.Y + at, ry);
        }
      }
      constexpr int PR = DK / 8;
      const int cp_ = tid % PR;
#pragma unroll
      for (int i = 0; i < 64 * PR / NT; ++i) {
        const int d = tid / PR + i * (NT / PR), d16 = cur.sl * 4 + (d >> 4);
        if (d16 >= n16) continue;
        const uint32_t at = swz<PK>(d, cp_);
        const uint4 u = rescale(s.S0 + at, sm.ratio[kRs][d16]), w = rescale(s.dS + at, sm.ratio[kRd][d16]);
        frob2 = fma2(unpack_h(u.x), unpack_h(w.x), frob2);
        frob2 = fma2(unpack_h(u.y), unpack_h(w.y), frob2);
        frob2 = fma2(unpack_h(u.z), unpack_h(w.z), frob2);
        frob2 = fma2(unpack_h(u.w), unpack_h(w.w), frob2);
      }
      if (new_item) {
        const float kf = inv_scale(sc[kScK]), qf = inv_scale(sc[kScQ]);
#pragma unroll
        for (int i = 0; i < kTc * PR / NT; ++i) {
          const uint32_t at = swz<PK>(tid / PR + i * (NT / PR), cp_);
          to_half(sm.K[kq] + at, kf);
          to_half(sm.Q[kq] + at, qf);
        }
      }
    }
    __syncthreads();
    GradPos nxt = cur;
    int nkq = kq;
    if (++nxt.sl == ns) {
      nxt.sl = 0;
      if (++nxt.hh == per) {
        next_item(nxt, cur.item + gridDim.x);
        nkq = kq ^ 1;
      }
    }
    if (nxt.item < items) fetch(nxt, stage ^ 1, nkq);

    // products over this slice of value columns
    const uint32_t dO = smem_u32(s.dO), E = smem_u32(s.E), Y = smem_u32(s.Y), S0 = smem_u32(s.S0), dS = smem_u32(s.dS);
    auto load_a = [&](uint32_t (&f)[4], uint32_t tile, int mt, int kk) {
      ldsm(f, tile + swz<128>(32 * rg + 16 * mt + (lane & 15), 2 * kk + (lane >> 4)));
    };
    // do S0, y S0 and e dS1: tokens x key columns; y e^T and do e^T: tokens x tokens
    const bool lower = 8 * NJ * cq < 32 * rg + 32;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      uint32_t bs[4], bd[4], be[4];
      load_b_rows_k<PK>(bs, S0, cq * 16, kk, lane);
      load_b_rows_k<PK>(bd, dS, cq * 16, kk, lane);
      if (lower) {
        if (NJ == 1) ldsm(be, E + swz<128>(8 * cq + (lane & 7), 2 * kk + ((lane >> 3) & 1)));
        else load_b_rows_n<128>(be, E, 16 * cq, kk, lane);
      }
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint32_t fo[4], fy[4], fe[4];
        load_a(fo, dO, mt, kk);
        load_a(fy, Y, mt, kk);
        load_a(fe, E, mt, kk);
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          mma_h(t_[0][mt][n], fo, bs[2 * n], bs[2 * n + 1]);
          mma_h(t_[1][mt][n], fy, bs[2 * n], bs[2 * n + 1]);
          mma_h(t_[2][mt][n], fe, bd[2 * n], bd[2 * n + 1]);
        }
        if (lower)
#pragma unroll
          for (int n = 0; n < NJ; ++n) {
            mma_h(N[mt][n], fy, be[2 * n], be[2 * n + 1]);
            mma_h(Pm[mt][n], fo, be[2 * n], be[2 * n + 1]);
          }
      }
    }

    if (cur.sl == ns - 1) {
      // the head is complete.  Adds t times f w[row] to acc; returns in dot the product of that with the rows of X16
      // (true scale by xi)
      auto fold = [&](const float (&t)[2][2][4], float (&acc)[2][2][4], float2 (&dot)[2][2], const float* w, const float* w2,
                      float f, const unsigned char* X16, float xi) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int i = 32 * rg + 16 * mt + 8 * half + r;
            const float2 g = both(w2 ? f * w[i] * w2[i] : f * w[i]);
            float2 d = both(0.f);
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              float* x = &acc[mt][n][2 * half];
              const float2 tt = make_float2(t[mt][n][2 * half], t[mt][n][2 * half + 1]);
              const float2 y = fma2(tt, g, make_float2(x[0], x[1]));
              x[0] = y.x;
              x[1] = y.y;
              d = fma2(tt, unpack_h(*reinterpret_cast<const uint32_t*>(X16 + swz<PK>(i, 2 * cq + n) + 2 * cc)), d);
            }
            dot[mt][half] = fma2(d, mul2(g, both(xi)), dot[mt][half]);
          }
      };
      const float ki = sc[kScK], qi = sc[kScQ];
      const float iS = sm.inv[kRs], iD = sm.inv[kRd], iE = sm.inv[kRe], iY = sm.inv[kRy], iO = sm.inv[kRo];
      float2 own[2][2], thru[2][2];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) own[mt][0] = own[mt][1] = thru[mt][0] = thru[mt][1] = both(0.f);
      fold(t_[0], dq, own, sm.eG, nullptr, a.scale * iO * iS, sm.Q[kq], qi);
      fold(t_[1], dk, own, sm.eG, sm.beta, -(iY * iS), sm.K[kq], ki);
      fold(t_[2], dk, thru, sm.eE, sm.beta, iE * iD, sm.K[kq], ki);
      // K K^T and Q K^T of this warp's block, the pair weights, their sums
      float kk_[2][NJ][4], qk_[2][NJ][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int n = 0; n < NJ; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) kk_[mt][n][e] = qk_[mt][n][e] = 0.f;
      if (8 * NJ * cq < 32 * rg + 32) {
#pragma unroll
        for (int k2 = 0; k2 < DK / 16; k2 += 2) {
          uint32_t be[2][4];
          if (NJ == 1) {
            uint32_t q4[4];
            ldsm(q4, ks + swz<PK>(8 * cq + (lane & 7), 2 * k2 + (lane >> 3)));
            be[0][0] = q4[0]; be[0][1] = q4[1]; be[1][0] = q4[2]; be[1][1] = q4[3];
          } else {
            load_b_rows_n<PK>(be[0], ks, 16 * cq, k2, lane);
            load_b_rows_n<PK>(be[1], ks, 16 * cq, k2 + 1, lane);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {
              uint32_t fk[4], fq[4];
              const uint32_t at = swz<PK>(32 * rg + 16 * mt + (lane & 15), 2 * (k2 + i) + (lane >> 4));
              ldsm(fk, ks + at);
              ldsm(fq, qs + at);
#pragma unroll
              for (int n = 0; n < NJ; ++n) {
                mma_h(kk_[mt][n], fk, be[i][2 * n], be[i][2 * n + 1]);
                mma_h(qk_[mt][n], fq, be[i][2 * n], be[i][2 * n + 1]);
              }
            }
        }
      }
      float rows[2][2] = {{0.f, 0.f}, {0.f, 0.f}}, cols[NJ][2], mp = 0.f, ma = 0.f;
#pragma unroll
      for (int n = 0; n < NJ; ++n) cols[n][0] = cols[n][1] = 0.f;
      const float kk2 = ki * ki, qk2 = qi * ki, sP = a.scale * iO * iE, sN = iY * iE;
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int n = 0; n < NJ; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = 32 * rg + 16 * mt + 8 * (e >> 1) + r, j = 8 * (NJ * cq + n) + cc + (e & 1);
            const float Db = j <= i ? __expf((sm.Gh[i] - sm.Gh[j]) + (sm.Gl[i] - sm.Gl[j])) * sm.beta[j] : 0.f;
            const float nn = N[mt][n][e] * sN;
            const float wp = Db * (Pm[mt][n][e] * sP);
            const float wa = j < i ? -Db * sm.beta[i] * nn : 0.f;
            if (i == j && i < nt)
              static_cast<__nv_bfloat16*>(p.dbeta)[a.row(cur.b, t0 + i) * a.Hv + h] = __float2bfloat16_rn(nn);
            Pm[mt][n][e] = wp;
            N[mt][n][e] = wa;
            mp = fmaxf(mp, fabsf(wp));
            ma = fmaxf(ma, fabsf(wa));
            const float x = wp * (qk_[mt][n][e] * qk2) + wa * (kk_[mt][n][e] * kk2);
            rows[mt][e >> 1] += x;
            cols[n][e & 1] += x;
          }
      mp = warp_max(mp);
      ma = warp_max(ma);
      float frob = (frob2.x + frob2.y) * iS * iD;
#pragma unroll
      for (int w = 16; w; w >>= 1) frob += __shfl_xor_sync(kFull, frob, w);
      if (lane == 0) {
        sm.mx[0][warp] = mp;
        sm.mx[1][warp] = ma;
        sm.red[warp] = frob;
      }
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float ow = own[mt][half].x + own[mt][half].y, th = thru[mt][half].x + thru[mt][half].y;
#pragma unroll
          for (int w = 1; w < 4; w <<= 1) {
            rows[mt][half] += __shfl_xor_sync(kFull, rows[mt][half], w);
            ow += __shfl_xor_sync(kFull, ow, w);
            th += __shfl_xor_sync(kFull, th, w);
          }
          if ((lane & 3) == 0) {
            const int i = 32 * rg + 16 * mt + 8 * half + r;
            sm.row[cq][i] = rows[mt][half];
            sm.own[cq][i] = ow;
            sm.thru[cq][i] = th;
          }
        }
#pragma unroll
      for (int n = 0; n < NJ; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) cols[n][e] += __shfl_xor_sync(kFull, cols[n][e], w);
          if (lane < 4) sm.col[rg][8 * (NJ * cq + n) + cc + e] = cols[n][e];
        }
      __syncthreads();
      mp = warp_max(sm.mx[0][lane % NW]);
      ma = warp_max(sm.mx[1][lane % NW]);
      const float pf = up_scale(mp), af = up_scale(ma);
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int n = 0; n < NJ; ++n)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int i = 32 * rg + 16 * mt + 8 * half + r;
            const uint32_t at = swz<128>(i, NJ * cq + n) + 2 * cc;
            *reinterpret_cast<uint32_t*>(sm.mP + at) = pack_h(Pm[mt][n][2 * half] * pf, Pm[mt][n][2 * half + 1] * pf);
            *reinterpret_cast<uint32_t*>(sm.mA + at) = pack_h(N[mt][n][2 * half] * af, N[mt][n][2 * half + 1] * af);
          }
      if (tid < kTc) {
        // dG of a token, and its part of <S1, dS1>
        float x = -(sm.col[0][tid] + sm.col[1][tid]), th = 0.f;
#pragma unroll
        for (int q = 0; q < CQ; ++q) {
          x += sm.row[q][tid] + sm.own[q][tid];
          th += sm.thru[q][tid];
        }
        sm.dG[tid] = x - th;
        sm.w[tid] = th;
      }
      if (warp == 2) {
        for (int t = max(nt, 0) + lane; t < min(kTc, a.T - t0); t += 32) {
          static_cast<__nv_bfloat16*>(p.dg)[a.row(cur.b, t0 + t) * a.Hv + h] = __float2bfloat16_rn(0.f);
          static_cast<__nv_bfloat16*>(p.dbeta)[a.row(cur.b, t0 + t) * a.Hv + h] = __float2bfloat16_rn(0.f);
        }
      }
      __syncthreads();
      if (warp == NW - 1) {
        // dg: suffix sums of dG, two tokens a lane
        const float2 x = *reinterpret_cast<const float2*>(sm.dG + 2 * lane), w2 = *reinterpret_cast<const float2*>(sm.w + 2 * lane);
        float w = w2.x + w2.y, f = lane < NW ? sm.red[lane] : 0.f, pair = x.x + x.y;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
          const float dn = __shfl_down_sync(kFull, pair, k);
          if (lane + k < 32) pair += dn;
          w += __shfl_xor_sync(kFull, w, k);
          f += __shfl_xor_sync(kFull, f, k);
        }
        const float last = w + sc[kScEnd] * f;
        const float out[2] = {pair + last, pair - x.x + last};
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (2 * lane + e < nt)
            static_cast<__nv_bfloat16*>(p.dg)[a.row(cur.b, t0 + 2 * lane + e) * a.Hv + h] = __float2bfloat16_rn(out[e]);
      }
      const uint32_t mPs = smem_u32(sm.mP), mAs = smem_u32(sm.mA);
      // x += M B with M taken as stored (rows i) or transposed (rows j)
      auto pairs = [&](float (&x)[2][2][4], uint32_t M, uint32_t B, bool trans) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          uint32_t bb[4];
          load_b_rows_k<PK>(bb, B, cq * 16, kk, lane);
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            const int blk = 2 * rg + mt, m0 = 16 * blk;          // 16-blocks on the far side of the diagonal are zero
            if (trans ? kk < blk : kk > blk) continue;
            uint32_t fa[4];
            if (trans)
              ldsm_t(fa, M + swz<128>(16 * kk + (lane & 7) + ((lane >> 4) << 3), (m0 >> 3) + ((lane >> 3) & 1)));
            else
              ldsm(fa, M + swz<128>(m0 + (lane & 15), 2 * kk + (lane >> 4)));
            mma_h(x[mt][0], fa, bb[0], bb[1]);
            mma_h(x[mt][1], fa, bb[2], bb[3]);
          }
        }
      };
      auto clear = [&](float (&x)[2][2][4]) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[mt][n][e] = 0.f;
      };
      auto add = [&](float (&acc)[2][2][4], const float (&x)[2][2][4], float f) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int n = 0; n < 2; ++n)
            set4(acc[mt][n], fma2(lo2(x[mt][n]), both(f), lo2(acc[mt][n])), fma2(hi2(x[mt][n]), both(f), hi2(acc[mt][n])));
      };
      clear(t_[0]);
      clear(t_[1]);
      clear(t_[2]);
      pairs(t_[0], mPs, ks, false);
      pairs(t_[1], mPs, qs, true);
      pairs(t_[2], mAs, ks, false);
      pairs(t_[2], mAs, ks, true);
      add(dq, t_[0], inv_scale(pf) * ki);
      add(dk, t_[1], inv_scale(pf) * qi);
      add(dk, t_[2], inv_scale(af) * ki);
      if (cur.hh == per - 1) {
        // masked rows are zeros, whatever the sums hold: a NaN in a token reaches them as a product with zero
        if (nt < kTc) {
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (32 * rg + 16 * mt + 8 * (e >> 1) + r >= nt) dq[mt][0][e] = dq[mt][1][e] = dk[mt][0][e] = dk[mt][1][e] = 0.f;
        }
        // lanes of a quad swap halves, so that each writes 8 bytes of one tile
        const bool odd = lane & 1;
        const int col = cq * 16 + (odd ? 8 : 0) + 2 * (cc & 4 ? 2 : 0);
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int t = t0 + 32 * rg + 16 * mt + 8 * half + r;
            const int64_t at = t < a.T ? a.row(cur.b, t) * qk_row + cur.hk * DK + col : 0;
            auto write = [&](void* out, const float (&x)[2][2][4]) {
              const uint32_t w0 = pack_b(x[mt][0][2 * half], x[mt][0][2 * half + 1]), w1 = pack_b(x[mt][1][2 * half], x[mt][1][2 * half + 1]);
              const uint32_t got = __shfl_xor_sync(kFull, odd ? w0 : w1, 1);
              if (t < a.T)
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) = odd ? make_uint2(got, w1) : make_uint2(w0, got);
            };
            write(p.dq, dq);
            write(p.dk, dk);
          }
      }
    }
    __syncthreads();              // everyone is done with this stage (and with the head's shared sums)
    cur = nxt;
    stage ^= 1;
    kq = nkq;
  }
}

template <int DK>
int backward(const DeltaTcBwdArgs& t, cudaStream_t s, int* launches) {
  const int gsm = sizeof(GradSmem<DK>);
  const int w = scan_slices(t.a, t.num_sms, kScanReverse);
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(t.a.B) * t.a.Hv * (t.a.Dv / (16 * w)));
  if constexpr (DK == 128)
    if (w == 8) delta_scan_bwd_kernel<DK, 8><<<grid, 256, sizeof(ScanSmem<DK, 8>), s>>>(t);
  if (w == 4) delta_scan_bwd_kernel<DK, 4><<<grid, 128, sizeof(ScanSmem<DK, 4>), s>>>(t);
  if (w == 2) delta_pair_bwd_kernel<DK><<<grid, 128, sizeof(PairSmem<DK>), s>>>(t);
  int rc = check_launch();
  if (rc) return rc;
  ++*launches;
  const int64_t items = static_cast<int64_t>(t.a.B) * t.a.Hk * ((t.a.T + kTc - 1) / kTc);
  delta_grad_kernel<DK><<<static_cast<unsigned>(items < t.num_sms ? items : t.num_sms), GradSmem<DK>::NT, gsm, s>>>(t);
  rc = check_launch();
  if (!rc) ++*launches;
  return rc;
}

template <int DK, int W>
int init_scans() {
  const int smem = sizeof(ScanSmem<DK, W>);
  return set_smem(delta_scan_fwd_kernel<DK, false, W>, smem) || set_smem(delta_scan_fwd_kernel<DK, true, W>, smem) ||
         set_smem(delta_scan_bwd_kernel<DK, W>, smem);
}
int init_wide() { return init_scans<128, 8>(); }
template <int DK>
int init() {
  const int gsm = sizeof(GradSmem<DK>);
  return set_smem(delta_prep_kernel<DK, false>, sizeof(PrepSmem<DK, false>)) ||
                 set_smem(delta_prep_kernel<DK, true>, sizeof(PrepSmem<DK, true>)) ||
                 init_scans<DK, 4>() || (DK == 128 && init_wide()) || set_smem(delta_grad_kernel<DK>, gsm) ||
                 set_smem(delta_pair_fwd_kernel<DK, false>, sizeof(PairSmem<DK>)) ||
                 set_smem(delta_pair_fwd_kernel<DK, true>, sizeof(PairSmem<DK>)) || set_smem(delta_pair_bwd_kernel<DK>, sizeof(PairSmem<DK>))
             ? RNN_CUDA_ERROR
             : 0;
}

}  // namespace

int delta_tc_init(int Dk) { return Dk == 64 ? init<64>() : init<128>(); }

bool delta_tc_supported(int Dk, int Dv, int is_bf16) { return is_bf16 && (Dk == 64 || Dk == 128) && Dv % 32 == 0; }

int launch_delta_tc_forward(const DeltaTcArgs& t, cudaStream_t s, int* launches) {
  *launches = 0;
  if (t.a.Dk == 64) return t.train ? forward<64, true>(t, s, launches) : forward<64, false>(t, s, launches);
  return t.train ? forward<128, true>(t, s, launches) : forward<128, false>(t, s, launches);
}

int launch_delta_tc_backward(const DeltaTcBwdArgs& t, cudaStream_t s, int* launches) {
  *launches = 0;
  return t.a.Dk == 64 ? backward<64>(t, s, launches) : backward<128>(t, s, launches);
}

}  // namespace rnn
