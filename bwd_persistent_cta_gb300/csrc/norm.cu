// norm.cu - the block norm: RMS norm of a block's output, its gate, the scaled
// residual and the next block's RMS norm in one pass over the rows, and the
// gradients of all of it in another.
#include "common.cuh"
#include "norm.h"

namespace rnn {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kVec = 8;        // elements a thread moves at a time (16 bytes of bf16)
constexpr int kBlock = 256;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[kVec]) {
  if constexpr (sizeof(T) == 2) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  } else {
    const float4 q0 = reinterpret_cast<const float4*>(p)[0], q1 = reinterpret_cast<const float4*>(p)[1];
    v[0] = q0.x; v[1] = q0.y; v[2] = q0.z; v[3] = q0.w;
    v[4] = q1.x; v[5] = q1.y; v[6] = q1.z; v[7] = q1.w;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[kVec]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}
template <typename T>
__device__ __forceinline__ void load8_or(const T* p, bool ok, float other, float (&v)[kVec]) {
  if (ok) {
    load8<T>(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = other;
  }
}

// Sums N values over the TPR consecutive threads of a row; every thread gets
// the sums.  Rows wider than a warp go through shared memory, ``red`` holding
// one value per warp and sum; consecutive calls alternate ``red`` buffers, so
// one barrier a call is enough.
template <int TPR, int N>
__device__ __forceinline__ void row_sum(float (&v)[N], float* red) {
#pragma unroll
  for (int w = 1; w < (TPR < 32 ? TPR : 32); w <<= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(kFull, v[n], w);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int warp = threadIdx.x >> 5, first = warp / W * W;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int n = 0; n < N; ++n) red[warp * N + n] = v[n];
    __syncthreads();
#pragma unroll
    for (int n = 0; n < N; ++n) {
      v[n] = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) v[n] += red[(first + w) * N + n];
    }
  }
}

struct Gate {
  float f, d;
};
// act(z) and its derivative.
__device__ __forceinline__ Gate gate_of(int kind, float z) {
  if (kind == RNN_GATE_NONE) return {1.f, 0.f};
  const float s = sigm(z);
  if (kind == RNN_GATE_SIGMOID) return {s, s * (1.f - s)};
  return {z * s, s * (1.f + z * (1.f - s))};
}

// TPR threads a row, IT vectors of 8 a thread: cols <= TPR * IT * 8.  The row
// stays in registers between the two norms, so each stream is moved once.
template <typename T, int TPR, int IT>
__global__ void __launch_bounds__(TPR > kBlock ? TPR : kBlock) norm_fwd_kernel(const NormArgs a) {
  constexpr int RPB = (TPR > kBlock ? TPR : kBlock) / TPR;
  __shared__ float red[2][32];
  const int l = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * RPB + sub;
  const int64_t total = static_cast<int64_t>(a.rows) * a.groups;
  const bool live = item < total;
  const int64_t row = live ? item / a.groups : 0;
  const int64_t off = live ? (item - row * a.groups) * a.cols : 0;
  const int64_t dense = row * a.groups * a.cols + off;
  float v[IT][kVec], xr[IT][kVec], zr[IT][kVec];
  float s1[1] = {0.f};
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int c = (i * TPR + l) * kVec;
    const bool ok = live && c < a.cols;
    load8_or<T>(static_cast<const T*>(a.y) + row * a.y_row + off + c, ok, 0.f, v[i]);
    load8_or<T>(static_cast<const T*>(a.z) + row * a.z_row + off + c, ok && a.gate != RNN_GATE_NONE, 0.f, zr[i]);
    load8_or<T>(static_cast<const T*>(a.x) + row * a.x_row + off + c, ok && a.residual, 0.f, xr[i]);
#pragma unroll
    for (int j = 0; j < kVec; ++j) s1[0] = fmaf(v[i][j], v[i][j], s1[0]);
  }
  float r1 = 1.f;
  if (a.norm_in) {
    row_sum<TPR, 1>(s1, red[0]);
    r1 = rsqrtf(s1[0] / a.cols + a.eps);
  }
  float s2[1] = {0.f};
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int c = (i * TPR + l) * kVec;
    const bool ok = live && c < a.cols;
    float w[kVec], sc[kVec];
    load8_or<T>(static_cast<const T*>(a.w_in) + c, ok && a.norm_in && a.w_in, 1.f, w);
    load8_or<T>(static_cast<const T*>(a.scale) + c, ok && a.residual && a.scale, 1.f, sc);
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      const float b = v[i][j] * r1 * w[j] * gate_of(a.gate, zr[i][j]).f;
      v[i][j] = a.residual ? fmaf(sc[j], b, xr[i][j]) : b;
      if (!ok) v[i][j] = 0.f;
      s2[0] = fmaf(v[i][j], v[i][j], s2[0]);
    }
    if (ok) store8<T>(static_cast<T*>(a.x_out) + dense + c, v[i]);
  }
  if (!a.norm_out) return;
  row_sum<TPR, 1>(s2, red[1]);
  const float r2 = rsqrtf(s2[0] / a.cols + a.eps);
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int c = (i * TPR + l) * kVec;
    if (!live || c >= a.cols) continue;
    float w[kVec];
    load8_or<T>(static_cast<const T*>(a.w_out) + c, a.w_out != nullptr, 1.f, w);
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[i][j] *= r2 * w[j];
    store8<T>(static_cast<T*>(a.n_out) + dense + c, v[i]);
  }
}

// The gradients.  With r1, r2 the two inverse root means, h = dn * w_out:
//   dc = dx' + r2 h - x' r2^3 mean(h x')                 (dx = dc)
//   dw_out += dn x' r2,  dscale += dc b,  db = scale dc
//   dz = db a act'(z),  da = db act(z),  dw_in += da y r1
//   dy = r1 (da w_in) - y r1^3 mean(da w_in y)
// x' is recomputed from the inputs, not read back rounded, so that the weights'
// fp32 gradients carry no bf16 rounding.  A CTA walks rows with a stride and
// keeps its columns' weight gradients in registers; the CTAs' partial sums are
// added by a second kernel in a fixed order.
template <typename T, int TPR, int IT>
__global__ void __launch_bounds__(TPR > kBlock ? TPR : kBlock) norm_bwd_kernel(const NormArgs a) {
  constexpr int NT = TPR > kBlock ? TPR : kBlock, RPB = NT / TPR;
  __shared__ float red[4][64];              // [1] and [3] alternate: without norm_in that sum is a row's only barrier
  extern __shared__ float fold[];           // [RPB][cols] when RPB > 1
  int odd = 0;
  const int l = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int64_t total = static_cast<int64_t>(a.rows) * a.groups;
  const float inv = 1.f / a.cols;
  float gw[3][IT][kVec];
#pragma unroll
  for (int w = 0; w < 3; ++w)
#pragma unroll
    for (int i = 0; i < IT; ++i)
#pragma unroll
      for (int j = 0; j < kVec; ++j) gw[w][i][j] = 0.f;

  for (int64_t base = static_cast<int64_t>(blockIdx.x) * RPB; base < total; base += static_cast<int64_t>(gridDim.x) * RPB) {
    const int64_t item = base + sub;
    const bool live = item < total;
    const int64_t row = live ? item / a.groups : 0;
    const int64_t off = live ? (item - row * a.groups) * a.cols : 0;
    const int64_t dense = row * a.groups * a.cols + off;
    float y[IT][kVec], z[IT][kVec], c_[IT][kVec], d[IT][kVec], dn[IT][kVec];
    float s1[1] = {0.f};
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * TPR + l) * kVec;
      const bool ok = live && c < a.cols;
      load8_or<T>(static_cast<const T*>(a.y) + row * a.y_row + off + c, ok, 0.f, y[i]);
      load8_or<T>(static_cast<const T*>(a.z) + row * a.z_row + off + c, ok && a.gate != RNN_GATE_NONE, 0.f, z[i]);
      load8_or<T>(static_cast<const T*>(a.x) + row * a.x_row + off + c, ok && a.residual && a.norm_out, 0.f, c_[i]);
      load8_or<T>(static_cast<const T*>(a.dx_out) + dense + c, ok && a.dx_out, 0.f, d[i]);
      load8_or<T>(static_cast<const T*>(a.dn_out) + dense + c, ok && a.norm_out && a.dn_out, 0.f, dn[i]);
#pragma unroll
      for (int j = 0; j < kVec; ++j) s1[0] = fmaf(y[i][j], y[i][j], s1[0]);
    }
    float r1 = 1.f;
    if (a.norm_in) {
      row_sum<TPR, 1>(s1, red[0]);
      r1 = rsqrtf(s1[0] * inv + a.eps);
    }
    float s2[2] = {0.f, 0.f}, r2 = 0.f, m2 = 0.f;
    if (a.norm_out) {
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int c = (i * TPR + l) * kVec;
        const bool ok = live && c < a.cols;
        float w[kVec], sc[kVec], wo[kVec];
        load8_or<T>(static_cast<const T*>(a.w_in) + c, ok && a.norm_in && a.w_in, 1.f, w);
        load8_or<T>(static_cast<const T*>(a.scale) + c, ok && a.residual && a.scale, 1.f, sc);
        load8_or<T>(static_cast<const T*>(a.w_out) + c, ok && a.w_out, 1.f, wo);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const float b = y[i][j] * r1 * w[j] * gate_of(a.gate, z[i][j]).f;
          c_[i][j] = a.residual ? fmaf(sc[j], b, c_[i][j]) : b;
          s2[0] = fmaf(c_[i][j], c_[i][j], s2[0]);
          s2[1] = fmaf(dn[i][j] * wo[j], c_[i][j], s2[1]);
        }
      }
      row_sum<TPR, 2>(s2, red[1 + 2 * odd]);
      odd ^= 1;
      r2 = rsqrtf(s2[0] * inv + a.eps);
      m2 = r2 * r2 * r2 * s2[1] * inv;
    }
    float s3[1] = {0.f};
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * TPR + l) * kVec;
      const bool ok = live && c < a.cols;
      float w[kVec], sc[kVec], wo[kVec], dz[kVec];
      load8_or<T>(static_cast<const T*>(a.w_in) + c, ok && a.norm_in && a.w_in, 1.f, w);
      load8_or<T>(static_cast<const T*>(a.scale) + c, ok && a.residual && a.scale, 1.f, sc);
      load8_or<T>(static_cast<const T*>(a.w_out) + c, ok && a.norm_out && a.w_out, 1.f, wo);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        float dc = d[i][j];
        if (a.norm_out) {
          dc += fmaf(r2 * dn[i][j], wo[j], -c_[i][j] * m2);
          gw[2][i][j] = fmaf(dn[i][j] * r2, c_[i][j], gw[2][i][j]);
        }
        const Gate gt = gate_of(a.gate, z[i][j]);
        const float yn = y[i][j] * r1;
        const float av = yn * w[j];
        d[i][j] = dc;                                     // dx
        const float db = a.residual ? dc * sc[j] : dc;
        gw[1][i][j] = fmaf(dc, av * gt.f, gw[1][i][j]);
        dz[j] = db * av * gt.d;
        const float da = db * gt.f;
        gw[0][i][j] = fmaf(da, yn, gw[0][i][j]);
        dn[i][j] = da * w[j];                             // gradient of the normalised y
        s3[0] = fmaf(dn[i][j], y[i][j], s3[0]);
      }
      if (ok && a.dx) store8<T>(static_cast<T*>(a.dx) + dense + c, d[i]);
      if (ok && a.dz) store8<T>(static_cast<T*>(a.dz) + dense + c, dz);
    }
    float m1 = 0.f;
    if (a.norm_in) {
      row_sum<TPR, 1>(s3, red[2]);
      m1 = r1 * r1 * r1 * s3[0] * inv;
    }
    if (a.dy) {
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int c = (i * TPR + l) * kVec;
        if (!live || c >= a.cols) continue;
        float o[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) o[j] = fmaf(r1, dn[i][j], -y[i][j] * m1);
        store8<T>(static_cast<T*>(a.dy) + dense + c, o);
      }
    }
  }
  if (!a.partial) return;
#pragma unroll
  for (int w = 0; w < 3; ++w) {
    float* out = a.partial + (static_cast<int64_t>(w) * gridDim.x + blockIdx.x) * a.cols;
    if constexpr (RPB == 1) {
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int c = (i * TPR + l) * kVec;
        if (c < a.cols) store8<float>(out + c, gw[w][i]);
      }
    } else {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int c = (i * TPR + l) * kVec;
        if (c < a.cols) store8<float>(fold + sub * a.cols + c, gw[w][i]);
      }
      __syncthreads();
      for (int c = threadIdx.x; c < a.cols; c += NT) {
        float s = 0.f;
        for (int r = 0; r < RPB; ++r) s += fold[r * a.cols + c];
        out[c] = s;
      }
    }
  }
}

// dw[w][c] = sum over CTAs of partial[w][cta][c], in CTA order per lane group:
// 32 columns x 8 groups of CTAs a block.
__global__ void __launch_bounds__(256) norm_reduce_kernel(const float* partial, int ctas, int cols, float* d0,
                                                          float* d1, float* d2) {
  __shared__ float sm[8][33];
  const int w = blockIdx.y;
  float* out = w == 0 ? d0 : w == 1 ? d1 : d2;
  if (!out) return;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
  float s = 0.f;
  if (c < cols)
    for (int i = g; i < ctas; i += 8) s += partial[(static_cast<int64_t>(w) * ctas + i) * cols + c];
  sm[g][threadIdx.x & 31] = s;
  __syncthreads();
  if (g == 0 && c < cols) {
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sm[i][threadIdx.x];
    out[c] = s;
  }
}

int check_launch() { return cudaGetLastError() == cudaSuccess ? 0 : RNN_CUDA_ERROR; }

// Threads a row: one vector a thread up to 256 threads, then two (cols <= 8192).
struct Shape {
  int tpr, it;
};
Shape shape_of(int cols) {
  const int v = cols / kVec;
  if (v <= 8) return {8, 1};
  if (v <= 16) return {16, 1};
  if (v <= 32) return {32, 1};
  if (v <= 64) return {64, 1};
  if (v <= 128) return {128, 1};
  if (v <= 256) return {256, 1};
  if (v <= 512) return {256, 2};
  return {512, 2};
}
int rows_per_block(Shape s) { return s.tpr >= kBlock ? 1 : kBlock / s.tpr; }
// CTAs of the backward: enough to fill the GPU, each with rows to amortise its
// partial sums.
int bwd_ctas(const NormArgs& a) {
  const Shape s = shape_of(a.cols);
  const int64_t need = (static_cast<int64_t>(a.rows) * a.groups + rows_per_block(s) - 1) / rows_per_block(s);
  const int64_t most = static_cast<int64_t>(a.num_sms) * (s.tpr <= kBlock ? 4 : 1);
  return static_cast<int>(need < most ? need : most);
}

template <typename T, int TPR, int IT>
int fwd(const NormArgs& a, cudaStream_t s) {
  constexpr int NT = TPR > kBlock ? TPR : kBlock, RPB = NT / TPR;
  const int64_t n = static_cast<int64_t>(a.rows) * a.groups;
  norm_fwd_kernel<T, TPR, IT><<<static_cast<unsigned>((n + RPB - 1) / RPB), NT, 0, s>>>(a);
  return check_launch();
}
template <typename T, int TPR, int IT>
int bwd(const NormArgs& a, cudaStream_t s) {
  constexpr int NT = TPR > kBlock ? TPR : kBlock, RPB = NT / TPR;
  const size_t smem = RPB > 1 ? static_cast<size_t>(RPB) * a.cols * 4 : 0;
  norm_bwd_kernel<T, TPR, IT><<<bwd_ctas(a), NT, smem, s>>>(a);
  return check_launch();
}

#define RNN_NORM_SHAPES(CALL)                       \
  switch (sh.tpr) {                                 \
    case 8: return CALL(8, 1);                      \
    case 16: return CALL(16, 1);                    \
    case 32: return CALL(32, 1);                    \
    case 64: return CALL(64, 1);                    \
    case 128: return CALL(128, 1);                  \
    case 256: return sh.it == 1 ? CALL(256, 1) : CALL(256, 2); \
    default: return CALL(512, 2);                   \
  }

template <typename T>
int fwd_t(const NormArgs& a, cudaStream_t s) {
  const Shape sh = shape_of(a.cols);
#define RNN_NORM_FWD(TPR, IT) (fwd<T, TPR, IT>(a, s))
  RNN_NORM_SHAPES(RNN_NORM_FWD)
#undef RNN_NORM_FWD
}
template <typename T>
int bwd_t(const NormArgs& a, cudaStream_t s) {
  const Shape sh = shape_of(a.cols);
#define RNN_NORM_BWD(TPR, IT) (bwd<T, TPR, IT>(a, s))
  RNN_NORM_SHAPES(RNN_NORM_BWD)
#undef RNN_NORM_BWD
}

}  // namespace

size_t norm_workspace_bytes(const NormArgs& a) { return static_cast<size_t>(3) * bwd_ctas(a) * a.cols * 4; }

int launch_norm_forward(const NormArgs& a, int is_bf16, cudaStream_t s) {
  return is_bf16 ? fwd_t<__nv_bfloat16>(a, s) : fwd_t<float>(a, s);
}

int launch_norm_backward(const NormArgs& a, int is_bf16, cudaStream_t s, int* launches) {
  *launches = 0;
  int rc = is_bf16 ? bwd_t<__nv_bfloat16>(a, s) : bwd_t<float>(a, s);
  if (rc) return rc;
  *launches = 1;
  if (!a.partial) return 0;
  const dim3 grid((a.cols + 31) / 32, 3);
  norm_reduce_kernel<<<grid, 256, 0, s>>>(a.partial, bwd_ctas(a), a.cols, a.dw_in, a.dscale, a.dw_out);
  rc = check_launch();
  if (!rc) *launches = 2;
  return rc;
}

}  // namespace rnn
