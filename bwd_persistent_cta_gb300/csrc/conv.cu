// conv.cu - the causal convolution over time: whole sequences forward and
// backward, and the serving step.
//
// A thread has 8 channels and walks a stretch of tokens with the last W inputs in
// registers, so each input is read once from memory (and W - 1 times more at the
// start of a stretch, mostly from L2).
#include "common.cuh"
#include "conv.h"
#include "pair.cuh"
#include "vec.cuh"

namespace rnn {

namespace {

constexpr int kThreads = 128;
constexpr int kStretch = 32;      // tokens a thread

template <typename T>
__device__ __forceinline__ float2 sigm2(float2 v) {
  if constexpr (sizeof(T) == 2)
    return make_float2(__fdividef(1.f, 1.f + __expf(-v.x)), __fdividef(1.f, 1.f + __expf(-v.y)));
  else
    return make_float2(sigm(v.x), sigm(v.y));
}

// The taps of a thread's 8 channels, [channels, W] in memory, as pairs of channels.
template <typename T, int W>
__device__ __forceinline__ void load_taps(float2 (&w)[W][4], const void* base, int64_t d) {
  const T* p = static_cast<const T*>(base) + d * W;
#pragma unroll
  for (int k = 0; k < W; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) w[k][j] = make_float2(to_f(p[2 * j * W + k]), to_f(p[(2 * j + 1) * W + k]));
}
template <typename T>
__device__ __forceinline__ void unpack(float2 (&v)[4], const Raw<T, 8>& r) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = r.pair(j);
}

// Where the input of extended row e (e - (W - 1) is its token) lies: the state's rows
// come first.
template <typename T, int W>
__device__ __forceinline__ void load_input(Raw<T, 8>& r, const ConvArgs& a, const void* s0, int b, int e, int len, int d) {
  const int t = e - (W - 1);
  if (t >= 0) load_or<T, 8>(r, a.x, t < len ? a.row(b, t) * a.x_row + d : 0, t < len, 0.f);
  else load_or<T, 8>(r, s0, (static_cast<int64_t>(b) * (W - 1) + e) * a.D + d, s0 != nullptr, 0.f);
}

struct Spot {
  int b, seg, d;
  bool in;
  __device__ __forceinline__ Spot(const ConvArgs& a) {
    const int per = (a.D / 8 + kThreads - 1) / kThreads, segs = (a.T + kStretch - 1) / kStretch;
    const int c = blockIdx.x % per, r = blockIdx.x / per;
    seg = r % segs;
    b = r / segs;
    d = (c * kThreads + threadIdx.x) * 8;
    in = d < a.D;
  }
};

template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_fwd_kernel(const ConvFwdArgs f) {
  const ConvArgs& a = f.a;
  const Spot p(a);
  if (!p.in) return;
  const int len = a.len ? a.len[p.b] : a.T, t0 = p.seg * kStretch;
  const int t1 = t0 + kStretch < a.T ? t0 + kStretch : a.T;
  float2 w[W][4], bias[4], win[W][4];
  load_taps<T, W>(w, a.w, p.d);
  Raw<T, 8> r;
  load_or<T, 8>(r, a.bias, p.d, a.bias != nullptr, 0.f);
  unpack<T>(bias, r);
#pragma unroll
  for (int k = 1; k < W; ++k) {
    load_input<T, W>(r, a, f.s0, p.b, t0 + k - 1, len, p.d);
    unpack<T>(win[k], r);
  }
  // the state out before anything else is written: sT may be s0
  if (p.seg == 0 && f.sT) {
    Raw<T, 8> q[W - 1];
#pragma unroll
    for (int k = 0; k < W - 1; ++k) load_input<T, W>(q[k], a, f.s0, p.b, len + k, len, p.d);
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
      *reinterpret_cast<Raw<T, 8>*>(static_cast<T*>(f.sT) + (static_cast<int64_t>(p.b) * (W - 1) + k) * a.D + p.d) = q[k];
  }
#pragma unroll 8
  for (int t = t0; t < t1; ++t) {
    load_or<T, 8>(r, a.x, t < len ? a.row(p.b, t) * a.x_row + p.d : 0, t < len, 0.f);
    float2 v[4];
#pragma unroll
    for (int k = 0; k + 1 < W; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) win[k][j] = win[k + 1][j];
    unpack<T>(win[W - 1], r);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = bias[j];
#pragma unroll
      for (int k = 0; k < W; ++k) v[j] = fma2(w[k][j], win[k][j], v[j]);
      if (a.silu) v[j] = mul2(v[j], sigm2<T>(v[j]));
      if (t >= len) v[j] = both(0.f);
    }
    store_vec<T, 8>(static_cast<T*>(f.y) + a.row(p.b, t) * a.D + p.d, v);
  }
}

// The gradients.  With dp_t = dy_t act'(pre_t): walking t forward, the last W values of
// dp give sum_k w[k] dp_{t-k}, the gradient of extended row t (a row of the state for
// t < W - 1, else token t - (W - 1)); x's window gives dw.
template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_bwd_kernel(const ConvBwdArgs g) {
  const ConvArgs& a = g.a;
  const Spot p(a);
  if (!p.in) return;
  const int len = a.len ? a.len[p.b] : a.T, t0 = p.seg * kStretch;
  const int t1 = t0 + kStretch < a.T ? t0 + kStretch : a.T;
  float2 w[W][4], bias[4], win[W][4], dp[W][4], dw[W][4], db[4];
  load_taps<T, W>(w, a.w, p.d);
  Raw<T, 8> r;
  load_or<T, 8>(r, a.bias, p.d, a.bias != nullptr, 0.f);
  unpack<T>(bias, r);
#pragma unroll
  for (int k = 0; k < W; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j) win[k][j] = dp[k][j] = dw[k][j] = db[j] = both(0.f);
#pragma unroll
  for (int k = 1; k < W; ++k) {
    load_input<T, W>(r, a, g.s0, p.b, t0 + k - 1, len, p.d);
    unpack<T>(win[k], r);
  }
#pragma unroll 4
  for (int t = t0; t < t1 + W - 1; ++t) {
    Raw<T, 8> rx, ry;
    const bool ok = t < len;
    load_or<T, 8>(rx, a.x, ok ? a.row(p.b, t) * a.x_row + p.d : 0, ok, 0.f);
    load_or<T, 8>(ry, g.dy, ok ? a.row(p.b, t) * a.D + p.d : 0, ok, 0.f);
#pragma unroll
    for (int k = 0; k + 1 < W; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        win[k][j] = win[k + 1][j];
        dp[W - 1 - k][j] = dp[W - 2 - k][j];
      }
    unpack<T>(win[W - 1], rx);
    unpack<T>(dp[0], ry);
    float2 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (a.silu) {
        float2 q = bias[j];
#pragma unroll
        for (int k = 0; k < W; ++k) q = fma2(w[k][j], win[k][j], q);
        const float2 s = sigm2<T>(q);
        // s + q s (1 - s)
        dp[0][j] = mul2(dp[0][j], fma2(mul2(q, s), make_float2(1.f - s.x, 1.f - s.y), s));
      }
      if (!ok) dp[0][j] = both(0.f);
      if (t < t1) {
#pragma unroll
        for (int k = 0; k < W; ++k)
          if (ok) dw[k][j] = fma2(dp[0][j], win[k][j], dw[k][j]);
        db[j] = add2(db[j], dp[0][j]);
      }
      v[j] = both(0.f);
#pragma unroll
      for (int k = 0; k < W; ++k) v[j] = fma2(w[k][j], dp[k][j], v[j]);
    }
    // extended row t of the state's gradient out
    if (t >= len && t < len + W - 1 && g.dsT) {
      load_or<T, 8>(r, g.dsT, (static_cast<int64_t>(p.b) * (W - 1) + t - len) * a.D + p.d, true, 0.f);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = add2(v[j], r.pair(j));
    }
    if (t >= t0 + W - 1) {
      const int s = t - (W - 1);
      if (s >= len)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = both(0.f);
      if (g.dx) store_vec<T, 8>(static_cast<T*>(g.dx) + a.row(p.b, s) * a.D + p.d, v);
    } else if (p.seg == 0 && g.ds0) {
      store_vec<T, 8>(static_cast<T*>(g.ds0) + (static_cast<int64_t>(p.b) * (W - 1) + t) * a.D + p.d, v);
    }
  }
  if (!g.partial) return;
  float* out = g.partial + (static_cast<int64_t>(p.b) * ((a.T + kStretch - 1) / kStretch) + p.seg) * (W + 1) * a.D + p.d;
#pragma unroll
  for (int k = 0; k < W; ++k) store_vec<float, 8>(out + static_cast<int64_t>(k) * a.D, dw[k]);
  store_vec<float, 8>(out + static_cast<int64_t>(W) * a.D, db);
}

// dw[d][k] and dbias[d]: the sums over the stretches, each of 8 groups in order and
// then the groups in order; 32 channels of one tap a block.
__global__ void __launch_bounds__(256) conv_reduce_kernel(const float* partial, int parts, int D, int W, float* dw,
                                                          float* dbias) {
  __shared__ float sm[8][32];
  const int k = blockIdx.y, c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
  float s = 0.f;
  if (c < D)
    for (int i = g; i < parts; i += 8) s += partial[(static_cast<int64_t>(i) * (W + 1) + k) * D + c];
  sm[g][threadIdx.x & 31] = s;
  __syncthreads();
  if (g || c >= D) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += sm[i][threadIdx.x];
  if (k < W && dw) dw[static_cast<int64_t>(c) * W + k] = s;
  if (k == W && dbias) dbias[c] = s;
}

template <typename T, int W>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const ConvStepArgs p) {
  const ConvArgs& a = p.a;
  const int per = (a.D / 8 + kThreads - 1) / kThreads, b = blockIdx.x / per;
  const int d = ((blockIdx.x - b * per) * kThreads + threadIdx.x) * 8;
  if (d >= a.D) return;
  const int slot = p.slots ? p.slots[b] : b;
  const bool live = slot >= 0 && slot < p.num_slots;
  const int len = live ? a.len ? a.len[b] : a.T : 0;
  T* st = static_cast<T*>(p.state) + static_cast<int64_t>(live ? slot : 0) * (W - 1) * a.D + d;
  float2 w[W][4], bias[4];
  Raw<T, 8> win[W];
  Raw<T, 8> r;
  if (len > 0) {
    load_taps<T, W>(w, a.w, d);
    load_or<T, 8>(r, a.bias, d, a.bias != nullptr, 0.f);
    unpack<T>(bias, r);
#pragma unroll
    for (int k = 1; k < W; ++k) win[k].load(st + static_cast<int64_t>(k - 1) * a.D);
  }
  for (int t = 0; t < a.T; ++t) {
    const int64_t at = a.row(b, t);
    float2 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = both(0.f);
    if (t < len) {
#pragma unroll
      for (int k = 0; k + 1 < W; ++k) win[k] = win[k + 1];
      win[W - 1].load(static_cast<const T*>(a.x) + at * a.x_row + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = bias[j];
#pragma unroll
        for (int k = 0; k < W; ++k) v[j] = fma2(w[k][j], win[k].pair(j), v[j]);
        if (a.silu) v[j] = mul2(v[j], sigm2<T>(v[j]));
      }
    }
    store_vec<T, 8>(static_cast<T*>(p.y) + at * a.D + d, v);
  }
  if (len > 0)
#pragma unroll
    for (int k = 1; k < W; ++k) *reinterpret_cast<Raw<T, 8>*>(st + static_cast<int64_t>(k - 1) * a.D) = win[k];
}

int check_launch() { return cudaGetLastError() == cudaSuccess ? 0 : RNN_CUDA_ERROR; }

int channel_ctas(const ConvArgs& a) { return (a.D / 8 + kThreads - 1) / kThreads; }
int stretches(const ConvArgs& a) { return (a.T + kStretch - 1) / kStretch; }
unsigned walk_ctas(const ConvArgs& a) {
  return static_cast<unsigned>(a.B) * stretches(a) * channel_ctas(a);
}

// CALL<type, width>(args)
#define RNN_CONV_WIDTHS(KERNEL, T, GRID, ARGS)                                          \
  switch ((ARGS).a.W) {                                                                 \
    case 2: KERNEL<T, 2><<<GRID, kThreads, 0, s>>>(ARGS); break;                        \
    case 3: KERNEL<T, 3><<<GRID, kThreads, 0, s>>>(ARGS); break;                        \
    default: KERNEL<T, 4><<<GRID, kThreads, 0, s>>>(ARGS);                              \
  }

}  // namespace

size_t conv_workspace_bytes(const ConvArgs& a) {
  return static_cast<size_t>(a.B) * stretches(a) * (a.W + 1) * a.D * 4;
}

int launch_conv_forward(const ConvFwdArgs& f, int is_bf16, cudaStream_t s) {
  if (is_bf16) RNN_CONV_WIDTHS(conv_fwd_kernel, __nv_bfloat16, walk_ctas(f.a), f)
  else RNN_CONV_WIDTHS(conv_fwd_kernel, float, walk_ctas(f.a), f)
  return check_launch();
}

int launch_conv_backward(const ConvBwdArgs& b, int is_bf16, cudaStream_t s, int* launches) {
  *launches = 0;
  if (is_bf16) RNN_CONV_WIDTHS(conv_bwd_kernel, __nv_bfloat16, walk_ctas(b.a), b)
  else RNN_CONV_WIDTHS(conv_bwd_kernel, float, walk_ctas(b.a), b)
  int rc = check_launch();
  if (rc) return rc;
  *launches = 1;
  if (!b.partial) return 0;
  conv_reduce_kernel<<<dim3((b.a.D + 31) / 32, b.a.W + 1), 256, 0, s>>>(b.partial, b.a.B * stretches(b.a), b.a.D, b.a.W,
                                                                        b.dw, b.dbias);
  if (!(rc = check_launch())) *launches = 2;
  return rc;
}

int launch_conv_step(const ConvStepArgs& p, int is_bf16, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(p.a.B) * channel_ctas(p.a);
  if (is_bf16) RNN_CONV_WIDTHS(conv_step_kernel, __nv_bfloat16, grid, p)
  else RNN_CONV_WIDTHS(conv_step_kernel, float, grid, p)
  return check_launch();
}

}  // namespace rnn
