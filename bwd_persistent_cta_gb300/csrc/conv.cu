// conv.cu - the causal convolution over time: whole sequences forward and
// backward, and the serving step.
//
// Memory bounds it.  A thread has 16 bytes of channels (forward; half as many backward in
// bf16, for the registers) and walks a stretch of 32 tokens with the last W inputs in
// registers, so each input is read once from memory (and W - 1 times more at the start
// of a stretch, mostly from L2); it loads four tokens while it works on the four before,
// since a store holds back the loads behind it.  A CTA has 128 channels of several
// stretches, whose sums for the weights' gradients it adds before they go to memory.
#include "common.cuh"
#include "conv.h"
#include "pair.cuh"
#include "vec.cuh"

#include <type_traits>

namespace rnn {

namespace {

constexpr int kThreads = 256, kStepThreads = 128;
constexpr int kStretch = 32;      // tokens a thread
constexpr int kSpan = 128;        // channels of a CTA; its threads of V channels have kThreads * V / kSpan stretches
constexpr int kAhead = 4;         // tokens loaded at once

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The sigmoid; with bf16 storage from the approximations, a few 2^-23 off.
template <typename T>
__device__ __forceinline__ float2 sigm2(float2 v) {
  if constexpr (sizeof(T) == 2) {
    const float2 q = mul2(v, both(-1.4426950408889634f)), d = add2(make_float2(ex2(q.x), ex2(q.y)), both(1.f));
    return make_float2(rcp(d.x), rcp(d.y));
  } else {
    return make_float2(sigm(v.x), sigm(v.y));
  }
}

// The taps of a thread's V channels, [channels, W] in memory, as pairs of channels.
template <typename T, int W, int V>
__device__ __forceinline__ void load_taps(float2 (&w)[W][V / 2], const void* base, int64_t d) {
  float f[V * W];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    Raw<T, V> r;
    r.load(static_cast<const T*>(base) + d * W + V * i);
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      f[V * i + 2 * j] = r.pair(j).x;
      f[V * i + 2 * j + 1] = r.pair(j).y;
    }
  }
#pragma unroll
  for (int k = 0; k < W; ++k)
#pragma unroll
    for (int j = 0; j < V / 2; ++j) w[k][j] = make_float2(f[2 * j * W + k], f[(2 * j + 1) * W + k]);
}
template <typename T, int V>
__device__ __forceinline__ void unpack(float2 (&v)[V / 2], const Raw<T, V>& r) {
#pragma unroll
  for (int j = 0; j < V / 2; ++j) v[j] = r.pair(j);
}
template <typename T, int V>
__device__ __forceinline__ void put(void* to, const Raw<T, V>& r) {
  float2 v[V / 2];
  unpack<T, V>(v, r);
  store_vec<T, V>(static_cast<T*>(to), v);
}

// Where the input of extended row e (e - (W - 1) is its token) lies: the state's rows
// come first.
template <typename T, int W, int V>
__device__ __forceinline__ void load_input(Raw<T, V>& r, const ConvArgs& a, const void* s0, int b, int e, int len, int d) {
  const int t = e - (W - 1);
  if (t >= 0) load_or<T, V>(r, a.x, t < len ? a.row(b, t) * a.x_row + d : 0, t < len, 0.f);
  else load_or<T, V>(r, s0, (static_cast<int64_t>(b) * (W - 1) + e) * a.D + d, s0 != nullptr, 0.f);
}

// A thread's channels and stretch; ``in`` is false beyond the last of either.
template <int V>
struct Spot {
  static constexpr int SIDE = kSpan / V, RUNS = kThreads / SIDE;
  int b, seg, d, part;                       // part: the CTA's place among those of its channels
  bool in;
  __host__ __device__ static int spans(const ConvArgs& a) { return (a.D + kSpan - 1) / kSpan; }
  // CTAs over the stretches of all sequences.
  __host__ __device__ static int parts(const ConvArgs& a) {
    const int64_t all = static_cast<int64_t>(a.B) * ((a.T + kStretch - 1) / kStretch);
    return static_cast<int>((all + RUNS - 1) / RUNS);
  }
  __device__ __forceinline__ Spot(const ConvArgs& a) {
    const int per = spans(a), segs = (a.T + kStretch - 1) / kStretch;
    part = blockIdx.x / per;
    const int64_t item = static_cast<int64_t>(part) * RUNS + threadIdx.x / SIDE;
    b = static_cast<int>(item / segs);
    seg = static_cast<int>(item - static_cast<int64_t>(b) * segs);
    d = (blockIdx.x - part * per) * kSpan + threadIdx.x % SIDE * V;
    in = d < a.D && b < a.B;
  }
};

// The forward.  8 x 1024 tokens of 4096 channels, four taps: bf16 33 us (4.1 TB/s), fp32
// 63 (4.2 TB/s).
template <typename T, int W, int V, bool SILU>
__global__ void __launch_bounds__(kThreads, 2) conv_fwd_kernel(const ConvFwdArgs f) {
  constexpr int U = kAhead, H = V / 2;
  const ConvArgs& a = f.a;
  const Spot<V> p(a);
  if (!p.in) return;
  const int len = a.len ? a.len[p.b] : a.T, t0 = p.seg * kStretch;
  const int t1 = t0 + kStretch < a.T ? t0 + kStretch : a.T, last = len < t1 ? len : t1;
  const int64_t hop = a.bfirst ? 1 : a.B, row0 = a.row(p.b, t0);
  const T* px = static_cast<const T*>(a.x) + row0 * a.x_row + p.d;
  T* py = static_cast<T*>(f.y) + row0 * a.D + p.d;
  Raw<T, V> r[U];
  auto load = [&](int t) {
#pragma unroll
    for (int i = 0; i < U; ++i) load_or<T, V>(r[i], px, i * hop * a.x_row, t + i < last, 0.f);
    px += U * hop * a.x_row;
  };
  float2 w[W][H], bias[H], win[W][H];
  Raw<T, V> q[W];
  load_or<T, V>(q[0], a.bias, p.d, a.bias != nullptr, 0.f);
#pragma unroll
  for (int k = 1; k < W; ++k) load_input<T, W, V>(q[k], a, f.s0, p.b, t0 + k - 1, len, p.d);
  load(t0);
  load_taps<T, W, V>(w, a.w, p.d);
  unpack<T, V>(bias, q[0]);
#pragma unroll
  for (int k = 1; k < W; ++k) unpack<T, V>(win[k], q[k]);
  // the state out after the state in, which it may be
  if (p.seg == 0 && f.sT) {
#pragma unroll
    for (int k = 0; k < W - 1; ++k) load_input<T, W, V>(q[k], a, f.s0, p.b, len + k, len, p.d);
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
      put<T, V>(static_cast<T*>(f.sT) + (static_cast<int64_t>(p.b) * (W - 1) + k) * a.D + p.d, q[k]);
  }
  for (int t = t0; t < t1; t += U) {
    Raw<T, V> x[U];
#pragma unroll
    for (int i = 0; i < U; ++i) x[i] = r[i];
    if (t + U < t1) load(t + U);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float2 v[H];
#pragma unroll
      for (int k = 0; k + 1 < W; ++k)
#pragma unroll
        for (int j = 0; j < H; ++j) win[k][j] = win[k + 1][j];
#pragma unroll
      for (int j = 0; j < H; ++j) {
        win[W - 1][j] = x[i].pair(j);
        v[j] = bias[j];
#pragma unroll
        for (int k = 0; k < W; ++k) v[j] = fma2(w[k][j], win[k][j], v[j]);
        if (SILU) v[j] = mul2(v[j], sigm2<T>(v[j]));
        if (t + i >= len) v[j] = both(0.f);
      }
      if (t + i < t1) store_vec<T, V>(py + i * hop * a.D, v);
    }
    py += U * hop * a.D;
  }
}

// The gradients.  With dp_t = dy_t act'(pre_t): walking t forward, the last W values of
// dp give sum_k w[k] dp_{t-k}, the gradient of extended row t (a row of the state for
// t < W - 1, else token t - (W - 1)); x's window gives dw.  8 x 1024 tokens of 4096
// channels, four taps: bf16 66 us (3.1 TB/s; issue of its 20 packed operations and one
// sigmoid an element bounds it, 54 % of the slots), fp32 123 (3.3 TB/s).
template <typename T, int W, int V, bool SILU>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 2 : 1) conv_bwd_kernel(const ConvBwdArgs g) {
  constexpr int U = kAhead, H = V / 2;
  __shared__ float fold[kThreads * V];
  const ConvArgs& a = g.a;
  const Spot<V> p(a);
  float2 dw[W + 1][H];                       // and the bias's
#pragma unroll
  for (int k = 0; k <= W; ++k)
#pragma unroll
    for (int j = 0; j < H; ++j) dw[k][j] = both(0.f);
  if (p.in) {
    const int len = a.len ? a.len[p.b] : a.T, t0 = p.seg * kStretch;
    const int t1 = t0 + kStretch < a.T ? t0 + kStretch : a.T, stop = t1 + W - 1, last = len < stop ? len : stop;
    const int64_t hop = a.bfirst ? 1 : a.B, row0 = a.row(p.b, t0);
    const T *px = static_cast<const T*>(a.x) + row0 * a.x_row + p.d, *pdy = static_cast<const T*>(g.dy) + row0 * a.D + p.d;
    Raw<T, V> rx[U], ry[U];
    auto load = [&](int t) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        load_or<T, V>(rx[i], px, i * hop * a.x_row, t + i < last, 0.f);
        load_or<T, V>(ry[i], pdy, i * hop * a.D, t + i < last, 0.f);
      }
      px += U * hop * a.x_row;
      pdy += U * hop * a.D;
    };
    float2 w[W][H], bias[H], win[W][H], dp[W][H];
    Raw<T, V> q[W];
    load_or<T, V>(q[0], a.bias, p.d, a.bias != nullptr, 0.f);
#pragma unroll
    for (int k = 1; k < W; ++k) load_input<T, W, V>(q[k], a, g.s0, p.b, t0 + k - 1, len, p.d);
    load(t0);
    load_taps<T, W, V>(w, a.w, p.d);
    unpack<T, V>(bias, q[0]);
#pragma unroll
    for (int k = 0; k < W; ++k)
#pragma unroll
      for (int j = 0; j < H; ++j) win[k][j] = dp[k][j] = both(0.f);
#pragma unroll
    for (int k = 1; k < W; ++k) unpack<T, V>(win[k], q[k]);
    T* pdx = static_cast<T*>(g.dx) + (row0 - (W - 1) * hop) * a.D + p.d;
    // U rows; INSIDE: all of them valid tokens of the stretch, whose rows out are tokens of
    // it too (U >= W - 1, so all but the first and the last ones)
    static_assert(U >= W - 1, "the rows out of the second U are tokens of the stretch");
    auto rows = [&](auto inside, int t) {
      constexpr bool INSIDE = decltype(inside)::value;
      Raw<T, V> x[U], d[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        x[i] = rx[i];
        d[i] = ry[i];
      }
      if (t + U < stop) load(t + U);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int e = t + i;
        const bool ok = INSIDE || e < len;
#pragma unroll
        for (int k = 0; k + 1 < W; ++k)
#pragma unroll
          for (int j = 0; j < H; ++j) {
            win[k][j] = win[k + 1][j];
            dp[W - 1 - k][j] = dp[W - 2 - k][j];
          }
        float2 v[H];
#pragma unroll
        for (int j = 0; j < H; ++j) {
          win[W - 1][j] = x[i].pair(j);
          dp[0][j] = d[i].pair(j);
          if (SILU) {
            float2 pre = bias[j];
#pragma unroll
            for (int k = 0; k < W; ++k) pre = fma2(w[k][j], win[k][j], pre);
            const float2 s = sigm2<T>(pre);
            // s + pre s (1 - s)
            dp[0][j] = mul2(dp[0][j], fma2(mul2(pre, s), add2(both(1.f), mul2(s, both(-1.f))), s));
          }
          if (!ok) dp[0][j] = both(0.f);
          // the tokens behind the stretch belong to the next one's sums
          if (INSIDE || (ok && e < t1)) {
#pragma unroll
            for (int k = 0; k < W; ++k) dw[k][j] = fma2(dp[0][j], win[k][j], dw[k][j]);
            dw[W][j] = add2(dw[W][j], dp[0][j]);
          }
          v[j] = mul2(w[0][j], dp[0][j]);
#pragma unroll
          for (int k = 1; k < W; ++k) v[j] = fma2(w[k][j], dp[k][j], v[j]);
        }
        if (INSIDE) {
          if (g.dx) store_vec<T, V>(pdx, v);
        } else {
          // extended row e of the state's gradient out
          if (e >= len && e < len + W - 1 && g.dsT) {
            Raw<T, V> r;
            r.load(static_cast<const T*>(g.dsT) + (static_cast<int64_t>(p.b) * (W - 1) + e - len) * a.D + p.d);
#pragma unroll
            for (int j = 0; j < H; ++j) v[j] = add2(v[j], r.pair(j));
          }
          if (e >= t0 + W - 1) {
            if (e - (W - 1) >= len)
#pragma unroll
              for (int j = 0; j < H; ++j) v[j] = both(0.f);
            if (g.dx && e < stop) store_vec<T, V>(pdx, v);
          } else if (p.seg == 0 && g.ds0) {
            store_vec<T, V>(static_cast<T*>(g.ds0) + (static_cast<int64_t>(p.b) * (W - 1) + e) * a.D + p.d, v);
          }
        }
        pdx += hop * a.D;
      }
    };
    rows(std::false_type{}, t0);
    int t = t0 + U;
    const int valid = len < t1 ? len : t1;
    for (; t + U <= valid; t += U) rows(std::true_type{}, t);
    for (; t < stop; t += U) rows(std::false_type{}, t);
  }
  if (!g.partial) return;
  // the CTA's stretches, in order
#pragma unroll
  for (int k = 0; k <= W; ++k) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < H; ++j) *reinterpret_cast<float2*>(&fold[threadIdx.x * V + 2 * j]) = dw[k][j];
    __syncthreads();
    const int c = static_cast<int>(threadIdx.x), d = p.d / kSpan * kSpan + c;
    if (c < kSpan && d < a.D) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < Spot<V>::RUNS; ++i) s += fold[i * kSpan + c];
      g.partial[(static_cast<int64_t>(p.part) * (W + 1) + k) * a.D + d] = s;
    }
  }
}

// dw[d][k] and dbias[d]: the sums over the CTAs, each of 8 groups in order and then the
// groups in order; 32 channels of one tap a block.
__global__ void __launch_bounds__(256) conv_reduce_kernel(const float* partial, int parts, int D, int W, float* dw,
                                                          float* dbias) {
  __shared__ float sm[8][32];
  const int k = blockIdx.y, c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
  float s = 0.f;
  if (c < D)
#pragma unroll 8
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
__global__ void __launch_bounds__(kStepThreads) conv_step_kernel(const ConvStepArgs p) {
  const ConvArgs& a = p.a;
  const int per = (a.D / 8 + kStepThreads - 1) / kStepThreads, b = blockIdx.x / per;
  const int d = ((blockIdx.x - b * per) * kStepThreads + threadIdx.x) * 8;
  if (d >= a.D) return;
  const int slot = p.slots ? p.slots[b] : b;
  const bool live = slot >= 0 && slot < p.num_slots;
  const int len = live ? a.len ? a.len[b] : a.T : 0;
  T* st = static_cast<T*>(p.state) + static_cast<int64_t>(live ? slot : 0) * (W - 1) * a.D + d;
  float2 w[W][4], bias[4];
  Raw<T, 8> win[W];
  Raw<T, 8> r;
  if (len > 0) {
    load_taps<T, W, 8>(w, a.w, d);
    load_or<T, 8>(r, a.bias, d, a.bias != nullptr, 0.f);
    unpack<T, 8>(bias, r);
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

// Channels a thread.
template <typename T> constexpr int kFwdV = sizeof(T) == 2 ? 8 : 4;
constexpr int kBwdV = 4;

template <typename T, int W>
int fwd(const ConvFwdArgs& f, cudaStream_t s) {
  using S = Spot<kFwdV<T>>;
  const unsigned grid = static_cast<unsigned>(S::parts(f.a)) * S::spans(f.a);
  if (f.a.silu) conv_fwd_kernel<T, W, kFwdV<T>, true><<<grid, kThreads, 0, s>>>(f);
  else conv_fwd_kernel<T, W, kFwdV<T>, false><<<grid, kThreads, 0, s>>>(f);
  return check_launch();
}
template <typename T, int W>
int bwd(const ConvBwdArgs& b, cudaStream_t s) {
  using S = Spot<kBwdV>;
  const unsigned grid = static_cast<unsigned>(S::parts(b.a)) * S::spans(b.a);
  if (b.a.silu) conv_bwd_kernel<T, W, kBwdV, true><<<grid, kThreads, 0, s>>>(b);
  else conv_bwd_kernel<T, W, kBwdV, false><<<grid, kThreads, 0, s>>>(b);
  return check_launch();
}
template <typename T, int W>
int step(const ConvStepArgs& p, cudaStream_t s) {
  conv_step_kernel<T, W><<<static_cast<unsigned>(p.a.B) * ((p.a.D / 8 + kStepThreads - 1) / kStepThreads), kStepThreads, 0, s>>>(p);
  return check_launch();
}
#define RNN_CONV_WIDTHS(CALL, T, ARGS)              \
  switch ((ARGS).a.W) {                             \
    case 2: return CALL<T, 2>(ARGS, s);             \
    case 3: return CALL<T, 3>(ARGS, s);             \
    default: return CALL<T, 4>(ARGS, s);            \
  }
template <typename T> int fwd_t(const ConvFwdArgs& f, cudaStream_t s) { RNN_CONV_WIDTHS(fwd, T, f) }
template <typename T> int bwd_t(const ConvBwdArgs& b, cudaStream_t s) { RNN_CONV_WIDTHS(bwd, T, b) }
template <typename T> int step_t(const ConvStepArgs& p, cudaStream_t s) { RNN_CONV_WIDTHS(step, T, p) }

}  // namespace

size_t conv_workspace_bytes(const ConvArgs& a) {
  return static_cast<size_t>(Spot<kBwdV>::parts(a)) * (a.W + 1) * a.D * 4;
}

int launch_conv_forward(const ConvFwdArgs& f, int is_bf16, cudaStream_t s) {
  return is_bf16 ? fwd_t<__nv_bfloat16>(f, s) : fwd_t<float>(f, s);
}

int launch_conv_backward(const ConvBwdArgs& b, int is_bf16, cudaStream_t s, int* launches) {
  *launches = 0;
  int rc = is_bf16 ? bwd_t<__nv_bfloat16>(b, s) : bwd_t<float>(b, s);
  if (rc) return rc;
  *launches = 1;
  if (!b.partial) return 0;
  conv_reduce_kernel<<<dim3((b.a.D + 31) / 32, b.a.W + 1), 256, 0, s>>>(b.partial, Spot<kBwdV>::parts(b.a), b.a.D, b.a.W, b.dw,
                                                                        b.dbias);
  if (!(rc = check_launch())) *launches = 2;
  return rc;
}

int launch_conv_step(const ConvStepArgs& p, int is_bf16, cudaStream_t s) {
  return is_bf16 ? step_t<__nv_bfloat16>(p, s) : step_t<float>(p, s);
}

}  // namespace rnn
