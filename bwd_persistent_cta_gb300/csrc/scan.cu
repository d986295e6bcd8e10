// scan.cu - the selective scan: whole sequences forward and backward, and the
// serving step.
//
// A warp holds 8 * C channels: lane = cl + 8 sl has the channels C cl .. and, of each,
// the states NS sl .. of 4 NS (states beyond N are held as zeros).  So the sum over a
// channel's states is two shuffles wide, the sum over a warp's channels three, and
// B, C and the steps come from shared memory as broadcasts of 16 bytes.
#include "common.cuh"
#include "pair.cuh"
#include "scan.h"
#include "vec.cuh"
#include <cstdlib>

namespace rnn {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int TT = kScanTile;
constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr float kLift = 2e-8f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 2^x.  bf16 storage takes the hardware's approximation, which is 5e-9 (|x| near
// 1e-3) to 3e-8 (0.01 to 1) low on average: kLift, added to the exponent by the same
// instruction that scales it, takes the middle of that out (states of 77 tokens, error
// against 64 bits: 1.3e-6 without, 5.5e-7 with; training's dA 1.9e-6 and 1.0e-6).  fp32
// storage takes the Taylor series of e^(f ln 2) on |f| <= 1/2, whose
// last rounding is of 1 + something small: half a step, and no bias that a memory of
// a thousand tokens would add up.  The ninth term is below 2^-27.
template <typename T>
__device__ __forceinline__ float decay(float x) {
  if constexpr (sizeof(T) == 2) {
    return ex2(x);
  } else {
    const float r = rintf(x), u = (x - r) * kLn2;
    float p = 1.f / 40320.f;
    p = fmaf(p, u, 1.f / 5040.f);
    p = fmaf(p, u, 1.f / 720.f);
    p = fmaf(p, u, 1.f / 120.f);
    p = fmaf(p, u, 1.f / 24.f);
    p = fmaf(p, u, 1.f / 6.f);
    p = fmaf(p, u, 0.5f);
    p = fmaf(p, u, 1.f);
    p = fmaf(p, u, 1.f);
    // in two steps, so that results below and above the normal range round as they should
    const float half = fminf(fmaxf(r, -250.f), 250.f) * 0.5f;
    const int i = __float2int_rd(half), j = __float2int_ru(half);
    const float s = __int_as_float((i + 127) << 23), t = __int_as_float((j + 127) << 23);
    return x != x || r < -250.f || r > 250.f ? ex2(x) : p * s * t;
  }
}

// log(1 + e^v) = max(v, 0) + log(1 + q), q = e^-|v|.  bf16 storage: log(1 + q) as
// 2 artanh(q / (2 + q)), whose series in (q / (2 + q))^2 <= 1/9 ends after eight
// terms (1e-8): relative accuracy at small steps, at a third of log1pf's instructions.
template <typename T>
__device__ __forceinline__ float softplus(float v) {
  if constexpr (sizeof(T) == 2) {
    const float q = ex2(-fabsf(v) * kLog2e), s = __fdividef(q, 2.f + q), w = s * s;
    float p = 1.f / 15.f;
    p = fmaf(p, w, 1.f / 13.f);
    p = fmaf(p, w, 1.f / 11.f);
    p = fmaf(p, w, 1.f / 9.f);
    p = fmaf(p, w, 1.f / 7.f);
    p = fmaf(p, w, 1.f / 5.f);
    p = fmaf(p, w, 1.f / 3.f);
    p = fmaf(p, w, 1.f);
    return (v > 0.f ? v : v != v ? v : 0.f) + 2.f * s * p;
  } else {
    return (v > 0.f ? v : v != v ? v : 0.f) + log1pf(expf(-fabsf(v)));
  }
}
template <typename T>
__device__ __forceinline__ float sigmoid(float v) {
  if constexpr (sizeof(T) == 2) return __fdividef(1.f, 1.f + __expf(-v));
  else return sigm(v);
}

// Sums M values (a power of two, 2 or 4) over the four state lanes: lane sl ends up
// with value (sl * M / 4), summed.
template <int M>
__device__ __forceinline__ float over_states(const float (&v)[M], int sl) {
  if constexpr (M == 1) {
    float r = v[0];
    r += __shfl_xor_sync(kFull, r, 8);
    return r + __shfl_xor_sync(kFull, r, 16);
  } else if constexpr (M == 2) {
    const bool up = sl & 2;
    float r = (up ? v[1] : v[0]) + __shfl_xor_sync(kFull, up ? v[0] : v[1], 16);
    return r + __shfl_xor_sync(kFull, r, 8);
  } else {
    const bool up = sl & 2, odd = sl & 1;
    const float a = (up ? v[2] : v[0]) + __shfl_xor_sync(kFull, up ? v[0] : v[2], 16);
    const float b = (up ? v[3] : v[1]) + __shfl_xor_sync(kFull, up ? v[1] : v[3], 16);
    return (odd ? b : a) + __shfl_xor_sync(kFull, odd ? a : b, 8);
  }
}

// Which tile of channels a CTA has: of a group, so that its B and C are one row.
template <int C>
struct Where {
  static constexpr int CT = kWarps * 8 * C;      // channels a CTA
  int b, g, tile, c0, width;                     // channels c0 .. c0 + width - 1 of the group's
  __host__ __device__ static int per_group(const ScanArgs& a) { return (a.D / a.G + CT - 1) / CT; }
  __device__ __forceinline__ Where(const ScanArgs& a) {
    const int per = per_group(a), all = per * a.G;
    b = blockIdx.x / all;
    tile = blockIdx.x - b * all;
    g = tile / per;
    const int dg = a.D / a.G, first = (tile - g * per) * CT;
    c0 = g * dg + first;
    width = dg - first < CT ? dg - first : CT;
  }
};

// A thread's share of a [TT][CT] tile: vectors of 8 channels of tokens tid / VC,
// tid / VC + step, ...; always the same channels.
template <int C>
struct Items {
  static constexpr int CT = Where<C>::CT, VC = CT / 8, ROWS = kThreads / VC;
  static constexpr int IT = (TT + ROWS - 1) / ROWS;
};

template <typename T, int IT, int ROWS>
__device__ __forceinline__ void load_items(Raw<T, 8> (&r)[IT], const ScanArgs& a, const void* base, int64_t stride, int b,
                                           int t0, int n, int row, int col, bool in) {
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    const int t = row + i * ROWS;
    const bool ok = in && base && t < n;
    load_or<T, 8>(r[i], base, ok ? a.row(b, t0 + t) * stride + col : 0, ok, 0.f);
  }
}

// The tile's rows of B and C, element by element (their rows need no alignment).
template <typename T, int NS>
struct Rows {
  static constexpr int NP = 4 * NS, PER = TT * NP / kThreads > 0 ? TT * NP / kThreads : 1;
  T v[PER];
  __device__ __forceinline__ void load(const ScanArgs& a, const void* base, int64_t stride, int b, int g, int t0, int n) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = threadIdx.x + i * kThreads, t = e / NP, s = e - t * NP;
      v[i] = from_f<T>(0.f);
      if (t < n && s < a.N)
        v[i] = static_cast<const T*>(base)[a.row(b, t0 + t) * stride + g * a.N + s];
    }
  }
  __device__ __forceinline__ void store(float* to) const {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = threadIdx.x + i * kThreads;
      if (e < TT * NP) to[e] = to_f(v[i]);
    }
  }
};

template <int V>
__device__ __forceinline__ void lds(float (&v)[V], const float* p) {
  if constexpr (V == 1) v[0] = *p;
  else if constexpr (V == 2) {
    const float2 q = *reinterpret_cast<const float2*>(p);
    v[0] = q.x; v[1] = q.y;
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 q = *reinterpret_cast<const float4*>(p + i);
      v[i] = q.x; v[i + 1] = q.y; v[i + 2] = q.z; v[i + 3] = q.w;
    }
  }
}
template <int P>
__device__ __forceinline__ void lds2(float2 (&v)[P], const float* p) {
#pragma unroll
  for (int i = 0; i < P; i += 2) {
    if (P == 1) {
      v[0] = *reinterpret_cast<const float2*>(p);
    } else {
      const float4 q = *reinterpret_cast<const float4*>(p + 2 * i);
      v[i] = make_float2(q.x, q.y);
      if (i + 1 < P) v[i + 1] = make_float2(q.z, q.w);
    }
  }
}

// A thread's C x NS states (or rates) of [.., D, N] memory.
template <int C, int NS>
__device__ __forceinline__ void load_states(float2 (&h)[C][NS / 2], const float* base, int N, int ch, int n0, int width) {
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < NS / 2; ++j) {
      h[c][j] = both(0.f);
      if (base && ch + c < width && n0 + 2 * j < N)
        h[c][j] = *reinterpret_cast<const float2*>(base + static_cast<int64_t>(ch + c) * N + n0 + 2 * j);
    }
}
template <int C, int NS>
__device__ __forceinline__ void store_states(const float2 (&h)[C][NS / 2], float* base, int N, int ch, int n0, int width) {
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < NS / 2; ++j)
      if (ch + c < width && n0 + 2 * j < N)
        *reinterpret_cast<float2*>(base + static_cast<int64_t>(ch + c) * N + n0 + 2 * j) = h[c][j];
}

// The exponent of a token's decay: A log2(e) times its step.
template <typename T>
__device__ __forceinline__ float2 step2(float2 A2, float d) {
  if constexpr (sizeof(T) == 2) return fma2(A2, both(d), both(kLift));
  else return mul2(A2, both(d));
}
template <typename T>
__device__ __forceinline__ float2 decay2(float2 x) { return make_float2(decay<T>(x.x), decay<T>(x.y)); }

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
// A warp works alone: it reads a tile of 16 tokens of its channels (the next tile's
// loads in flight meanwhile), leaves the steps in shared memory, runs the recurrence
// and finishes the outputs, with no barrier but its own.
template <int C>
struct Warp {
  static constexpr int CT = 8 * C, VC = C, ROWS = 32 / VC, IT = TT / ROWS > 0 ? TT / ROWS : 1;
  int b, g, seg, tile, c0, width;
  __host__ __device__ static int per_group(const ScanArgs& a) { return (a.D / a.G + CT - 1) / CT; }
  __device__ __forceinline__ Warp(const ScanArgs& a, int nseg) {
    const int per = per_group(a), all = per * a.G;
    tile = blockIdx.x % all;
    const int r = blockIdx.x / all;
    seg = r % nseg;
    b = r / nseg;
    g = tile / per;
    const int dg = a.D / a.G, first = (tile - g * per) * CT;
    c0 = g * dg + first;
    width = dg - first < CT ? dg - first : CT;
  }
};

// A tile's rows of B or C: [TT][4 NS] floats, zeros beyond N.  Vectors where the rows
// start on 16-byte boundaries, else element by element (no tile ahead then).
template <typename T, int NS>
struct Tile {
  static constexpr int NP = 4 * NS, VECS = TT * NP / 8, PER = VECS / 32 > 0 ? VECS / 32 : 1;
  Raw<T, 8> v[PER];
  __device__ __forceinline__ void load(const ScanArgs& a, const void* base, int64_t stride, bool vec, int b, int g, int t0, int n,
                                       int lane) {
    if (!vec) return;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = lane + 32 * i, t = e / (NP / 8), s = e % (NP / 8) * 8;
      const bool ok = e < VECS && t < n && s < a.N;
      load_or<T, 8>(v[i], base, ok ? a.row(b, t0 + t) * stride + g * a.N + s : 0, ok, 0.f);
    }
  }
  __device__ __forceinline__ void store(float* to, const ScanArgs& a, const void* base, int64_t stride, bool vec, int b, int g,
                                        int t0, int n, int lane) const {
    if (vec) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int e = lane + 32 * i;
        if (e >= VECS) break;
        float2 f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = v[i].pair(j);
        store_vec<float, 8>(to + e * 8, f);
      }
    } else {
#pragma unroll 8
      for (int e = lane; e < TT * NP; e += 32) {
        const int t = e / NP, s = e % NP;
        to[e] = t < n && s < a.N ? to_f(static_cast<const T*>(base)[a.row(b, t0 + t) * stride + g * a.N + s]) : 0.f;
      }
    }
  }
};
template <typename T>
__device__ __forceinline__ bool on_16(const void* base, int64_t stride) {
  return ((reinterpret_cast<uintptr_t>(base) | static_cast<uintptr_t>(stride * sizeof(T))) & 15) == 0;
}

// The states of a thread after segments 0 .. seg - 1, from what each alone leaves.
template <int C, int NS>
__device__ __forceinline__ void join(float2 (&h)[C][NS / 2], const float2 (&A2)[C][NS / 2], const ScanFwdArgs& f, int b, int seg,
                                     int len, int c0, int ch, int n0, int width) {
  const ScanArgs& a = f.a;
#pragma unroll 2
  for (int i = 0; i < seg; ++i) {
    if (i * f.seg >= len) break;
    const int64_t at = (static_cast<int64_t>(b) * f.nseg + i) * a.D + c0;
    float2 e[C][NS / 2];
    load_states<C, NS>(e, f.ends + at * a.N, a.N, ch, n0, width);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float sum = ch + c < width ? f.sums[at + ch + c] : 0.f;
#pragma unroll
      for (int j = 0; j < NS / 2; ++j) h[c][j] = fma2(decay2<float>(mul2(A2[c][j], both(sum))), h[c][j], e[c][j]);
    }
  }
}

enum { kInfer = 0, kTrain = 1, kAlone = 2 };      // kAlone: only what a segment leaves by itself

template <typename T, int NS, int C, int MODE>
__global__ void __launch_bounds__(32) scan_fwd_kernel(const ScanFwdArgs f) {
  using W = Warp<C>;
  constexpr int CT = W::CT, NP = 4 * NS, P = NS / 2;
  constexpr bool OUT = MODE != kAlone;
  __shared__ __align__(16) float sdt[TT][CT], sdx[TT][CT], sB[TT][NP], sC[OUT ? TT : 1][NP], sy[OUT ? TT : 1][CT];
  const ScanArgs& a = f.a;
  const W w(a, OUT ? f.nseg : f.nseg - 1);
  const int lane = threadIdx.x, cl = lane & 7, sl = lane >> 3, ch = cl * C, n0 = sl * NS;
  const int row = lane / W::VC, col = lane % W::VC * 8;
  const bool in = col < w.width && row < TT;
  const int len = a.len ? a.len[w.b] : a.T, begin = w.seg * f.seg, end = begin + f.seg < a.T ? begin + f.seg : a.T;
  const int64_t bD = static_cast<int64_t>(w.b) * a.D + w.c0;
  const bool vB = on_16<T>(a.Bm, a.B_row), vC = on_16<T>(a.Cm, a.C_row);

  Raw<T, 8> x[W::IT], dt[W::IT], z[W::IT];
  Tile<T, NS> rB, rC;
  auto items = [&](Raw<T, 8> (&r)[W::IT], const void* base, int64_t stride, int t0) {
#pragma unroll
    for (int i = 0; i < W::IT; ++i) {
      const int t = t0 + row + i * W::ROWS;
      const bool ok = in && base && t < len && t < end;
      load_or<T, 8>(r[i], base, ok ? a.row(w.b, t) * stride + w.c0 + col : 0, ok, 0.f);
    }
  };
  auto fetch = [&](int t0) {
    items(x, a.x, a.x_row, t0);
    items(dt, a.dt, a.dt_row, t0);
    if (OUT) items(z, a.z, a.z_row, t0);
    rB.load(a, a.Bm, a.B_row, vB, w.b, w.g, t0, len - t0, lane);
    if (OUT) rC.load(a, a.Cm, a.C_row, vC, w.b, w.g, t0, len - t0, lane);
  };
  fetch(begin);
  float2 A2[C][P], h[C][P];
  load_states<C, NS>(A2, a.A + static_cast<int64_t>(w.c0) * a.N, a.N, ch, n0, w.width);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < P; ++j) A2[c][j] = mul2(A2[c][j], both(kLog2e));
  load_states<C, NS>(h, OUT && f.h0 ? f.h0 + bD * a.N : nullptr, a.N, ch, n0, w.width);
  if (!OUT && f.first && w.seg == 0) {
    float2 h0[C][P];
    load_states<C, NS>(h0, f.h0 + bD * a.N, a.N, ch, n0, w.width);
    store_states<C, NS>(h0, f.first + bD * a.N, a.N, ch, n0, w.width);
  }
  if (OUT && w.seg) join<C, NS>(h, A2, f, w.b, w.seg, len, w.c0, ch, n0, w.width);
  float bias[8], skip[8], sum[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    bias[j] = in && a.bias ? a.bias[w.c0 + col + j] : 0.f;
    if (OUT) skip[j] = in && a.skip ? a.skip[w.c0 + col + j] : 0.f;
    sum[j] = 0.f;
  }
  for (int t0 = begin; t0 < end; t0 += TT) {
    if (MODE == kTrain)
      store_states<C, NS>(h, f.kept + ((static_cast<int64_t>(w.b) * a.tiles() + t0 / TT) * a.D + w.c0) * a.N, a.N, ch, n0,
                          w.width);
    const int n = len - t0 < TT ? len - t0 : TT;
#pragma unroll
    for (int i = 0; i < W::IT; ++i) {
      const int t = row + i * W::ROWS;
      if (t >= TT) break;
      float2 d[4], u[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        d[j] = add2(dt[i].pair(j), make_float2(bias[2 * j], bias[2 * j + 1]));
        if (a.softplus) d[j] = make_float2(softplus<T>(d[j].x), softplus<T>(d[j].y));
        u[j] = mul2(d[j], x[i].pair(j));
        if (!OUT && t < n) {
          sum[2 * j] += d[j].x;
          sum[2 * j + 1] += d[j].y;
        }
      }
      store_vec<float, 8>(&sdt[t][col], d);
      store_vec<float, 8>(&sdx[t][col], u);
    }
    rB.store(&sB[0][0], a, a.Bm, a.B_row, vB, w.b, w.g, t0, n, lane);
    if (OUT) rC.store(&sC[0][0], a, a.Cm, a.C_row, vC, w.b, w.g, t0, n, lane);
    Raw<T, 8> xo[W::IT], zo[W::IT];
#pragma unroll
    for (int i = 0; i < W::IT; ++i) {
      xo[i] = x[i];
      zo[i] = z[i];
    }
    __syncwarp();
    if (t0 + TT < end) fetch(t0 + TT);
    auto token = [&](int t) {
      float d[C], u[C], y[C];
      float2 Bv[P], Cv[P];
      lds<C>(d, &sdt[t][ch]);
      lds<C>(u, &sdx[t][ch]);
      lds2<P>(Bv, &sB[t][n0]);
      if (OUT) lds2<P>(Cv, &sC[t][n0]);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float2 s = both(0.f);
#pragma unroll
        for (int j = 0; j < P; ++j) {
          const float2 e = decay2<T>(step2<T>(A2[c][j], d[c]));
          h[c][j] = fma2(e, h[c][j], mul2(Bv[j], both(u[c])));
          if (OUT) s = j ? fma2(Cv[j], h[c][j], s) : mul2(Cv[j], h[c][j]);
        }
        y[c] = s.x + s.y;
      }
      if (OUT) {
        const float r = over_states<C>(y, sl);
        if (C == 4 || sl % (4 / C) == 0) sy[t][ch + sl * C / 4] = r;
      }
    };
    if (n == TT) {
#pragma unroll 4
      for (int t = 0; t < TT; ++t) token(t);
    } else {
      for (int t = 0; t < n; ++t) token(t);
    }
    __syncwarp();
    if (OUT) {
#pragma unroll
      for (int i = 0; i < W::IT; ++i) {
        const int t = row + i * W::ROWS;
        if (!in || t >= TT || t0 + t >= end) break;
        float2 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 s = *reinterpret_cast<const float2*>(&sy[t][col + 2 * j]), xp = xo[i].pair(j), zp = zo[i].pair(j);
          v[j] = fma2(make_float2(skip[2 * j], skip[2 * j + 1]), xp, s);
          if (a.z) v[j] = mul2(v[j], make_float2(zp.x * sigmoid<T>(zp.x), zp.y * sigmoid<T>(zp.y)));
          if (t >= n) v[j] = both(0.f);
        }
        store_vec<T, 8>(static_cast<T*>(f.y) + a.row(w.b, t0 + t) * a.D + w.c0 + col, v);
      }
    }
  }
  if (OUT) {
    if (f.hT && end == a.T) store_states<C, NS>(h, f.hT + bD * a.N, a.N, ch, n0, w.width);
    return;
  }
  const int64_t at = (static_cast<int64_t>(w.b) * f.nseg + w.seg) * a.D + w.c0;
  store_states<C, NS>(h, f.ends + at * a.N, a.N, ch, n0, w.width);
  // the rows' sums of steps, in a fixed order
#pragma unroll
  for (int m = W::VC; m < 32; m <<= 1)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] += __shfl_xor_sync(kFull, sum[j], m);
  if (row == 0 && in)
#pragma unroll
    for (int j = 0; j < 8; ++j) f.sums[at + col + j] = sum[j];
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// A CTA goes through its channels' tiles from the last to the first.  In each it
// computes the tile's states again from the kept one, holds them in registers, and
// runs the gradient g of the state back through the tile:
//     g += dy_t C_t;  dC_t += dy_t h_t;  dB_t += g delta_t x_t;  s1_t = sum g B_t
//     g = a_t g;  P = g h_{t-1};  s2_t = sum P A;  dA += P delta_t
// then, channel by channel, dx = delta s1 + D dy, ddelta = x s1 + s2, and dz from y.
template <typename T, int NS, int C>
struct BwdSmem {
  static constexpr int CT = Where<C>::CT, NP = 4 * NS;
  float dt[TT][CT], dx[TT][CT], dy[TT][CT], s1[TT][CT], s2[TT][CT], y[TT][CT];
  float B[TT][NP], C_[TT][NP];
  float part[kWarps][TT][2 * NP];
};

// Sums 2 NS values over the eight channel lanes; lane cl ends up with NS / 4 of them
// (2 NS >= 8), or with one that two lanes share (2 NS = 4).
template <int V>
__device__ __forceinline__ void over_channels(float (&v)[V], int cl, float (&r)[V >= 8 ? V / 8 : 1]) {
#pragma unroll
  for (int bit = 4, m = V; bit >= 1; bit >>= 1) {
    if (m > 1) {
      m /= 2;
#pragma unroll
      for (int i = 0; i < V / 2; ++i)
        if (i < m) {
          const bool up = cl & bit;
          const float keep = up ? v[i + m] : v[i], send = up ? v[i] : v[i + m];
          v[i] = keep + __shfl_xor_sync(kFull, send, bit);
        }
    } else {
      v[0] += __shfl_xor_sync(kFull, v[0], bit);
    }
  }
#pragma unroll
  for (int i = 0; i < (V >= 8 ? V / 8 : 1); ++i) r[i] = v[i];
}

template <typename T, int NS, int C>
__global__ void __launch_bounds__(kThreads) scan_bwd_kernel(const ScanBwdArgs g_, float* bc, float* pA, float* pD, float* pbias) {
  using I = Items<C>;
  using S = BwdSmem<T, NS, C>;
  constexpr int CT = I::CT, NP = 4 * NS, P = NS / 2;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  S& s = *reinterpret_cast<S*>(smem_raw);
  const ScanArgs& a = g_.a;
  const rnn_scan_grad_t& out = g_.grad;
  const Where<C> w(a);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cl = lane & 7, sl = lane >> 3;
  const int ch = warp * 8 * C + cl * C, n0 = sl * NS;
  const int row = tid / I::VC, col = tid % I::VC * 8;
  const bool in = col < w.width;
  const int len = a.len ? a.len[w.b] : a.T;
  const int64_t bD = static_cast<int64_t>(w.b) * a.D + w.c0;
  const int tiles_c = Where<C>::per_group(a);            // tiles of a group: the partial sums of dB and dC

  float2 A2[C][P], g[C][P], dA[C][P];
  load_states<C, NS>(A2, a.A + static_cast<int64_t>(w.c0) * a.N, a.N, ch, n0, w.width);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < P; ++j) {
      A2[c][j] = mul2(A2[c][j], both(kLog2e));
      dA[c][j] = both(0.f);
    }
  load_states<C, NS>(g, g_.dhT ? g_.dhT + bD * a.N : nullptr, a.N, ch, n0, w.width);
  float bias[8], skip[8], dD[8], dbias[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    bias[j] = in && a.bias ? a.bias[w.c0 + col + j] : 0.f;
    skip[j] = in && a.skip ? a.skip[w.c0 + col + j] : 0.f;
    dD[j] = dbias[j] = 0.f;
  }
  for (int tile = a.tiles() - 1; tile >= 0; --tile) {
    const int t0 = tile * TT, n = len - t0 < 0 ? 0 : len - t0 < TT ? len - t0 : TT;
    Raw<T, 8> x[I::IT], dt[I::IT], z[I::IT], dy[I::IT];
    load_items<T, I::IT, I::ROWS>(x, a, a.x, a.x_row, w.b, t0, n, row, w.c0 + col, in);
    load_items<T, I::IT, I::ROWS>(dt, a, a.dt, a.dt_row, w.b, t0, n, row, w.c0 + col, in);
    load_items<T, I::IT, I::ROWS>(z, a, a.z, a.z_row, w.b, t0, n, row, w.c0 + col, in);
    load_items<T, I::IT, I::ROWS>(dy, a, g_.dy, a.D, w.b, t0, n, row, w.c0 + col, in);
    Rows<T, NS> rB, rC;
    rB.load(a, a.Bm, a.B_row, w.b, w.g, t0, n);
    rC.load(a, a.Cm, a.C_row, w.b, w.g, t0, n);
#pragma unroll
    for (int i = 0; i < I::IT; ++i) {
      const int t = row + i * I::ROWS;
      if (t >= TT) break;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 dp = dt[i].pair(j), xp = x[i].pair(j), zp = z[i].pair(j), op = dy[i].pair(j);
        float2 d = make_float2(dp.x + bias[2 * j], dp.y + bias[2 * j + 1]);
        if (a.softplus) d = make_float2(softplus<T>(d.x), softplus<T>(d.y));
        *reinterpret_cast<float2*>(&s.dt[t][col + 2 * j]) = d;
        *reinterpret_cast<float2*>(&s.dx[t][col + 2 * j]) = mul2(d, xp);
        float2 o = op;
        if (a.z) o = mul2(o, make_float2(zp.x * sigmoid<T>(zp.x), zp.y * sigmoid<T>(zp.y)));
        *reinterpret_cast<float2*>(&s.dy[t][col + 2 * j]) = o;
      }
    }
    rB.store(&s.B[0][0]);
    rC.store(&s.C_[0][0]);
    // the states of the tile, again
    float2 h[TT + 1][C][P];
    load_states<C, NS>(h[0], g_.kept + ((static_cast<int64_t>(w.b) * a.tiles() + tile) * a.D + w.c0) * a.N, a.N, ch, n0,
                       w.width);
    __syncthreads();
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      if (t < n) {
        float d[C], u[C];
        float2 Bv[P];
        lds<C>(d, &s.dt[t][ch]);
        lds<C>(u, &s.dx[t][ch]);
        lds2<P>(Bv, &s.B[t][n0]);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int j = 0; j < P; ++j)
            h[t + 1][c][j] = fma2(decay2<T>(step2<T>(A2[c][j], d[c])), h[t][c][j], mul2(Bv[j], both(u[c])));
      }
    }
#pragma unroll
    for (int t = TT - 1; t >= 0; --t) {
      if (t < n) {
        float d[C], u[C], o[C], s1[C], s2[C], yy[C];
        float2 Bv[P], Cv[P], dB[P], dC[P];
        lds<C>(d, &s.dt[t][ch]);
        lds<C>(u, &s.dx[t][ch]);
        lds<C>(o, &s.dy[t][ch]);
        lds2<P>(Bv, &s.B[t][n0]);
        lds2<P>(Cv, &s.C_[t][n0]);
#pragma unroll
        for (int j = 0; j < P; ++j) dB[j] = dC[j] = both(0.f);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float2 q1 = both(0.f), q2 = both(0.f), q3 = both(0.f);
#pragma unroll
          for (int j = 0; j < P; ++j) {
            const float2 e = decay2<T>(step2<T>(A2[c][j], d[c]));
            g[c][j] = fma2(Cv[j], both(o[c]), g[c][j]);
            dC[j] = fma2(h[t + 1][c][j], both(o[c]), dC[j]);
            q3 = fma2(h[t + 1][c][j], Cv[j], q3);
            dB[j] = fma2(g[c][j], both(u[c]), dB[j]);
            q1 = fma2(g[c][j], Bv[j], q1);
            g[c][j] = mul2(e, g[c][j]);
            const float2 p = mul2(g[c][j], h[t][c][j]);
            q2 = fma2(p, A2[c][j], q2);
            dA[c][j] = fma2(p, both(d[c]), dA[c][j]);
          }
          s1[c] = q1.x + q1.y;
          s2[c] = q2.x + q2.y;
          yy[c] = q3.x + q3.y;
        }
        const float r1 = over_states<C>(s1, sl), r2 = over_states<C>(s2, sl), r3 = over_states<C>(yy, sl);
        if (C == 4 || sl % (4 / C) == 0) {
          const int c = ch + sl * C / 4;
          s.s1[t][c] = r1;
          s.s2[t][c] = r2 * kLn2;
          s.y[t][c] = r3;
        }
        float v[2 * NS], r[2 * NS >= 8 ? NS / 4 : 1];
#pragma unroll
        for (int j = 0; j < P; ++j) {
          v[2 * j] = dB[j].x; v[2 * j + 1] = dB[j].y;
          v[NS + 2 * j] = dC[j].x; v[NS + 2 * j + 1] = dC[j].y;
        }
        over_channels<2 * NS>(v, cl, r);
        if constexpr (NS >= 4) {
          // lane cl: values cl * NS / 4 .. of (dB, dC)
#pragma unroll
          for (int i = 0; i < NS / 4; ++i) {
            const int k = cl * (NS / 4) + i;
            s.part[warp][t][(k / NS) * NP + n0 + k % NS] = r[i];
          }
        } else if (!(cl & 1)) {
          const int k = cl >> 1;
          s.part[warp][t][(k / NS) * NP + n0 + k % NS] = r[0];
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < I::IT; ++i) {
      const int t = row + i * I::ROWS;
      if (t >= TT) break;
      if (!in || t0 + t >= a.T) continue;
      float2 vx[4], vt[4], vz[4];
      const bool live = t < n;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = col + 2 * j;
        vx[j] = vt[j] = vz[j] = both(0.f);
        if (live) {
          const float2 d = *reinterpret_cast<const float2*>(&s.dt[t][c]), o = *reinterpret_cast<const float2*>(&s.dy[t][c]);
          const float2 q1 = *reinterpret_cast<const float2*>(&s.s1[t][c]), q2 = *reinterpret_cast<const float2*>(&s.s2[t][c]);
          const float2 q3 = *reinterpret_cast<const float2*>(&s.y[t][c]);
          const float2 xp = x[i].pair(j), zp = z[i].pair(j), op = dy[i].pair(j), dp = dt[i].pair(j);
          const float2 sk = make_float2(skip[2 * j], skip[2 * j + 1]);
          vx[j] = fma2(d, q1, mul2(sk, o));
          vt[j] = fma2(xp, q1, q2);
          if (a.softplus) {
            vt[j].x *= sigmoid<T>(dp.x + bias[2 * j]);
            vt[j].y *= sigmoid<T>(dp.y + bias[2 * j + 1]);
          }
          dD[2 * j] += o.x * xp.x;
          dD[2 * j + 1] += o.y * xp.y;
          dbias[2 * j] += vt[j].x;
          dbias[2 * j + 1] += vt[j].y;
          if (a.z) {
            const float2 yv = fma2(sk, xp, q3), sg = make_float2(sigmoid<T>(zp.x), sigmoid<T>(zp.y));
            vz[j].x = op.x * yv.x * sg.x * (1.f + zp.x * (1.f - sg.x));
            vz[j].y = op.y * yv.y * sg.y * (1.f + zp.y * (1.f - sg.y));
          }
        }
      }
      const int64_t at = a.row(w.b, t0 + t) * a.D + w.c0 + col;
      if (out.dx) store_vec<T, 8>(static_cast<T*>(out.dx) + at, vx);
      if (out.ddt) store_vec<T, 8>(static_cast<T*>(out.ddt) + at, vt);
      if (out.dz) store_vec<T, 8>(static_cast<T*>(out.dz) + at, vz);
    }
    if (bc) {
      for (int e = tid; e < TT * 2 * NP; e += kThreads) {
        const int t = e / (2 * NP), k = e - t * 2 * NP;
        if (t0 + t >= a.T) break;
        float v = 0.f;
        if (t < n)
#pragma unroll
          for (int q = 0; q < kWarps; ++q) v += s.part[q][t][k];
        bc[(((static_cast<int64_t>(w.b) * a.T + t0 + t) * a.G + w.g) * tiles_c + (w.tile - w.g * tiles_c)) * (2 * NP) + k] = v;
      }
    }
    __syncthreads();
  }
  if (out.dh0) store_states<C, NS>(g, static_cast<float*>(out.dh0) + bD * a.N, a.N, ch, n0, w.width);
  if (pA) store_states<C, NS>(dA, pA + bD * a.N, a.N, ch, n0, w.width);
  // the threads that share channels, in order
  float* fold = reinterpret_cast<float*>(smem_raw);        // [ROWS][CT] twice
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    fold[row * CT + col + j] = dD[j];
    fold[(I::ROWS + row) * CT + col + j] = dbias[j];
  }
  __syncthreads();
  for (int c = tid; c < w.width; c += kThreads) {
    float v = 0.f, u = 0.f;
    for (int r = 0; r < I::ROWS; ++r) {
      v += fold[r * CT + c];
      u += fold[(I::ROWS + r) * CT + c];
    }
    if (pD) pD[bD + c] = v;
    if (pbias) pbias[bD + c] = u;
  }
}

// dB and dC: the sum over a group's tiles of channels, in order.
template <typename T>
__global__ void __launch_bounds__(256) scan_bc_kernel(const ScanArgs a, const float* bc, int tiles, int NP, T* dB, T* dC) {
  const int64_t rows = static_cast<int64_t>(a.B) * a.T * a.G, all = rows * 2 * NP;
  for (int64_t e = blockIdx.x * 256LL + threadIdx.x; e < all; e += gridDim.x * 256LL) {
    const int64_t r = e / (2 * NP);
    const int k = static_cast<int>(e - r * 2 * NP), n = k % NP;
    if (n >= a.N) continue;
    float v = 0.f;
    for (int i = 0; i < tiles; ++i) v += bc[(r * tiles + i) * (2 * NP) + k];
    const int g = static_cast<int>(r % a.G);
    const int64_t bt = r / a.G;
    const int b = static_cast<int>(bt / a.T), t = static_cast<int>(bt - static_cast<int64_t>(b) * a.T);
    T* out = k < NP ? dB : dC;
    if (out) out[(a.row(b, t) * a.G + g) * a.N + n] = from_f<T>(v);
  }
}

// out[e] = sum over sequences of part[b][e], in order.
__global__ void __launch_bounds__(256) scan_sum_kernel(const float* part, int B, int64_t n, float* out) {
  const int64_t e = blockIdx.x * 256LL + threadIdx.x;
  if (e >= n) return;
  float v = 0.f;
  for (int b = 0; b < B; ++b) v += part[b * n + e];
  out[e] = v;
}

// ---------------------------------------------------------------------------
// the serving step
// ---------------------------------------------------------------------------
// SL lanes a channel, four states each.
template <typename T, int SL>
__global__ void __launch_bounds__(256) scan_step_kernel(const ScanStepArgs p) {
  const ScanArgs& a = p.a;
  constexpr int PER = 256 / SL;
  const int per = (a.D + PER - 1) / PER;
  const int b = blockIdx.x / per, d = (blockIdx.x - b * per) * PER + threadIdx.x / SL, n0 = threadIdx.x % SL * 4;
  const int len = a.len ? a.len[b] : a.T;
  const int slot = p.slots ? p.slots[b] : b;
  const bool in = d < a.D, live = slot >= 0 && slot < p.num_slots, st = in && live && n0 < a.N;
  const int g = in ? d / (a.D / a.G) : 0;
  float* at = p.state + (static_cast<int64_t>(slot) * a.D + d) * a.N + n0;
  float4 h = make_float4(0.f, 0.f, 0.f, 0.f), A = h;
  if (st) {
    h = *reinterpret_cast<const float4*>(at);
    A = *reinterpret_cast<const float4*>(a.A + static_cast<int64_t>(d) * a.N + n0);
  }
  const float bias = in && a.bias ? a.bias[d] : 0.f, skip = in && a.skip ? a.skip[d] : 0.f;
  const int n = live ? len : 0;
  for (int t = 0; t < a.T; ++t) {
    const int64_t r = a.row(b, t);
    float y = 0.f;
    if (t < n && in) {
      const float xv = to_f(static_cast<const T*>(a.x)[r * a.x_row + d]);
      float dv = to_f(static_cast<const T*>(a.dt)[r * a.dt_row + d]) + bias;
      if (a.softplus) dv = softplus<T>(dv);
      if (st) {
        const T* Bp = static_cast<const T*>(a.Bm) + r * a.B_row + g * a.N + n0;
        const T* Cp = static_cast<const T*>(a.Cm) + r * a.C_row + g * a.N + n0;
        const float e = dv * kLog2e, u = dv * xv;
        const float lift = sizeof(T) == 2 ? kLift : 0.f;
        h.x = fmaf(decay<T>(fmaf(A.x, e, lift)), h.x, u * to_f(Bp[0]));
        h.y = fmaf(decay<T>(fmaf(A.y, e, lift)), h.y, u * to_f(Bp[1]));
        h.z = fmaf(decay<T>(fmaf(A.z, e, lift)), h.z, u * to_f(Bp[2]));
        h.w = fmaf(decay<T>(fmaf(A.w, e, lift)), h.w, u * to_f(Bp[3]));
        y = fmaf(to_f(Cp[3]), h.w, fmaf(to_f(Cp[2]), h.z, fmaf(to_f(Cp[1]), h.y, to_f(Cp[0]) * h.x)));
      }
    }
#pragma unroll
    for (int m = 1; m < SL; m <<= 1) y += __shfl_xor_sync(kFull, y, m);
    if (in && threadIdx.x % SL == 0) {
      if (t < n) {
        y = fmaf(skip, to_f(static_cast<const T*>(a.x)[r * a.x_row + d]), y);
        if (a.z) {
          const float zv = to_f(static_cast<const T*>(a.z)[r * a.z_row + d]);
          y *= zv * sigmoid<T>(zv);
        }
      }
      static_cast<T*>(p.y)[r * a.D + d] = from_f<T>(t < n ? y : 0.f);
    }
  }
  if (st && n > 0) *reinterpret_cast<float4*>(at) = h;
}

int check_launch() { return cudaGetLastError() == cudaSuccess ? 0 : RNN_CUDA_ERROR; }

// States a lane: a quarter of the channel's, rounded up to a power of two.
int lane_states(int N) { return N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }
constexpr int fwd_channels(int NS) { return NS <= 4 ? 4 : NS == 8 ? 2 : 1; }
constexpr int bwd_channels(int NS) { return NS <= 4 ? 2 : 1; }


template <typename T, int NS, int C>
int fwd(ScanFwdArgs f, cudaStream_t s, int* launches) {
  const unsigned warps = static_cast<unsigned>(f.a.B) * f.a.G * Warp<C>::per_group(f.a);
  int rc;
  if (f.nseg > 1) {
    scan_fwd_kernel<T, NS, C, kAlone><<<warps * (f.nseg - 1), 32, 0, s>>>(f);
    if ((rc = check_launch())) return rc;
    ++*launches;
    if (f.first) f.h0 = f.first;
  }
  if (f.kept) scan_fwd_kernel<T, NS, C, kTrain><<<warps * f.nseg, 32, 0, s>>>(f);
  else scan_fwd_kernel<T, NS, C, kInfer><<<warps * f.nseg, 32, 0, s>>>(f);
  if (!(rc = check_launch())) ++*launches;
  return rc;
}
template <typename T>
int fwd_t(const ScanFwdArgs& f, cudaStream_t s, int* launches) {
  switch (lane_states(f.a.N)) {
    case 2: return fwd<T, 2, 4>(f, s, launches);
    case 4: return fwd<T, 4, 4>(f, s, launches);
    case 8: return fwd<T, 8, 2>(f, s, launches);
    default: return fwd<T, 16, 1>(f, s, launches);
  }
}

int bwd_tiles(const ScanArgs& a) {
  const int C = bwd_channels(lane_states(a.N)), ct = kWarps * 8 * C;
  return (a.D / a.G + ct - 1) / ct;
}

template <typename T, int NS>
int bwd(const ScanBwdArgs& b, cudaStream_t s, float* bc, float* pA, float* pD, float* pbias) {
  constexpr int C = bwd_channels(NS), smem = sizeof(BwdSmem<T, NS, C>);
  static_assert(smem <= 227 * 1024 && smem >= 2 * Items<C>::ROWS * Items<C>::CT * 4, "the tile and the folded sums fit");
  if (cudaFuncSetAttribute(scan_bwd_kernel<T, NS, C>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
    return RNN_CUDA_ERROR;
  const unsigned grid = static_cast<unsigned>(b.a.B) * b.a.G * Where<C>::per_group(b.a);
  scan_bwd_kernel<T, NS, C><<<grid, kThreads, smem, s>>>(b, bc, pA, pD, pbias);
  return check_launch();
}

template <typename T>
int bwd_t(const ScanBwdArgs& b, cudaStream_t s, int* launches) {
  const ScanArgs& a = b.a;
  const ScanBwdLayout l = scan_bwd_layout(a);
  auto part = [&](const void* want, size_t off) { return want ? reinterpret_cast<float*>(b.work + off) : nullptr; };
  float *bc = part(b.grad.dB ? b.grad.dB : b.grad.dC, l.bc), *pA = part(b.grad.dA, l.dA), *pD = part(b.grad.dD, l.dD),
        *pbias = part(b.grad.ddt_bias, l.dbias);
  int rc;
  switch (lane_states(a.N)) {
    case 2: rc = bwd<T, 2>(b, s, bc, pA, pD, pbias); break;
    case 4: rc = bwd<T, 4>(b, s, bc, pA, pD, pbias); break;
    case 8: rc = bwd<T, 8>(b, s, bc, pA, pD, pbias); break;
    default: rc = bwd<T, 16>(b, s, bc, pA, pD, pbias);
  }
  if (rc) return rc;
  ++*launches;
  if (bc) {
    const int NP = 4 * lane_states(a.N);
    const int64_t blocks = (static_cast<int64_t>(a.B) * a.T * a.G * 2 * NP + 255) / 256;
    scan_bc_kernel<T><<<static_cast<unsigned>(blocks < 16 * a.num_sms ? blocks : 16 * a.num_sms), 256, 0, s>>>(
        a, bc, bwd_tiles(a), NP, static_cast<T*>(b.grad.dB), static_cast<T*>(b.grad.dC));
    if ((rc = check_launch())) return rc;
    ++*launches;
  }
  auto sum = [&](const float* from, int64_t n, void* to) {
    if (!from || rc) return;
    scan_sum_kernel<<<static_cast<unsigned>((n + 255) / 256), 256, 0, s>>>(from, a.B, n, static_cast<float*>(to));
    if (!(rc = check_launch())) ++*launches;
  };
  sum(pA, static_cast<int64_t>(a.D) * a.N, b.grad.dA);
  sum(pD, a.D, b.grad.dD);
  sum(pbias, a.D, b.grad.ddt_bias);
  return rc;
}

template <typename T, int SL>
int step(const ScanStepArgs& p, cudaStream_t s) {
  constexpr int PER = 256 / SL;
  scan_step_kernel<T, SL><<<static_cast<unsigned>(p.a.B) * ((p.a.D + PER - 1) / PER), 256, 0, s>>>(p);
  return check_launch();
}
template <typename T>
int step_t(const ScanStepArgs& p, cudaStream_t s) {
  if (p.a.N <= 8) return step<T, 2>(p, s);
  if (p.a.N <= 16) return step<T, 4>(p, s);
  return p.a.N <= 32 ? step<T, 8>(p, s) : step<T, 16>(p, s);
}

}  // namespace

ScanSplit scan_split(const ScanArgs& a, int is_bf16) {
  const int C = fwd_channels(lane_states(a.N)), per = (a.D / a.G + 8 * C - 1) / (8 * C);
  const int64_t warps = static_cast<int64_t>(a.B) * a.G * per, want = static_cast<int64_t>(a.num_sms) * 16;
  const int tiles = a.tiles();
  int64_t n = warps * 2 > want ? 1 : want / warps;
  const char* env = getenv("V_NSEG");
  if (env) n = atoi(env);
  if (n > tiles / 4) n = tiles / 4;
  if (n < 1) n = 1;
  ScanSplit p{};
  p.len = (tiles + static_cast<int>(n) - 1) / static_cast<int>(n) * kScanTile;
  p.nseg = (a.T + p.len - 1) / p.len;
  if (p.nseg == 1) return p;
  auto up = [](size_t v) { return (v + 255) & ~static_cast<size_t>(255); };
  const size_t rows = static_cast<size_t>(a.B) * p.nseg * a.D;
  p.sums = up(rows * a.N * 4);
  p.first = p.sums + up(rows * 4);
  p.bytes = p.first + up(static_cast<size_t>(a.B) * a.D * a.N * 4);
  return p;
}

int launch_scan_forward(const ScanFwdArgs& f_, void* work, int is_bf16, cudaStream_t s, int* launches) {
  ScanFwdArgs f = f_;
  const ScanSplit p = scan_split(f.a, is_bf16);
  f.nseg = p.nseg;
  f.seg = p.len;
  f.ends = reinterpret_cast<float*>(static_cast<char*>(work) + p.ends);
  f.sums = reinterpret_cast<float*>(static_cast<char*>(work) + p.sums);
  f.first = p.nseg > 1 && f.h0 && f.h0 == f.hT ? reinterpret_cast<float*>(static_cast<char*>(work) + p.first) : nullptr;
  *launches = 0;
  return is_bf16 ? fwd_t<__nv_bfloat16>(f, s, launches) : fwd_t<float>(f, s, launches);
}

ScanBwdLayout scan_bwd_layout(const ScanArgs& a) {
  ScanBwdLayout l{};
  size_t off = 0;
  auto take = [&](size_t n) {
    const size_t o = off;
    off += (n * 4 + 255) & ~static_cast<size_t>(255);
    return o;
  };
  const size_t bd = static_cast<size_t>(a.B) * a.D;
  l.bc = take(static_cast<size_t>(a.B) * a.T * a.G * bwd_tiles(a) * 8 * lane_states(a.N));
  l.dA = take(bd * a.N);
  l.dD = take(bd);
  l.dbias = take(bd);
  l.bytes = off;
  return l;
}

int launch_scan_backward(const ScanBwdArgs& b, int is_bf16, cudaStream_t s, int* launches) {
  *launches = 0;
  return is_bf16 ? bwd_t<__nv_bfloat16>(b, s, launches) : bwd_t<float>(b, s, launches);
}

int launch_scan_step(const ScanStepArgs& p, int is_bf16, cudaStream_t s) {
  return is_bf16 ? step_t<__nv_bfloat16>(p, s) : step_t<float>(p, s);
}

}  // namespace rnn
