// scan.cu - the selective scan: whole sequences forward and backward, and the
// serving step.
//
// What bounds it: for each token, channel and state one exponential (4 cycles of a
// scheduler's special function unit for a warp) and four multiply-adds forward, one and
// twelve backward; memory is a third of that at 16 states.  So the recurrence is kept at
// two values an instruction and everything around it small: a warp holds the states of its
// channels in registers, lane = cl + CL sl with C channels and NS states of each, sums over
// a channel's states and over the warp's channels are a few shuffles, and steps, B and C
// come from shared memory as broadcasts of 16 bytes.
#include "common.cuh"
#include "pair.cuh"
#include "scan.h"
#include "vec.cuh"

#include <algorithm>
#include <type_traits>

namespace rnn {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

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

// A token's decay 2^(A log2(e) delta), two states at a time, by the hardware's
// approximation, which is low on average by (relative, in bins of |x|): 8e-9 to 5e-9 from
// 1e-5 to 2e-3, 1e-8 at 4e-3, 1.6e-8 at 6e-3, 1e-8 to 3e-8 from 0.01 to 0.8, 5e-8 above one;
// below 1.2e-7 it is exactly one (a token behind the last leaves the state as it is).
// A memory of M tokens would add that up M times, so the exponent is lifted by it.
//
// bf16 storage: one constant, which the multiply-add that makes the exponent adds for
// nothing.  It is the middle, so decays nearer to one than 2^-0.002 come out 8e-9 high: a
// state that remembers 1e4 tokens 8e-5, against inputs that are rounded at 2e-3 each.
//
// fp32 storage: what belongs to the size of the exponent, a constant and a slope up to a
// knee (states of 8192 tokens, error against 64 bits 4.9e-5 with one constant, 1.5e-5 so).
// W tokens' slope at once: a bias is a sum over many tokens, so a sequence adds it at one
// token in four.  8 x 1024 tokens of 2048 channels and 64 states 440 us, 432 with the constant,
// 473 with the slope at every token.  A polynomial for exponents below 2^-6, which would
// also take the approximation's own roundings out (3e-8 instead of 1.7e-8): 538 us.
constexpr float kLift = 2e-8f, kLow = 9e-9f, kSlope = 2.7e-6f, kKnee = 0.0085f;
template <typename T, int W = 1>
__device__ __forceinline__ float2 decay2(float2 A2, float d) {
  float2 x = fma2(A2, both(d), both(sizeof(T) == 2 ? kLift : kLow));
  if constexpr (sizeof(T) == 4 && W > 0)
    x = fma2(make_float2(fminf(fabsf(x.x), kKnee), fminf(fabsf(x.y), kKnee)), both(W * kSlope), x);
  return make_float2(ex2(x.x), ex2(x.y));
}

// The same for one state; ``slope`` is that of the tokens whose lift this one adds.
template <typename T, bool ADDS>
__device__ __forceinline__ float decay1(float A2, float d, float slope) {
  float x = fmaf(A2, d, sizeof(T) == 2 ? kLift : kLow);
  if (sizeof(T) == 4 && ADDS) x = fmaf(fminf(fabsf(x), kKnee), slope, x);
  return ex2(x);
}

// log(1 + e^v) = max(v, 0) + log(1 + q), q = e^-|v|, two at a time.  log(1 + q) is
// 2 artanh(s), s = q / (2 + q) <= 1/3, as s times a polynomial in s^2 (interpolated at
// the Chebyshev nodes of [0, 1/9], off by 1.5e-8, the logarithm by 5e-9 or a relative
// 8e-9), in a third of log1pf's instructions.  The exponent |v| log2(e) is rounded, and with
// it q by a relative |v| 2^-24 or so: 2 to 4e-7 of the steps in use (v of -7 to -2), which
// scales a channel's rates by as much; expf would hold 1e-7 for ten more instructions.
__device__ __forceinline__ float2 softplus2(float2 v) {
  const float2 q = make_float2(ex2(-fabsf(v.x) * kLog2e), ex2(-fabsf(v.y) * kLog2e));
  const float2 d = add2(q, both(2.f)), s = mul2(q, make_float2(rcp(d.x), rcp(d.y))), w = mul2(s, s);
  float2 p = fma2(both(0.28157778f), w, both(0.27965158f));
  p = fma2(p, w, both(0.40024596f));
  p = fma2(p, w, both(0.66666322f));
  p = fma2(p, w, both(2.f));
  return fma2(p, s, make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));         // a NaN comes in through s
}
// 1 / (1 + e^-v) from the approximations, a few 2^-24 off and, for negative v, |v| 2^-24 more.
__device__ __forceinline__ float2 sigmoid2(float2 v) {
  const float2 q = mul2(v, both(-kLog2e)), d = add2(make_float2(ex2(q.x), ex2(q.y)), both(1.f));
  return make_float2(rcp(d.x), rcp(d.y));
}

template <int V>
__device__ __forceinline__ void lds(float (&v)[V], const float* p) {
  if constexpr (V == 1) {
    v[0] = *p;
  } else if constexpr (V == 2) {
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
// 2 P values, four of them every HOP.
template <int P, int HOP = 4>
__device__ __forceinline__ void lds2(float2 (&v)[P], const float* p) {
#pragma unroll
  for (int i = 0; i < P; i += 2) {
    const float4 q = *reinterpret_cast<const float4*>(p + i / 2 * HOP);
    v[i] = make_float2(q.x, q.y);
    v[i + 1] = make_float2(q.z, q.w);
  }
}

// A thread's C x NS states (or rates) of [.., D, N] memory, four of them every HOP from n0
// on, zeros beyond D and N (a multiple of 8).  The lanes of a channel take turns of four
// states, so that a store covers whole sectors.
template <int C, int NS, int HOP>
__device__ __forceinline__ void load_states(float2 (&h)[C][NS / 2], const float* base, int N, int ch, int n0, int width) {
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int k = 0; k < NS / 4; ++k) {
      float4 q = make_float4(0.f, 0.f, 0.f, 0.f);
      if (base && ch + c < width && n0 + k * HOP < N)
        q = *reinterpret_cast<const float4*>(base + static_cast<int64_t>(ch + c) * N + n0 + k * HOP);
      h[c][2 * k] = make_float2(q.x, q.y);
      h[c][2 * k + 1] = make_float2(q.z, q.w);
    }
}
template <int C, int NS, int HOP>
__device__ __forceinline__ void store_states(const float2 (&h)[C][NS / 2], float* base, int N, int ch, int n0, int width) {
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int k = 0; k < NS / 4; ++k)
      if (ch + c < width && n0 + k * HOP < N)
        *reinterpret_cast<float4*>(base + static_cast<int64_t>(ch + c) * N + n0 + k * HOP) =
            make_float4(h[c][2 * k].x, h[c][2 * k].y, h[c][2 * k + 1].x, h[c][2 * k + 1].y);
}
// A token behind the last one, and one whose step is zero, must leave the state as it is, so
// a rate of minus infinity is held as a large number: a reset at every step above 1e-28.
__device__ __forceinline__ float finite_rate(float a) {
  float r;
  asm("{.reg .f32 t;\n\tmax.NaN.f32 t, %1, %2;\n\tmin.NaN.f32 %0, t, %3;}" : "=f"(r) : "f"(a), "f"(-1e30f), "f"(1e30f));
  return r;
}
// The rates in units of log2(e).
template <int C, int NS, int HOP>
__device__ __forceinline__ void load_rates(float2 (&A2)[C][NS / 2], const ScanArgs& a, int c0, int ch, int n0, int width) {
  load_states<C, NS, HOP>(A2, a.A + static_cast<int64_t>(c0) * a.N, a.N, ch, n0, width);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < NS / 2; ++j) {
      A2[c][j] = mul2(A2[c][j], both(kLog2e));
      A2[c][j] = make_float2(finite_rate(A2[c][j].x), finite_rate(A2[c][j].y));
    }
}

// Which channels of which segment a warp has: of one group, so that its B and C are one row.
template <int CT>
struct Where {
  int b, g, seg, tile, c0, width;                // channels c0 .. c0 + width - 1; tile: of the group
  __host__ __device__ static int per_group(const ScanArgs& a) { return (a.D / a.G + CT - 1) / CT; }
  __device__ __forceinline__ Where(const ScanArgs& a, int nseg, int at) {
    const int per = per_group(a), all = per * a.G;
    const int i = at % all, r = at / all;
    seg = r % nseg;
    b = r / nseg;
    g = i / per;
    tile = i - g * per;
    const int dg = a.D / a.G, first = tile * CT;
    c0 = g * dg + first;
    width = dg - first < CT ? dg - first : CT;
  }
};

__device__ __forceinline__ void async16(void* to, const void* from, bool ok) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(smem_u32(to)), "l"(from), "r"(ok ? 16 : 0) : "memory");
}
// A thread's 8 elements to its own place, or zeros.
template <typename T>
__device__ __forceinline__ void async_item(Raw<T, 8>* to, const void* base, int64_t at, bool ok, const void* any) {
  const char* from = ok ? reinterpret_cast<const char*>(static_cast<const T*>(base) + at) : static_cast<const char*>(any);
#pragma unroll
  for (int v = 0; v < static_cast<int>(sizeof(Raw<T, 8>)); v += 16)
    async16(reinterpret_cast<char*>(to) + v, ok ? from + v : from, ok);
}

// A tile of TT rows of B or C as [TT][NP] floats, zeros beyond N and behind the last token.
// Rows that start on 16-byte boundaries come as vectors into the lanes' own places in
// shared memory, tiles ahead (in registers the compiler has them waited for at once: 442
// instead of 290 us for 8 x 2048 tokens of 2048 channels), others element by element when
// they are needed.
template <typename T>
__device__ __forceinline__ bool on_16(const void* base, int64_t stride) {
  return ((reinterpret_cast<uintptr_t>(base) | static_cast<uintptr_t>(stride * sizeof(T))) & 15) == 0;
}
template <typename T, int TT, int NP>
struct Rows {
  static constexpr int VECS = TT * NP / 8, PER = VECS / 32 > 0 ? VECS / 32 : 1, PT = 32 * 8 / NP;   // tokens between two of a lane's
  using Stage = Raw<T, 8>[PER][32];
  const T* at;                 // the row of token 0 of the tile to come
  int64_t token;               // elements from a token to the next
  bool vec;
  int t, s, N;                 // of the lane's first vector
  __device__ __forceinline__ Rows(const ScanArgs& a, const void* base, int64_t stride, int b, int g, int t0, int lane) {
    vec = on_16<T>(base, stride);
    token = (a.bfirst ? 1 : a.B) * stride;
    at = static_cast<const T*>(base) + a.row(b, t0) * stride + g * a.N;
    N = a.N;
    t = lane / (NP / 8);
    s = lane % (NP / 8) * 8;
  }
  // The tile whose first row is ``at``, n of its tokens, then on by ``move`` tokens.
  __device__ __forceinline__ void load(Stage& to, int n, int move, int lane, const void* any) {
    if (!vec) return;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const bool ok = (VECS >= 32 || t < TT) && t + i * PT < n && s < N;
      async_item<T>(&to[i][lane], at, (t + i * PT) * token + s, ok, any);
    }
    at += move * token;
  }
  __device__ __forceinline__ void store(float* to, const Stage& from, int n, int move, int lane) {
    if (vec) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (VECS < 32 && t >= TT) break;
        const Raw<T, 8> r = from[i][lane];
        float2 f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = r.pair(j);
        store_vec<float, 8>(to + (lane + 32 * i) * 8, f);
      }
    } else {
#pragma unroll 4
      for (int e = lane; e < TT * NP; e += 32) {
        const int q = e / NP, k = e % NP;
        to[e] = q < n && k < N ? to_f(at[q * token + k]) : 0.f;
      }
      at += move * token;
    }
  }
};

// Adds one segment's own end to what went through it: h = exp(A sum) h + end.
template <typename T, int C, int NS, int HOP>
__device__ __forceinline__ void through(float2 (&h)[C][NS / 2], const float2 (&A2)[C][NS / 2], const ScanArgs& a, const ScanSegs& g,
                                        int b, int i, int c0, int ch, int n0, int width) {
  const int64_t at = (static_cast<int64_t>(b) * g.nseg + i) * a.D + c0;
  float2 e[C][NS / 2];
  load_states<C, NS, HOP>(e, g.ends + at * a.N, a.N, ch, n0, width);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const float sum = ch + c < width ? g.sums[at + ch + c] : 0.f;
#pragma unroll
    for (int j = 0; j < NS / 2; ++j) h[c][j] = fma2(decay2<T>(A2[c][j], sum), h[c][j], e[c][j]);
  }
}

// ---------------------------------------------------------------------------
// forward, and what a segment leaves by itself in either direction
// ---------------------------------------------------------------------------
// A warp works alone: one or three tiles of 8 or 16 tokens of its channels are on their way
// into shared memory while it works on the one before; it leaves the steps in shared memory,
// runs the recurrence and finishes the outputs, with no barrier but its own.  Nothing but the
// states, their rates and the token at hand stays in registers, so that two or three warps a
// scheduler hide the latencies of each other.  Eight states a lane: at 16 states two lanes
// share a channel, and a sum over the states is one exchange.
//
// Measured, bf16: 8 x 2048 tokens of 2048 channels and 16 states, keeping for the gradients,
// 255 us (3.7 TB/s with what it keeps; 57 us are the exponentials alone, 79 the
// multiply-adds), 8 x 1000 tokens without keeping 108 us.
// Warps an SM holds: up to 16 states 12 (the former 255 us; 16, with 128 registers, 288);
// above that the two channels a lane need more than 168 registers, and 8 leave 255 (8 x 1024
// tokens of 2048 channels and 64 states, 499 us with 12, which spill 36 bytes, 397 with 8,
// 350 since they fit the shared memory).  Kept states that go out through shared memory by
// bulk copies, one a warp and four tokens, cost more than the lanes' stores: 311 us.
constexpr int fwd_warps(int SL) { return SL > 2 ? 8 : 12; }
constexpr int kFwdNS = 8, kStretch = 8;
enum { kInfer, kTrain, kAlone, kAloneBack };

template <typename T, int SL, int C, bool OUT>
struct Fwd {
  static constexpr int CL = 32 / SL, CT = CL * C, NP = SL * kFwdNS, P = kFwdNS / 2;
  static constexpr int VC = CT / 8, ROWS = 32 / VC, TT = ROWS < 16 ? ROWS : 16;     // an item a lane
  static_assert(TT % kStretch == 0 && kStretch % kScanKeep == 0, "whole stretches, whole distances between kept states");
  static constexpr int LD = CT + 4;      // a row in shared memory: rows of a store on banks of their own
  // Tiles on their way.  Where the warps that an SM can hold by their registers would not
  // fit its shared memory with three, one: fp32, 8 x 1024 tokens of 2048 channels, 32 states
  // 176 us, 240 with three; 64 states bf16 350 and 399, fp32 432 and 530; fp32, 16 states, 4
  // x 2048 tokens 150 and 190.  With few short tiles a warp (8 states) one is too late: 137
  // us, 100 with three.
  static constexpr int AHEAD = SL > 2 || (SL == 2 && sizeof(T) == 4) ? 1 : 3;
  using R = Rows<T, TT, NP>;
  Raw<T, 8> raw[AHEAD + 1][3][32];       // x, dt, z of a lane's item
  typename R::Stage rawB[AHEAD + 1], rawC[OUT ? AHEAD + 1 : 1];
  float bias[CT], skip[CT];
  float dt[TT][LD], dx[TT][LD], y[OUT ? TT : 1][LD];
  float B[TT][NP], C_[OUT ? TT : 1][NP];
};

// Sums C values over the SL state lanes; lane sl < C ends up with value sl (all of them
// where SL is one).
template <int SL, int C>
__device__ __forceinline__ void over_states(float (&v)[C], int sl) {
  constexpr int CL = 32 / SL;
  if constexpr (SL > 1) {
    int m = CL;
    if constexpr (C == 2) {
      const bool up = sl & 1;
      v[0] = (up ? v[1] : v[0]) + __shfl_xor_sync(kFull, up ? v[0] : v[1], m);
      m *= 2;
    }
#pragma unroll
    for (; m < 32; m *= 2) v[0] += __shfl_xor_sync(kFull, v[0], m);
  }
}

template <typename T, int SL, int C, int MODE>
__global__ void __launch_bounds__(32, fwd_warps(SL)) scan_fwd_kernel(const ScanFwdArgs f) {
  constexpr bool OUT = MODE == kInfer || MODE == kTrain, BACK = MODE == kAloneBack;
  using W = Fwd<T, SL, C, OUT>;
  constexpr int CT = W::CT, NP = W::NP, P = W::P, NS = kFwdNS, HOP = 4 * SL, TT = W::TT;
  __shared__ __align__(16) W s;
  const ScanArgs& a = f.a;
  // forward the last segment, backward the first has no other that wants its end
  Where<CT> w(a, OUT ? f.g.nseg : f.g.nseg - 1, blockIdx.x);
  if (BACK) ++w.seg;
  const int lane = threadIdx.x, cl = lane % W::CL, sl = lane / W::CL, ch = cl * C, n0 = sl * 4;
  const int row = lane / W::VC, col = lane % W::VC * 8;
  const bool in = col < w.width && row < TT, gate = a.z != nullptr;
  const int len = a.len ? a.len[w.b] : a.T, begin = w.seg * f.g.len, end = begin + f.g.len < a.T ? begin + f.g.len : a.T;
  const int last = len < end ? len : end;
  const int64_t bD = static_cast<int64_t>(w.b) * a.D + w.c0;
  const int tiles = (end - begin + TT - 1) / TT;
  const int first = BACK ? begin + (tiles - 1) * TT : begin, move = BACK ? -TT : TT;

  // where the lane's item of the tile to come lies; backward, x is the gradient of the
  // gated output, and B is C
  const int64_t hop = a.bfirst ? move : static_cast<int64_t>(move) * a.B, row0 = a.row(w.b, first + row);
  const T *px = static_cast<const T*>(a.x) + row0 * a.x_row + w.c0 + col, *pdt = static_cast<const T*>(a.dt) + row0 * a.dt_row + w.c0 + col,
          *pz = static_cast<const T*>(a.z) + row0 * a.z_row + w.c0 + col;
  Rows<T, TT, NP> rB(a, a.Bm, a.B_row, w.b, w.g, first, lane), rC(a, OUT ? a.Cm : a.Bm, OUT ? a.C_row : a.B_row, w.b, w.g, first, lane);
  auto fetch = [&](int t0, int stage) {
    const bool ok = in && t0 + row < last;
    async_item<T>(&s.raw[stage][0][lane], px, 0, ok, a.A);
    async_item<T>(&s.raw[stage][1][lane], pdt, 0, ok, a.A);
    if ((OUT || BACK) && gate) async_item<T>(&s.raw[stage][2][lane], pz, 0, ok, a.A);
    rB.load(s.rawB[stage], last - t0, move, lane, a.A);
    if (OUT) rC.load(s.rawC[stage], last - t0, move, lane, a.A);
    asm volatile("cp.async.commit_group;" ::: "memory");
    px += hop * a.x_row;
    pdt += hop * a.dt_row;
    pz += hop * a.z_row;
  };
  // tiles beyond the segment are fetched as zeros: nothing is read for them
#pragma unroll
  for (int k = 0; k < W::AHEAD; ++k) fetch(k < tiles ? first + k * move : last, k);
  for (int c = lane; c < CT; c += 32) {
    s.bias[c] = a.bias && c < w.width ? a.bias[w.c0 + c] : 0.f;
    s.skip[c] = OUT && a.skip && c < w.width ? a.skip[w.c0 + c] : 0.f;
  }
  float2 A2[C][P], h[C][P], sum[4];
  load_rates<C, NS, HOP>(A2, a, w.c0, ch, n0, w.width);
  load_states<C, NS, HOP>(h, OUT && f.h0 ? f.h0 + bD * a.N : nullptr, a.N, ch, n0, w.width);
  if (MODE == kAlone && f.first && w.seg == 0) {
    float2 h0[C][P];
    load_states<C, NS, HOP>(h0, f.h0 + bD * a.N, a.N, ch, n0, w.width);
    store_states<C, NS, HOP>(h0, f.first + bD * a.N, a.N, ch, n0, w.width);
  }
  if (OUT)
#pragma unroll 2
    for (int i = 0; i < w.seg && i * f.g.len < len; ++i) through<T, C, NS, HOP>(h, A2, a, f.g, w.b, i, w.c0, ch, n0, w.width);
#pragma unroll
  for (int j = 0; j < 4; ++j) sum[j] = both(0.f);
  float* pu = MODE == kTrain && gate ? f.ungated + row0 * a.D + w.c0 + col : nullptr;
  T* py = static_cast<T*>(f.y) + row0 * a.D + w.c0 + col;
  float* pk = MODE == kTrain ? f.kept + ((static_cast<int64_t>(w.b) * a.keeps() + begin / kScanKeep) * a.D + w.c0) * a.N : nullptr;
  __syncwarp();
  for (int k = 0; k < tiles; ++k) {
    const int stage = k % (W::AHEAD + 1), t0 = first + k * move, n = last - t0;
    asm volatile("cp.async.wait_group %0;" :: "n"(W::AHEAD - 1) : "memory");
    if (W::ROWS == TT || row < TT) {
      const Raw<T, 8> x = s.raw[stage][0][lane], dt = s.raw[stage][1][lane];
      float2 d[4], u[4];
      lds2<4>(d, &s.bias[col]);
#pragma unroll
      for (int j = 0; j < 4; ++j) d[j] = add2(dt.pair(j), d[j]);
      if (a.softplus)
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = softplus2(d[j]);
      if (row >= n)                                    // behind the last token: changes nothing
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = both(0.f);
      store_vec<float, 8>(&s.dt[row][col], d);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u[j] = BACK ? x.pair(j) : mul2(d[j], x.pair(j));
        if (!OUT) sum[j] = add2(sum[j], d[j]);
      }
      if (BACK && gate) {
        const Raw<T, 8> z = s.raw[stage][2][lane];
#pragma unroll
        for (int j = 0; j < 4; ++j) u[j] = mul2(u[j], mul2(z.pair(j), sigmoid2(z.pair(j))));
      }
      store_vec<float, 8>(&s.dx[row][col], u);
    }
    rB.store(&s.B[0][0], s.rawB[stage], n, move, lane);
    if (OUT) rC.store(&s.C_[0][0], s.rawC[stage], n, move, lane);
    __syncwarp();
    fetch(k + W::AHEAD < tiles ? t0 + W::AHEAD * move : last, (k + W::AHEAD) % (W::AHEAD + 1));
#pragma unroll 1
    for (int half = 0; half < TT; half += kStretch) {
      // outputs are written when the stretch is through: a store among them would hold back
      // the loads behind it
      float y[OUT ? kStretch : 1][SL == 1 ? C : 1];
#pragma unroll
      for (int q = 0; q < kStretch; ++q) {
        if (MODE == kTrain && q % kScanKeep == 0 && t0 + half + q < end) {
          store_states<C, NS, HOP>(h, pk, a.N, ch, n0, w.width);
          pk += static_cast<int64_t>(a.D) * a.N;
        }
        const int t = BACK ? TT - 1 - half - q : half + q;
        const bool t4 = q % 4 == (BACK ? 3 : 0);             // t is a multiple of four
        float d[C], u[C], yc[C];
        float2 Bv[P], Cv[P];
        lds<C>(d, &s.dt[t][ch]);
        lds<C>(u, &s.dx[t][ch]);
        lds2<P, HOP>(Bv, &s.B[t][n0]);
        if (OUT) lds2<P, HOP>(Cv, &s.C_[t][n0]);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float2 r = both(0.f);
#pragma unroll
          for (int j = 0; j < P; ++j) {
            const float2 e = t4 ? decay2<T, 4>(A2[c][j], d[c]) : decay2<T, 0>(A2[c][j], d[c]);
            if (BACK) h[c][j] = mul2(e, fma2(Bv[j], both(u[c]), h[c][j]));
            else h[c][j] = fma2(e, h[c][j], mul2(Bv[j], both(u[c])));
            if (OUT) r = j ? fma2(Cv[j], h[c][j], r) : mul2(Cv[j], h[c][j]);
          }
          yc[c] = r.x + r.y;
        }
        if (OUT) {
          over_states<SL, C>(yc, sl);
#pragma unroll
          for (int c = 0; c < (SL == 1 ? C : 1); ++c) y[q][c] = yc[c];
        }
      }
      if (OUT && (SL <= C || sl < C))
#pragma unroll
        for (int t = 0; t < kStretch; ++t)
#pragma unroll
          for (int c = 0; c < (SL == 1 ? C : 1); ++c) s.y[half + t][ch + (SL == 1 ? c : sl)] = y[t][c];
    }
    if (OUT) {
      __syncwarp();
      if (in && t0 + row < end) {
        const Raw<T, 8> x = s.raw[stage][0][lane];
        float2 v[4], sk[4];
        lds2<4>(v, &s.y[row][col]);
        lds2<4>(sk, &s.skip[col]);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = fma2(sk[j], x.pair(j), v[j]);
        if (gate) {
          const Raw<T, 8> z = s.raw[stage][2][lane];
          if (MODE == kTrain) store_vec<float, 8>(pu, v);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = mul2(v[j], mul2(z.pair(j), sigmoid2(z.pair(j))));
        }
        if (row >= n)
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = both(0.f);
        store_vec<T, 8>(py, v);
      }
      py += hop * a.D;
      if (MODE == kTrain) pu += hop * a.D;
    } else {
      __syncwarp();
    }
  }
  if (OUT) {
    if (f.hT && end == a.T) store_states<C, NS, HOP>(h, f.hT + bD * a.N, a.N, ch, n0, w.width);
    return;
  }
  const int64_t at = (static_cast<int64_t>(w.b) * f.g.nseg + w.seg) * a.D + w.c0;
  store_states<C, NS, HOP>(h, f.g.ends + at * a.N, a.N, ch, n0, w.width);
  // the rows' sums of steps, in a fixed order
#pragma unroll
  for (int m = W::VC; m < 32; m <<= 1)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      sum[j].x += __shfl_xor_sync(kFull, sum[j].x, m);
      sum[j].y += __shfl_xor_sync(kFull, sum[j].y, m);
    }
  if (row == 0 && in)
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<float2*>(f.g.sums + at + col + 2 * j) = sum[j];
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// A warp goes through its segment from the last token to the first, four tokens at a time:
// it computes their decays and states again from the kept one, holds them in registers, and
// runs the gradient g of the state back through them:
//     g += dy_t C_t;  dC_t += dy_t h_t;  dB_t += g delta_t x_t;  s1_t = sum g B_t
//     g = a_t g;  P = g h_{t-1};  s2_t = sum P A;  dA += P delta_t
// then, channel by channel, dx = delta s1 + D dy, ddelta = x s1 + s2, and dz from y as the
// forward kept it before the gate.  Four channels and four states a lane: sums over the
// states (of s1 and s2) and over the channels (of dB and dC) then take the fewest
// exchanges together.  Inputs and kept states of the next tile of eight tokens are on
// their way into shared memory meanwhile.
//
// Measured, bf16: 8 x 2048 tokens of 2048 channels and 16 states 612 us: 100 what the
// segments leave by themselves, 485 this kernel (2.9 TB/s; 57 us are its exponentials
// alone, 215 its multiply-adds), 23 and 5 the sums behind it.  Issue bounds it, 55 % of
// the slots with two warps a scheduler: states and decays of the four tokens take the
// registers.  Kept states eight tokens apart leave no room for the decays, and computing
// them twice cost 110 us.
// Warps an SM: what the registers allow.  Shared memory leaves as many in bf16 above 8 states,
// 5 up to there, and in fp32 4, 6, 7 and 6 at 8, 16, 32 and 64 states.
constexpr int kBwdWarps = 8;
constexpr int kBT = 8, kBSub = kScanKeep, kBNS = 4, kBC = 4;

template <typename T, int SL>
struct Bwd {
  static constexpr int CL = 32 / SL, CT = CL * kBC, NP = SL * kBNS, P = kBNS / 2;
  static constexpr int VC = CT / 8, ROWS = 32 / VC, IT = kBT / ROWS > 0 ? kBT / ROWS : 1, LD = CT + 4;
  static constexpr int OS = SL == 2 ? 2 : 1;               // channels of a lane's sums over states
  static constexpr int OC = CL >= 8 ? 1 : 8 / CL;          // states of a lane's sums over channels
  Raw<T, 8> raw[2][4][IT][32];                   // x, dt, z, dy of a lane's items
  Raw<float, 8> y[2][IT][32];
  typename Rows<T, kBT, NP>::Stage rawB[2], rawC[2];
  float4 kept[2][kBT / kBSub][kBC][32];
  float bias[CT], skip[CT];
  float dt[kBT][LD], dx[kBT][LD], dy[kBT][LD], sg[kBT][LD], s1[kBT][LD], s2[kBT][LD];
  float B[kBT][NP], C[kBT][NP];
  float4 acc[4][32];                             // a lane's sums for dD and the bias
};

// Sums four values over the SL state lanes: lane sl < 4 ends up with that of channel
// 2 (sl & 1) + (sl >> 1), or, where SL is two, with two of them.
template <int SL>
__device__ __forceinline__ void sum_states(const float2 (&a)[2], int sl, float (&r)[SL == 2 ? 2 : 1]) {
  constexpr int CL = 32 / SL;
  const bool up = sl & 1;
  float v = (up ? a[1].x : a[0].x) + __shfl_xor_sync(kFull, up ? a[0].x : a[1].x, CL);
  const float u = (up ? a[1].y : a[0].y) + __shfl_xor_sync(kFull, up ? a[0].y : a[1].y, CL);
  if constexpr (SL == 2) {
    r[0] = v;
    r[1] = u;
  } else {
    const bool odd = sl & 2;
    v = (odd ? u : v) + __shfl_xor_sync(kFull, odd ? v : u, 2 * CL);
#pragma unroll
    for (int m = 4 * CL; m < 32; m *= 2) v += __shfl_xor_sync(kFull, v, m);
    r[0] = v;
  }
}
// Sums dB and dC (four states each) over the CL channel lanes: lane cl ends up with OC
// states of one of them.
template <int CL, int OC>
__device__ __forceinline__ void sum_channels(const float2 (&dB)[2], const float2 (&dC)[2], int cl, float (&r)[OC]) {
  const bool up = cl & 1;
  float v[4];
  const float b[4] = {dB[0].x, dB[0].y, dB[1].x, dB[1].y}, c[4] = {dC[0].x, dC[0].y, dC[1].x, dC[1].y};
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (up ? c[i] : b[i]) + __shfl_xor_sync(kFull, up ? b[i] : c[i], 1);
  if constexpr (CL > 2) {
    const bool hi = cl & 2;
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = (hi ? v[i + 2] : v[i]) + __shfl_xor_sync(kFull, hi ? v[i] : v[i + 2], 2);
  }
  if constexpr (CL > 4) {
    const bool top = cl & 4;
    v[0] = (top ? v[1] : v[0]) + __shfl_xor_sync(kFull, top ? v[0] : v[1], 4);
#pragma unroll
    for (int m = 8; m < CL; m *= 2) v[0] += __shfl_xor_sync(kFull, v[0], m);
  }
#pragma unroll
  for (int i = 0; i < OC; ++i) r[i] = v[i];
}

template <typename T, int SL>
__global__ void __launch_bounds__(32, kBwdWarps) scan_bwd_kernel(const ScanBwdArgs p) {
  using W = Bwd<T, SL>;
  constexpr int CT = W::CT, NP = W::NP, P = W::P, C = kBC, NS = kBNS, TT = kBT, CL = W::CL;
  __shared__ __align__(16) W s;
  const ScanArgs& a = p.a;
  const rnn_scan_grad_t& out = p.grad;
  const int lane = threadIdx.x;
  const Where<CT> w(a, p.g.nseg, blockIdx.x);
  const int cl = lane % CL, sl = lane / CL, ch = cl * C, n0 = sl * NS;
  const int row = lane / W::VC, col = lane % W::VC * 8;
  const bool in = col < w.width && row < TT, gate = a.z != nullptr;
  const int len = a.len ? a.len[w.b] : a.T, begin = w.seg * p.g.len, end = begin + p.g.len < a.T ? begin + p.g.len : a.T;
  const int64_t bD = static_cast<int64_t>(w.b) * a.D + w.c0;
  const int tiles = (end - begin + TT - 1) / TT;
  const int last = len < end ? len : end, first = begin + (tiles - 1) * TT;

  // where the lane's items of the tile to come lie, and a token's distance
  const int64_t hop = a.bfirst ? 1 : a.B, row0 = a.row(w.b, first + row);
  const T *px = static_cast<const T*>(a.x) + row0 * a.x_row + w.c0 + col, *pdt = static_cast<const T*>(a.dt) + row0 * a.dt_row + w.c0 + col,
          *pz = static_cast<const T*>(a.z) + row0 * a.z_row + w.c0 + col, *pdy = static_cast<const T*>(p.dy) + row0 * a.D + w.c0 + col;
  const float* py = p.ungated + row0 * a.D + w.c0 + col;
  const int64_t DN = static_cast<int64_t>(a.D) * a.N;
  const float* pk = p.kept + (static_cast<int64_t>(w.b) * a.keeps() + first / kBSub) * DN + static_cast<int64_t>(w.c0 + ch) * a.N + n0;
  Rows<T, TT, NP> rB(a, a.Bm, a.B_row, w.b, w.g, first, lane), rC(a, a.Cm, a.C_row, w.b, w.g, first, lane);
  auto fetch = [&](int t0, int stage) {
#pragma unroll
    for (int i = 0; i < W::IT; ++i) {
      const bool ok = in && t0 + row + i * W::ROWS < last;
      const int64_t r = i * W::ROWS * hop;
      async_item<T>(&s.raw[stage][0][i][lane], px, r * a.x_row, ok, a.A);
      async_item<T>(&s.raw[stage][1][i][lane], pdt, r * a.dt_row, ok, a.A);
      async_item<T>(&s.raw[stage][3][i][lane], pdy, r * a.D, ok, a.A);
      if (gate) {
        async_item<T>(&s.raw[stage][2][i][lane], pz, r * a.z_row, ok, a.A);
        async_item<float>(&s.y[stage][i][lane], py, r * a.D, ok, a.A);
      }
    }
    px -= TT * hop * a.x_row;
    pdt -= TT * hop * a.dt_row;
    pz -= TT * hop * a.z_row;
    pdy -= TT * hop * a.D;
    py -= TT * hop * a.D;
#pragma unroll
    for (int q = 0; q < TT / kBSub; ++q) {
      const float* from = pk + q * DN;
      const bool on = n0 < a.N && t0 + q * kBSub < end;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const bool ok = on && ch + c < w.width;
        async16(&s.kept[stage][q][c][lane], ok ? from : a.A, ok);
        from += a.N;
      }
    }
    pk -= TT / kBSub * DN;
    rB.load(s.rawB[stage], last - t0, -TT, lane, a.A);
    rC.load(s.rawC[stage], last - t0, -TT, lane, a.A);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  fetch(first, 0);
  for (int c = lane; c < CT; c += 32) {
    s.bias[c] = a.bias && c < w.width ? a.bias[w.c0 + c] : 0.f;
    s.skip[c] = a.skip && c < w.width ? a.skip[w.c0 + c] : 0.f;
  }
  float2 A2[C][P], g[C][P], dA[C][P];
  load_rates<C, NS, 4>(A2, a, w.c0, ch, n0, w.width);
  load_states<C, NS, 4>(g, p.dhT ? p.dhT + bD * a.N : nullptr, a.N, ch, n0, w.width);
#pragma unroll 2
  for (int i = p.g.nseg - 1; i > w.seg; --i)
    if (i * p.g.len < len) through<T, C, NS, 4>(g, A2, a, p.g, w.b, i, w.c0, ch, n0, w.width);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < P; ++j) dA[c][j] = both(0.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) s.acc[i][lane] = make_float4(0.f, 0.f, 0.f, 0.f);
  // a token's sums over the warp's channels go to memory as they are
  const int on = CL >= 8 ? (cl & 1) * NP + (cl & 2) + ((cl >> 2) & 1) : CL == 4 ? (cl & 1) * NP + (cl & 2) : cl * NP;
  const int64_t bc_token = static_cast<int64_t>(a.G) * Where<CT>::per_group(a) * (2 * NP);
  float* pbc = p.bc + (static_cast<int64_t>(w.b) * a.T + first) * bc_token +
               (static_cast<int64_t>(w.g) * Where<CT>::per_group(a) + w.tile) * (2 * NP) + n0 + on;
  int64_t po = row0 * a.D + w.c0 + col;
  __syncwarp();

  for (int k = 0; k < tiles; ++k) {
    const int stage = k & 1, t0 = first - k * TT, n = last - t0;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
    for (int i = 0; i < W::IT; ++i) {
      const int t = row + i * W::ROWS;
      if (W::ROWS > TT && t >= TT) break;
      const Raw<T, 8> x = s.raw[stage][0][i][lane], dt = s.raw[stage][1][i][lane], dy = s.raw[stage][3][i][lane];
      float2 d[4], u[4], o[4];
      lds2<4>(d, &s.bias[col]);
#pragma unroll
      for (int j = 0; j < 4; ++j) d[j] = add2(dt.pair(j), d[j]);
      if (a.softplus)
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = softplus2(d[j]);
      if (t >= n)                                      // behind the last token: changes nothing
#pragma unroll
        for (int j = 0; j < 4; ++j) d[j] = both(0.f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u[j] = mul2(d[j], x.pair(j));
        o[j] = dy.pair(j);
      }
      store_vec<float, 8>(&s.dt[t][col], d);
      store_vec<float, 8>(&s.dx[t][col], u);
      if (gate) {
        const Raw<T, 8> z = s.raw[stage][2][i][lane];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          d[j] = sigmoid2(z.pair(j));
          o[j] = mul2(o[j], mul2(z.pair(j), d[j]));
        }
        store_vec<float, 8>(&s.sg[t][col], d);
      }
      store_vec<float, 8>(&s.dy[t][col], o);
    }
    rB.store(&s.B[0][0], s.rawB[stage], n, -TT, lane);
    rC.store(&s.C[0][0], s.rawC[stage], n, -TT, lane);
    __syncwarp();
    if (k + 1 < tiles) fetch(t0 - TT, stage ^ 1);
#pragma unroll 1
    for (int q0 = TT - kBSub; q0 >= 0; q0 -= kBSub) {
      // the states of these tokens, again
      float2 h[kBSub + 1][C][P];
      float2 e[kBSub][C][P];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float4 q = s.kept[stage][q0 / kBSub][c][lane];
        h[0][c][0] = make_float2(q.x, q.y);
        h[0][c][1] = make_float2(q.z, q.w);
      }
#pragma unroll
      for (int q = 0; q < kBSub; ++q) {
        float d[C], u[C];
        float2 Bv[P];
        lds<C>(d, &s.dt[q0 + q][ch]);
        lds<C>(u, &s.dx[q0 + q][ch]);
        lds2<P>(Bv, &s.B[q0 + q][n0]);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int j = 0; j < P; ++j) {
            e[q][c][j] = q % 4 ? decay2<T, 0>(A2[c][j], d[c]) : decay2<T, 4>(A2[c][j], d[c]);
            h[q + 1][c][j] = fma2(e[q][c][j], h[q][c][j], mul2(Bv[j], both(u[c])));
          }
      }
      // sums are written when the tokens are through: a store among them would hold back the
      // loads behind it
      float o1[kBSub][W::OS], o2[kBSub][W::OS], oc[kBSub][W::OC];
#pragma unroll
      for (int q = kBSub - 1; q >= 0; --q) {
        const int t = q0 + q;
        float d[C], u[C], o[C];
        float2 Bv[P], Cv[P], dB[P], dC[P], s1[C / 2], s2[C / 2];
        lds<C>(d, &s.dt[t][ch]);
        lds<C>(u, &s.dx[t][ch]);
        lds<C>(o, &s.dy[t][ch]);
        lds2<P>(Bv, &s.B[t][n0]);
        lds2<P>(Cv, &s.C[t][n0]);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float2 q1, q2;
#pragma unroll
          for (int j = 0; j < P; ++j) {
            g[c][j] = fma2(Cv[j], both(o[c]), g[c][j]);
            dC[j] = c ? fma2(h[q + 1][c][j], both(o[c]), dC[j]) : mul2(h[q + 1][c][j], both(o[c]));
            dB[j] = c ? fma2(g[c][j], both(u[c]), dB[j]) : mul2(g[c][j], both(u[c]));
            q1 = j ? fma2(g[c][j], Bv[j], q1) : mul2(g[c][j], Bv[j]);
            g[c][j] = mul2(e[q][c][j], g[c][j]);
            const float2 r = mul2(g[c][j], h[q][c][j]);
            q2 = j ? fma2(r, A2[c][j], q2) : mul2(r, A2[c][j]);
            dA[c][j] = fma2(r, both(d[c]), dA[c][j]);
          }
          (c & 1 ? s1[c / 2].y : s1[c / 2].x) = q1.x + q1.y;
          (c & 1 ? s2[c / 2].y : s2[c / 2].x) = q2.x + q2.y;
        }
        sum_states<SL>(s1, sl, o1[q]);
        sum_states<SL>(s2, sl, o2[q]);
        sum_channels<CL, W::OC>(dB, dC, cl, oc[q]);
      }
      const int och = ch + (SL == 2 ? 2 * sl : 2 * (sl & 1) + ((sl >> 1) & 1));
      float* to = pbc + q0 * bc_token;
#pragma unroll
      for (int q = 0; q < kBSub; ++q) {
        if (SL <= 4 || sl < 4)
#pragma unroll
          for (int i = 0; i < W::OS; ++i) {
            s.s1[q0 + q][och + i] = o1[q][i];
            s.s2[q0 + q][och + i] = o2[q][i];
          }
        if (p.bc && (CL <= 8 || cl < 8) && t0 + q0 + q < end)
#pragma unroll
          for (int i = 0; i < W::OC; ++i) to[i] = q0 + q < n ? oc[q][i] : 0.f;
        to += bc_token;
      }
    }
    pbc -= TT * bc_token;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < W::IT; ++i) {
      const int t = row + i * W::ROWS;
      if (!in || t >= TT || t0 + t >= end) break;
      const Raw<T, 8> x = s.raw[stage][0][i][lane], dt = s.raw[stage][1][i][lane], dy = s.raw[stage][3][i][lane];
      const int64_t at = po + i * W::ROWS * hop * a.D;
      float2 v[4], o[4], q1[4], r[4];
      lds2<4>(o, &s.dy[t][col]);
      lds2<4>(q1, &s.s1[t][col]);
      lds2<4>(v, &s.dt[t][col]);
      lds2<4>(r, &s.skip[col]);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = t < n ? fma2(v[j], q1[j], mul2(r[j], o[j])) : both(0.f);
      if (out.dx) store_vec<T, 8>(static_cast<T*>(out.dx) + at, v);
      lds2<4>(v, &s.s2[t][col]);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = fma2(x.pair(j), q1[j], mul2(v[j], both(kLn2)));
      if (a.softplus) {
        lds2<4>(r, &s.bias[col]);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = mul2(v[j], sigmoid2(add2(dt.pair(j), r[j])));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = t < n ? v[j] : both(0.f);
        o[j] = t < n ? mul2(o[j], x.pair(j)) : both(0.f);
      }
      if (out.ddt) store_vec<T, 8>(static_cast<T*>(out.ddt) + at, v);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float4 q = s.acc[j][lane];
        s.acc[j][lane] = make_float4(q.x + o[2 * j].x, q.y + o[2 * j].y, q.z + o[2 * j + 1].x, q.w + o[2 * j + 1].y);
        q = s.acc[2 + j][lane];
        s.acc[2 + j][lane] = make_float4(q.x + v[2 * j].x, q.y + v[2 * j].y, q.z + v[2 * j + 1].x, q.w + v[2 * j + 1].y);
      }
      if (gate && out.dz) {
        const Raw<T, 8> z = s.raw[stage][2][i][lane];
        const Raw<float, 8> y = s.y[stage][i][lane];
        lds2<4>(r, &s.sg[t][col]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // sigma + z sigma (1 - sigma)
          v[j] = mul2(mul2(dy.pair(j), y.pair(j)), fma2(mul2(z.pair(j), r[j]), make_float2(1.f - r[j].x, 1.f - r[j].y), r[j]));
          if (t >= n) v[j] = both(0.f);
        }
        store_vec<T, 8>(static_cast<T*>(out.dz) + at, v);
      }
    }
    po -= TT * hop * a.D;
  }
  if (out.dh0 && begin == 0) store_states<C, NS, 4>(g, static_cast<float*>(out.dh0) + bD * a.N, a.N, ch, n0, w.width);
  const int64_t at = (static_cast<int64_t>(w.b) * p.g.nseg + w.seg) * a.D + w.c0;
  if (p.pA) store_states<C, NS, 4>(dA, p.pA + at * a.N, a.N, ch, n0, w.width);
  // the rows' sums, in order
  __syncwarp();
  for (int c = lane; c < w.width; c += 32) {
    float v = 0.f, u = 0.f;
    for (int r = 0; r < W::ROWS && r < TT; ++r) {
      const int l = r * W::VC + c / 8;
      v += reinterpret_cast<const float*>(&s.acc[(c & 7) / 4][l])[c & 3];
      u += reinterpret_cast<const float*>(&s.acc[2 + (c & 7) / 4][l])[c & 3];
    }
    if (p.pD) p.pD[at + c] = v;
    if (p.pbias) p.pbias[at + c] = u;
  }
}

// dB and dC: the sum over the warps of a group, a warp for each token and group: its lanes
// read whole rows of partial sums, 32 / V of them at a time (V vectors of four states a
// row), each lane in order and then the lanes in order.  Memory bounds it: 134 MB (16384
// tokens, 64 warps of 32 channels, 16 states) in 23 us, 5.8 TB/s.
template <typename T, int V>
__global__ void __launch_bounds__(256) scan_bc_kernel(const ScanArgs a, const float* bc, int parts, T* dB, T* dC) {
  constexpr int NP = 2 * V, SUB = 32 / V;
  const int64_t rows = static_cast<int64_t>(a.B) * a.T * a.G;
  const int lane = threadIdx.x & 31, k = lane % V * 4, sub = lane / V;
  for (int64_t r = blockIdx.x * 8LL + (threadIdx.x >> 5); r < rows; r += gridDim.x * 8LL) {
    const float* from = bc + (r * parts + sub) * (2 * NP) + k;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = sub; i < parts; i += SUB, from += SUB * 2 * NP) {
      const float4 q = *reinterpret_cast<const float4*>(from);
      v = make_float4(v.x + q.x, v.y + q.y, v.z + q.z, v.w + q.w);
    }
#pragma unroll
    for (int m = V; m < 32; m *= 2) {
      v.x += __shfl_xor_sync(kFull, v.x, m);
      v.y += __shfl_xor_sync(kFull, v.y, m);
      v.z += __shfl_xor_sync(kFull, v.z, m);
      v.w += __shfl_xor_sync(kFull, v.w, m);
    }
    T* out = k < NP ? dB : dC;
    const int n = k % NP;
    if (sub || n >= a.N || !out) continue;
    const int g = static_cast<int>(r % a.G);
    const int64_t bt = r / a.G;
    const int b = static_cast<int>(bt / a.T), t = static_cast<int>(bt - static_cast<int64_t>(b) * a.T);
    const float f[4] = {v.x, v.y, v.z, v.w};
    Vec4<T>::store(out + (a.row(b, t) * a.G + g) * a.N + n, f);
  }
}

// dA, dD and the bias's gradient: the sums over sequences and segments, in order.
__global__ void __launch_bounds__(128) scan_sum_kernel(const ScanBwdArgs p) {
  const ScanArgs& a = p.a;
  const int parts = a.B * p.g.nseg;
  const int64_t n[3] = {static_cast<int64_t>(a.D) * a.N, a.D, a.D};
  int64_t e = blockIdx.x * 128LL + threadIdx.x;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (e < n[k]) {
      const float* from = (k == 0 ? p.pA : k == 1 ? p.pD : p.pbias) + e;
      float* to = static_cast<float*>(k == 0 ? p.grad.dA : k == 1 ? p.grad.dD : p.grad.ddt_bias);
      if (!to) return;
      float v = 0.f;
#pragma unroll 8
      for (int b = 0; b < parts; ++b) v += from[b * n[k]];
      to[e] = v;
      return;
    }
    e -= n[k];
  }
}

// ---------------------------------------------------------------------------
// the serving step
// ---------------------------------------------------------------------------
// SL lanes have CH = min(SL, 4) channels, four states of each a lane.  A lane prepares one
// of the channels (its step, and at the end its output) and hands the step to the others.
// Memory bounds it, the states in and out: 256 sequences of 4096 channels and 16 states in
// 28 us, 5.2 TB/s (a cold call 33; 35 with 56 registers a thread for more warps, 45 with
// 42); four tokens of each in 56 us (cold 59), where issue does.
constexpr int kStepThreads = 128;
template <typename T, int SL>
__global__ void __launch_bounds__(kStepThreads) scan_step_kernel(const ScanStepArgs p) {
  const ScanArgs& a = p.a;
  constexpr int CH = SL < 4 ? SL : 4, PER = kStepThreads / SL * CH;          // channels a CTA
  const int dg = a.D / a.G, per = (dg + PER - 1) / PER, all = per * a.G;
  const int b = blockIdx.x / all, tile = blockIdx.x - b * all, g = tile / per, sl = threadIdx.x % SL, n0 = sl * 4;
  const int base = (tile - g * per) * PER + threadIdx.x / SL * CH, width = dg - base;    // of the group's channels; may be <= 0
  const int mine = sl % CH, d = g * dg + base + mine;                        // the channel that the lane prepares
  const bool own = mine < width, states = n0 < a.N;
  const int slot = p.slots ? p.slots[b] : b;
  const bool live = slot >= 0 && slot < p.num_slots;
  const int n = live ? a.len ? a.len[b] : a.T : 0;
  const int64_t at = static_cast<int64_t>(g * dg + base) * a.N + n0;
  float* state = p.state + static_cast<int64_t>(live ? slot : 0) * a.D * a.N + at;
  float4 h[CH], A[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    h[i] = A[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < width && n > 0 && states) {
      h[i] = *reinterpret_cast<const float4*>(state + static_cast<int64_t>(i) * a.N);
      A[i] = *reinterpret_cast<const float4*>(a.A + at + static_cast<int64_t>(i) * a.N);
    }
  }
  const float bias = own && a.bias ? a.bias[d] : 0.f, skip = own && a.skip ? a.skip[d] : 0.f;
  for (int t = 0; t < a.T; ++t) {
    const int64_t r = a.row(b, t);
    const bool on = t < n;
    if (!on) {
      if (own && sl < CH) static_cast<T*>(p.y)[r * a.D + d] = from_f<T>(0.f);
      continue;                                          // the CTA's threads have one sequence
    }
    float xv = 0.f, dv = 0.f, zv = 0.f, Bv[4] = {}, Cv[4] = {};
    if (own) {
      xv = to_f(static_cast<const T*>(a.x)[r * a.x_row + d]);
      dv = to_f(static_cast<const T*>(a.dt)[r * a.dt_row + d]);
      if (a.z) zv = to_f(static_cast<const T*>(a.z)[r * a.z_row + d]);
    }
    if (states) {
      const T *Bp = static_cast<const T*>(a.Bm) + r * a.B_row + g * a.N + n0, *Cp = static_cast<const T*>(a.Cm) + r * a.C_row + g * a.N + n0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        Bv[k] = to_f(Bp[k]);
        Cv[k] = to_f(Cp[k]);
      }
    }
    dv += bias;
    if (a.softplus) dv = softplus2(both(dv)).x;
    const float e = dv * kLog2e, u = dv * xv;
    // only a step next to zero needs it, and at the start of the kernel the rates would be
    // waited for before a token is asked for (28.1 us become 30.7)
    if (__any_sync(kFull, own && fabsf(e) < 1e-20f))
#pragma unroll
      for (int i = 0; i < CH; ++i) A[i] = make_float4(finite_rate(A[i].x), finite_rate(A[i].y), finite_rate(A[i].z), finite_rate(A[i].w));
    float y[CH];
    auto update = [&](auto adds) {
      const float slope = decltype(adds)::value ? kSlope * static_cast<float>(n - t < 4 ? n - t : 4) : 0.f;
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const float ei = __shfl_sync(kFull, e, i, SL), ui = __shfl_sync(kFull, u, i, SL);
        h[i].x = fmaf(decay1<T, decltype(adds)::value>(A[i].x, ei, slope), h[i].x, ui * Bv[0]);
        h[i].y = fmaf(decay1<T, decltype(adds)::value>(A[i].y, ei, slope), h[i].y, ui * Bv[1]);
        h[i].z = fmaf(decay1<T, decltype(adds)::value>(A[i].z, ei, slope), h[i].z, ui * Bv[2]);
        h[i].w = fmaf(decay1<T, decltype(adds)::value>(A[i].w, ei, slope), h[i].w, ui * Bv[3]);
        y[i] = fmaf(Cv[3], h[i].w, fmaf(Cv[2], h[i].z, fmaf(Cv[1], h[i].y, Cv[0] * h[i].x)));
      }
    };
    if (sizeof(T) == 4 && t % 4 == 0) update(std::true_type{});
    else update(std::false_type{});
    // lane sl of each four ends up with the sum of channel sl
    if constexpr (CH == 4) {
      const bool up = sl & 2;
#pragma unroll
      for (int i = 0; i < 2; ++i) y[i] = (up ? y[i + 2] : y[i]) + __shfl_xor_sync(kFull, up ? y[i] : y[i + 2], 2);
    }
    const bool odd = sl & 1;
    float v = (odd ? y[1] : y[0]) + __shfl_xor_sync(kFull, odd ? y[0] : y[1], 1);
#pragma unroll
    for (int m = 4; m < SL; m <<= 1) v += __shfl_xor_sync(kFull, v, m);
    if (own && sl < CH) {
      v = fmaf(skip, xv, v);
      if (a.z) v *= zv * sigmoid2(both(zv)).x;
      static_cast<T*>(p.y)[r * a.D + d] = from_f<T>(v);
    }
  }
  if (n > 0 && states)
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (i < width) *reinterpret_cast<float4*>(state + static_cast<int64_t>(i) * a.N) = h[i];
}

int check_launch() { return cudaGetLastError() == cudaSuccess ? 0 : RNN_CUDA_ERROR; }

// Lanes a channel: eight states each forward, four backward, rounded up to a power of two.
int fwd_lanes(int N) { return N <= 8 ? 1 : N <= 16 ? 2 : N <= 32 ? 4 : 8; }
int fwd_width(int N, bool split) { return (N <= 8 || (N <= 16 && !split) ? 32 : 64) / fwd_lanes(N); }
int bwd_width(int N) { return kBC * 16 / fwd_lanes(N); }
int per_group(const ScanArgs& a, int width) { return (a.D / a.G + width - 1) / width; }

template <typename T, int SL, int C>
int fwd(ScanFwdArgs f, cudaStream_t s, int* launches) {
  const unsigned warps = static_cast<unsigned>(f.a.B) * f.a.G * Where<32 / SL * C>::per_group(f.a);
  int rc;
  if (f.g.nseg > 1) {
    scan_fwd_kernel<T, SL, C, kAlone><<<warps * (f.g.nseg - 1), 32, 0, s>>>(f);
    if ((rc = check_launch())) return rc;
    ++*launches;
    if (f.first) f.h0 = f.first;
  }
  if (f.kept) scan_fwd_kernel<T, SL, C, kTrain><<<warps * f.g.nseg, 32, 0, s>>>(f);
  else scan_fwd_kernel<T, SL, C, kInfer><<<warps * f.g.nseg, 32, 0, s>>>(f);
  if (!(rc = check_launch())) ++*launches;
  return rc;
}
template <typename T>
int fwd_t(const ScanFwdArgs& f, cudaStream_t s, int* launches) {
  switch (fwd_lanes(f.a.N)) {
    case 1: return fwd<T, 1, 1>(f, s, launches);
    case 2: return f.g.nseg > 1 ? fwd<T, 2, 2>(f, s, launches) : fwd<T, 2, 1>(f, s, launches);
    case 4: return fwd<T, 4, 2>(f, s, launches);
    default: return fwd<T, 8, 2>(f, s, launches);
  }
}

template <typename T, int SL, int C>
int bwd(const ScanBwdArgs& p, cudaStream_t s, int* launches) {
  int rc;
  if (p.g.nseg > 1) {
    ScanFwdArgs f{};
    f.a = p.a;
    f.a.x = p.dy;
    f.a.x_row = p.a.D;
    f.a.Bm = p.a.Cm;
    f.a.B_row = p.a.C_row;
    f.g = p.g;
    const unsigned warps = static_cast<unsigned>(f.a.B) * f.a.G * Where<32 / SL * C>::per_group(f.a);
    scan_fwd_kernel<T, SL, C, kAloneBack><<<warps * (p.g.nseg - 1), 32, 0, s>>>(f);
    if ((rc = check_launch())) return rc;
    ++*launches;
  }
  static_assert(sizeof(Bwd<T, 2 * SL>) <= 48 * 1024, "a warp's tiles fit");
  const unsigned warps = static_cast<unsigned>(p.a.B) * p.a.G * Where<Bwd<T, 2 * SL>::CT>::per_group(p.a);
  scan_bwd_kernel<T, 2 * SL><<<warps * p.g.nseg, 32, 0, s>>>(p);
  if (!(rc = check_launch())) ++*launches;
  return rc;
}
template <typename T>
int bwd_t(const ScanBwdArgs& p, cudaStream_t s, int* launches) {
  const ScanArgs& a = p.a;
  int rc;
  switch (fwd_lanes(a.N)) {
    case 1: rc = bwd<T, 1, 1>(p, s, launches); break;
    case 2: rc = bwd<T, 2, 2>(p, s, launches); break;
    case 4: rc = bwd<T, 4, 2>(p, s, launches); break;
    default: rc = bwd<T, 8, 2>(p, s, launches);
  }
  if (rc) return rc;
  if (p.bc) {
    const int64_t blocks = (static_cast<int64_t>(a.B) * a.T * a.G + 7) / 8;
    const unsigned grid = static_cast<unsigned>(blocks < 32 * a.num_sms ? blocks : 32 * a.num_sms);
    const int parts = per_group(a, bwd_width(a.N));
    T *dB = static_cast<T*>(p.grad.dB), *dC = static_cast<T*>(p.grad.dC);
    switch (fwd_lanes(a.N)) {
      case 1: scan_bc_kernel<T, 4><<<grid, 256, 0, s>>>(a, p.bc, parts, dB, dC); break;
      case 2: scan_bc_kernel<T, 8><<<grid, 256, 0, s>>>(a, p.bc, parts, dB, dC); break;
      case 4: scan_bc_kernel<T, 16><<<grid, 256, 0, s>>>(a, p.bc, parts, dB, dC); break;
      default: scan_bc_kernel<T, 32><<<grid, 256, 0, s>>>(a, p.bc, parts, dB, dC);
    }
    if ((rc = check_launch())) return rc;
    ++*launches;
  }
  if (p.pA || p.pD || p.pbias) {
    const int64_t n = static_cast<int64_t>(a.D) * (a.N + 2);
    scan_sum_kernel<<<static_cast<unsigned>((n + 127) / 128), 128, 0, s>>>(p);
    if ((rc = check_launch())) return rc;
    ++*launches;
  }
  return 0;
}

template <typename T, int SL>
int step(const ScanStepArgs& p, cudaStream_t s) {
  constexpr int PER = kStepThreads / SL * (SL < 4 ? SL : 4);
  scan_step_kernel<T, SL><<<static_cast<unsigned>(p.a.B) * p.a.G * per_group(p.a, PER), kStepThreads, 0, s>>>(p);
  return check_launch();
}
template <typename T>
int step_t(const ScanStepArgs& p, cudaStream_t s) {
  if (p.a.N <= 8) return step<T, 2>(p, s);
  if (p.a.N <= 16) return step<T, 4>(p, s);
  return p.a.N <= 32 ? step<T, 8>(p, s) : step<T, 16>(p, s);
}

size_t up(size_t v) { return (v + 255) & ~static_cast<size_t>(255); }

ScanSegs segments(const ScanSplit& p, void* work) {
  char* w = static_cast<char*>(work);
  return {p.nseg, p.len, reinterpret_cast<float*>(w + p.ends), reinterpret_cast<float*>(w + p.sums)};
}

}  // namespace

namespace {

// n segments, as near as whole tiles allow.
ScanSplit split(const ScanArgs& a, int64_t n, bool first) {
  const int tiles = (a.T + 15) / 16;
  ScanSplit p{};
  p.len = (tiles + static_cast<int>(n) - 1) / static_cast<int>(n) * 16;
  p.nseg = (a.T + p.len - 1) / p.len;
  if (p.nseg == 1) return p;
  const size_t rows = static_cast<size_t>(a.B) * p.nseg * a.D;
  p.sums = up(rows * a.N * 4);
  p.first = p.sums + up(rows * 4);
  p.bytes = p.first + (first ? up(static_cast<size_t>(a.B) * a.D * a.N * 4) : 0);
  return p;
}

}  // namespace

// Segments.  Forward, a warp's tokens follow one another every 85 to 110 ns as long as a
// scheduler has at most two warps, and a second pass over the tokens (what each segment
// leaves by itself) costs half as much again.  So they begin below five warps an SM, and
// then have 32 channels a warp (two a lane: 1 x 16384 tokens of 4096 channels 500 us, 547
// with one a lane; 1.1 ms in one piece).  They fill the SMs once with as many warps as these
// hold: 12, above 16 states (registers) and in fp32 up to 8 states (shared memory) 8.  4 x
// 2048 tokens of 2048 channels, 16 states: bf16 141 us in 7 pieces, 164 in 4, 158 in one,
// fp32 150, 174, 172; 2 x 2048 tokens of 2048 channels, 8 states, fp32: 72 us with 8 warps
// an SM, 86 with 12.  Above 32 pieces it is 8 always, since each loads what all before it
// left (1 x 4096 tokens of 1024 channels, bf16, 70 us in 52 pieces, 59 in 37).  Fewer than
// five do not pay up to 16 states (8 x 1024 tokens of 2048 channels, 8 states, fp32: 108 us
// in one piece, 128 in three; training 121 and 148), above that fewer than three (2 x 1024
// tokens of 1024 channels, 64 states: 125 us in one piece, 104 in four; 4 x 1024 of 2048, 32
// states: 113 and 125 in two).  64 tokens each at least, so up to 16 states less than 320 tokens
// are one piece (1 x 300 tokens of 2048 channels, bf16, 16 states 23 us and 23 in four pieces,
// 8 states 30 and 17; in nine pieces of 32 tokens 17 and 13, but 4 x 300 25 and 29).
ScanSplit scan_split_forward(const ScanArgs& a, int is_bf16) {
  const int64_t all = static_cast<int64_t>(a.B) * a.G, wide = all * per_group(a, fwd_width(a.N, true));
  int64_t n = 1;
  if (all * per_group(a, fwd_width(a.N, false)) < 5 * a.num_sms) {
    n = (a.N > 16 || (a.N <= 8 && !is_bf16) ? 8 : 12) * a.num_sms / wide;
    if (n > 32) n = std::max<int64_t>(8 * a.num_sms / wide, 32);
    n = std::min<int64_t>(n, a.T / 64);
    if (n < (a.N <= 16 ? 5 : 3)) n = 1;
  }
  return split(a, n, true);
}

// Backward, reckoned with eight warps an SM (16 states: 512 warps, 2048 tokens, bf16, 744 us in
// one piece, 648 in 2, 625 in 8): from four warps an SM on it is in one piece, else it fills the
// SMs three times, with 32 tokens a segment at least (513 tokens of 3 x 528 channels, fp32: 50
// us, 60 with 64).  Where shared memory holds fewer warps it is the same rule, not measured.
ScanSplit scan_split_backward(const ScanArgs& a) {
  const int64_t warps = static_cast<int64_t>(a.B) * a.G * per_group(a, bwd_width(a.N));
  int64_t n = 1;
  if (warps < 4 * a.num_sms) n = std::min<int64_t>(3 * kBwdWarps * a.num_sms / warps, a.T / 32);
  return split(a, n < 3 ? 1 : n, false);
}

ScanReserve scan_reserve(const ScanArgs& a) {
  ScanReserve r{};
  r.ungated = up(static_cast<size_t>(a.B) * a.keeps() * a.D * a.N * 4);
  r.bytes = r.ungated + up(static_cast<size_t>(a.B) * a.T * a.D * 4);
  return r;
}

int launch_scan_forward(const ScanFwdArgs& f_, void* work, int is_bf16, cudaStream_t s, int* launches) {
  ScanFwdArgs f = f_;
  const ScanSplit p = scan_split_forward(f.a, is_bf16);
  f.g = segments(p, work);
  f.first = p.nseg > 1 && f.h0 && f.h0 == f.hT ? reinterpret_cast<float*>(static_cast<char*>(work) + p.first) : nullptr;
  *launches = 0;
  return is_bf16 ? fwd_t<__nv_bfloat16>(f, s, launches) : fwd_t<float>(f, s, launches);
}

ScanBwdLayout scan_bwd_layout(const ScanArgs& a) {
  const ScanSplit p = scan_split_backward(a);
  ScanBwdLayout l{};
  size_t off = p.bytes;
  auto take = [&](size_t n) {
    const size_t o = off;
    off += up(n * 4);
    return o;
  };
  const size_t rows = static_cast<size_t>(a.B) * p.nseg * a.D;
  l.bc = take(static_cast<size_t>(a.B) * a.T * a.G * per_group(a, bwd_width(a.N)) * 16 * fwd_lanes(a.N));
  l.dA = take(rows * a.N);
  l.dD = take(rows);
  l.dbias = take(rows);
  l.bytes = off;
  return l;
}

int launch_scan_backward(const ScanBwdArgs& b, int is_bf16, cudaStream_t s, int* launches) {
  ScanBwdArgs p = b;
  const ScanBwdLayout l = scan_bwd_layout(p.a);
  p.g = segments(scan_split_backward(p.a), p.work);
  auto part = [&](const void* want, size_t off) { return want ? reinterpret_cast<float*>(p.work + off) : nullptr; };
  p.bc = part(p.grad.dB ? p.grad.dB : p.grad.dC, l.bc);
  p.pA = part(p.grad.dA, l.dA);
  p.pD = part(p.grad.dD, l.dD);
  p.pbias = part(p.grad.ddt_bias, l.dbias);
  *launches = 0;
  return is_bf16 ? bwd_t<__nv_bfloat16>(p, s, launches) : bwd_t<float>(p, s, launches);
}

int launch_scan_step(const ScanStepArgs& p, int is_bf16, cudaStream_t s) {
  return is_bf16 ? step_t<__nv_bfloat16>(p, s) : step_t<float>(p, s);
}

}  // namespace rnn
