// norm.cu - the block norm: RMS norm of a block's output, its gate, the scaled
// residual and the next block's RMS norm in one pass over the rows, and the
// gradients of all of it in another.
#include "common.cuh"
#include "norm.h"
#include "pair.cuh"

namespace rnn {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kBlock = 256;

// V elements as they are stored: a row in flight costs half the registers of
// its fp32 form.
template <typename T, int V> struct Raw;
template <int V> struct alignas(16) Raw<__nv_bfloat16, V> {
  uint32_t w[V / 2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    if constexpr (V == 8) {
      const uint4 q = *reinterpret_cast<const uint4*>(p);
      w[0] = q.x; w[1] = q.y; w[2] = q.z; w[3] = q.w;
    } else {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      w[0] = q.x; w[1] = q.y;
    }
  }
  __device__ __forceinline__ void fill(float v) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v, v);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  __device__ __forceinline__ float2 pair(int i) const {
    return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
};
template <int V> struct alignas(16) Raw<float, V> {
  float4 q[V / 4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) q[i] = reinterpret_cast<const float4*>(p)[i];
  }
  __device__ __forceinline__ void fill(float v) {
#pragma unroll
    for (int i = 0; i < V / 4; ++i) q[i] = make_float4(v, v, v, v);
  }
  __device__ __forceinline__ float2 pair(int i) const {
    return i & 1 ? make_float2(q[i / 2].z, q[i / 2].w) : make_float2(q[i / 2].x, q[i / 2].y);
  }
};
template <typename T, int V>
__device__ __forceinline__ void load_or(Raw<T, V>& r, const void* base, int64_t at, bool ok, float other) {
  if (ok) r.load(static_cast<const T*>(base) + at);
  else r.fill(other);
}
template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float2 (&v)[V / 2]) {
  if constexpr (sizeof(T) == 2) {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const __nv_bfloat162 h = __float22bfloat162_rn(v[i]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if constexpr (V == 8) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; i += 2)
      *reinterpret_cast<float4*>(p + 2 * i) = make_float4(v[i].x, v[i].y, v[i + 1].x, v[i + 1].y);
  }
}

// Copies a thread's V elements to its own slot in shared memory, or zeros.
template <typename T, int V>
__device__ __forceinline__ void raw_async(Raw<T, V>* slot, const void* base, int64_t at, bool ok) {
  const uint32_t dst = smem_u32(slot);
  const char* src = reinterpret_cast<const char*>(static_cast<const T*>(base) + (ok ? at : 0));
  const int n = ok ? 16 : 0;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(Raw<T, V>)); i += 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst + i), "l"(ok ? src + i : src), "r"(n) : "memory");
}

// Sums N values over the TPR consecutive threads of a row; every thread gets
// the sums.  Rows wider than a warp go through shared memory, ``red`` holding
// N values per warp; consecutive calls alternate ``red`` buffers, so one
// barrier a call is enough.
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

// With bf16 storage the sigmoid takes the hardware's approximate exponential
// and reciprocal (a few 2^-23 against the storage's 2^-9): the IEEE division
// alone would cost more instructions than the rest of the row.
template <typename T>
__device__ __forceinline__ float2 sigm2(float2 z) {
  if constexpr (sizeof(T) == 2)
    return make_float2(__fdividef(1.f, 1.f + __expf(-z.x)), __fdividef(1.f, 1.f + __expf(-z.y)));
  else
    return make_float2(sigm(z.x), sigm(z.y));
}
// act(z) from s = sigma(z) (one without a gate), and its derivative.
__device__ __forceinline__ float2 act2(int kind, float2 z, float2 s) { return kind == RNN_GATE_SILU ? mul2(z, s) : s; }
__device__ __forceinline__ float2 dact2(int kind, float2 f, float2 s) {
  const float2 t = make_float2(1.f - s.x, 1.f - s.y);         // zero without a gate
  return kind == RNN_GATE_SILU ? fma2(f, t, s) : mul2(s, t);
}
template <typename T, int V>
__device__ __forceinline__ void sigm_vec(int kind, const Raw<T, V>& z, float2 (&s)[V / 2]) {
#pragma unroll
  for (int j = 0; j < V / 2; ++j) s[j] = make_float2(1.f, 1.f);
  if (kind == RNN_GATE_NONE) return;
#pragma unroll
  for (int j = 0; j < V / 2; ++j) s[j] = sigm2<T>(z.pair(j));
}

// The rows a group of TPR threads walks: row-group ``first + n * step``, kept
// as (row, group) without divisions inside the loop.
struct Walk {
  int64_t item, total, step;
  int row, grp, drow, dgrp, groups;
  __device__ __forceinline__ Walk(const NormArgs& a, int64_t first, int64_t step_) {
    groups = a.groups;
    item = first;
    step = step_;
    total = static_cast<int64_t>(a.rows) * groups;
    row = static_cast<int>(first / groups);
    grp = static_cast<int>(first - static_cast<int64_t>(row) * groups);
    drow = static_cast<int>(step / groups);
    dgrp = static_cast<int>(step - static_cast<int64_t>(drow) * groups);
  }
  __device__ __forceinline__ bool live() const { return item < total; }
  __device__ __forceinline__ void next() {
    item += step;
    row += drow;
    grp += dgrp;
    if (grp >= groups) {
      grp -= groups;
      ++row;
    }
  }
};

// TPR threads a row, IT vectors of kVec a thread: cols <= TPR * IT * kVec.  The row
// stays in registers between the two norms, so each stream is moved once.  FULL:
// with a residual or an outgoing norm (else both are compiled out).  A thread
// keeps its columns' weights, and loads its next row before it works on this
// one (IT = 1), which keeps the memory busy through the row sums.
// bf16, all parts on, 16384 rows of 2048: 60 us, 5.6 TB/s; 262144 groups of 128
// with a gate: 37 us, 5.4 TB/s.
template <typename T, int kVec, int TPR, int IT, bool FULL>
__global__ void __launch_bounds__(TPR > kBlock ? TPR : kBlock) norm_fwd_kernel(const NormArgs a) {
  constexpr int RPB = (TPR > kBlock ? TPR : kBlock) / TPR, V2 = kVec / 2;
  __shared__ float red[4][32];
  const int l = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  Walk w(a, static_cast<int64_t>(blockIdx.x) * RPB + sub, static_cast<int64_t>(gridDim.x) * RPB);
  const float inv = 1.f / a.cols;
  const bool gate = a.gate != RNN_GATE_NONE, residual = FULL && a.residual, norm_out = FULL && a.norm_out;
  bool in[IT];
  int c[IT];
  Raw<T, kVec> wi[IT], sc[IT], wo[IT];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    c[i] = (i * TPR + l) * kVec;
    in[i] = c[i] < a.cols;
    load_or<T, kVec>(wi[i], a.w_in, c[i], in[i] && a.w_in, 1.f);
    if (FULL) load_or<T, kVec>(sc[i], a.scale, c[i], in[i] && a.scale, 1.f);
    if (FULL) load_or<T, kVec>(wo[i], a.w_out, c[i], in[i] && a.w_out, 1.f);
  }
  Raw<T, kVec> y[IT], z[IT], x[IT], yn[IT], zn[IT], xn[IT];
  auto load = [&](const Walk& at, Raw<T, kVec> (&yy)[IT], Raw<T, kVec> (&zz)[IT], Raw<T, kVec> (&xx)[IT]) {
    const bool live = at.live();
    const int64_t off = static_cast<int64_t>(at.grp) * a.cols;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const bool ok = live && in[i];
      load_or<T, kVec>(yy[i], a.y, at.row * a.y_row + off + c[i], ok, 0.f);
      load_or<T, kVec>(zz[i], a.z, at.row * a.z_row + off + c[i], ok && gate, 0.f);
      if (FULL) load_or<T, kVec>(xx[i], a.x, at.row * a.x_row + off + c[i], ok && residual, 0.f);
    }
  };
  load(w, y, z, x);
  int odd = 0;
  // every thread of the CTA takes part in every turn: the row sums have barriers
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * RPB; base < w.total; base += w.step) {
    Walk next = w;
    next.next();
    if (IT == 1) load(next, yn, zn, xn);
    const bool live = w.live();
    const int64_t dense = (static_cast<int64_t>(w.row) * a.groups + w.grp) * a.cols;
    float r1 = 1.f;
    if (a.norm_in) {
      float2 q = both(0.f);
#pragma unroll
      for (int i = 0; i < IT; ++i)
#pragma unroll
        for (int j = 0; j < V2; ++j) q = fma2(y[i].pair(j), y[i].pair(j), q);
      float s1[1] = {q.x + q.y};
      row_sum<TPR, 1>(s1, red[odd]);
      r1 = rsqrtf(s1[0] * inv + a.eps);
    }
    float2 v[IT][V2], q2 = both(0.f);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      float2 sg[V2];
      sigm_vec<T, kVec>(a.gate, z[i], sg);
#pragma unroll
      for (int j = 0; j < V2; ++j)
        v[i][j] = mul2(mul2(mul2(y[i].pair(j), both(r1)), wi[i].pair(j)), act2(a.gate, z[i].pair(j), sg[j]));
      if (residual)
#pragma unroll
        for (int j = 0; j < V2; ++j) v[i][j] = fma2(sc[i].pair(j), v[i][j], x[i].pair(j));
      if (live && in[i]) store_vec<T, kVec>(static_cast<T*>(a.x_out) + dense + c[i], v[i]);
      if (norm_out)
#pragma unroll
        for (int j = 0; j < V2; ++j) q2 = fma2(v[i][j], v[i][j], q2);     // zero beyond the row: y and x are
    }
    if (norm_out) {
      float s2[1] = {q2.x + q2.y};
      row_sum<TPR, 1>(s2, red[2 + odd]);
      const float r2 = rsqrtf(s2[0] * inv + a.eps);
#pragma unroll
      for (int i = 0; i < IT; ++i) {
#pragma unroll
        for (int j = 0; j < V2; ++j) v[i][j] = mul2(v[i][j], mul2(both(r2), wo[i].pair(j)));
        if (live && in[i]) store_vec<T, kVec>(static_cast<T*>(a.n_out) + dense + c[i], v[i]);
      }
    }
    odd ^= 1;
    w = next;
    if (IT == 1) {
      y[0] = yn[0];
      z[0] = zn[0];
      if (FULL) x[0] = xn[0];
    } else {
      load(w, y, z, x);
    }
  }
}

// r^3 m, where r^3 alone may leave the range (a row's root mean square from 1e13
// up or 1e-13 down): m is of the size of the row, so each product is in range.
__device__ __forceinline__ float cube_times(float r, float m) { return r * (r * (r * m)); }

// The gradients.  With r1, r2 the two inverse root means, h = dn * w_out:
//   dc = dx' + r2 h - x' r2^3 mean(h x')                 (dx = dc)
//   dw_out += dn x' r2,  dscale += dc b,  db = scale dc
//   dz = db a act'(z),  da = db act(z),  dw_in += da y r1
//   dy = r1 (da w_in) - y r1^3 mean(da w_in y)
// x' is recomputed from the inputs, not read back rounded, so that the weights'
// fp32 gradients carry no bf16 rounding.  A CTA walks rows with a stride and
// keeps its columns' weight gradients in registers; the CTAs' partial sums are
// added by a second kernel in a fixed order.  A row costs three dependent sums,
// so its rows to come wait in shared memory (NS deep, each thread its own slots,
// no barrier), not in registers: three CTAs an SM hide the sums.  bf16, all parts
// on, 16384 rows of 2048: 124 us, 4.3 TB/s, 60 % of the issue slots (rows ahead in
// registers, two CTAs: 142 us; half the columns a thread: 187 us); 262144 groups
// of 128 with a gate: 56 us, 6.0 TB/s.
template <typename T, int V, int TPR, int IT, bool FULL>
struct BwdSmem {
  static constexpr int NT = TPR > kBlock ? TPR : kBlock, STREAMS = FULL ? 5 : 3, WEIGHTS = FULL ? 3 : 1;
  static constexpr int stage = STREAMS * IT * NT * static_cast<int>(sizeof(Raw<T, V>));
  // the weights too, where there is room (all but the widest fp32 rows)
  static constexpr int all_weights = WEIGHTS * IT * NT * static_cast<int>(sizeof(Raw<T, V>));
  static constexpr int weights = stage + all_weights <= (220 << 10) ? all_weights : 0;
  static constexpr int NS = stage <= (20 << 10) ? 3 : stage + weights <= (100 << 10) ? 2 : 1;
  static constexpr int bytes = NS * stage + weights;
};

template <typename T, int kVec, int TPR, int IT, bool FULL>
__global__ void __launch_bounds__(TPR > kBlock ? TPR : kBlock, IT > 1 || sizeof(T) > 2 ? 1 : FULL && TPR < 64 ? 2 : 3)
    norm_bwd_kernel(const NormArgs a) {
  using L = BwdSmem<T, kVec, TPR, IT, FULL>;
  constexpr int NT = L::NT, RPB = NT / TPR, NW = FULL ? 3 : 1, V2 = kVec / 2, NS = L::NS;
  __shared__ float red[6][64];
  extern __shared__ __align__(16) unsigned char smem_raw[];
  using Slot = Raw<T, kVec>;
  Slot* slots = reinterpret_cast<Slot*>(smem_raw);                       // [NS][stream][IT][NT]
  Slot* wts = slots + NS * L::STREAMS * IT * NT;                         // [weight][IT][NT]
  const int tid = threadIdx.x, l = tid % TPR, sub = tid / TPR;
  Walk w(a, static_cast<int64_t>(blockIdx.x) * RPB + sub, static_cast<int64_t>(gridDim.x) * RPB);
  const float inv = 1.f / a.cols;
  const bool gate = a.gate != RNN_GATE_NONE, residual = FULL && a.residual, norm_out = FULL && a.norm_out;
  bool in[IT];
  int c[IT];
  float2 gw[NW][IT][V2];
#pragma unroll
  for (int i = 0; i < IT; ++i) {
    c[i] = (i * TPR + l) * kVec;
    in[i] = c[i] < a.cols;
    if (L::weights) {
      load_or<T, kVec>(wts[i * NT + tid], a.w_in, c[i], in[i] && a.w_in, 1.f);
      if (FULL) load_or<T, kVec>(wts[(IT + i) * NT + tid], a.scale, c[i], in[i] && a.scale, 1.f);
      if (FULL) load_or<T, kVec>(wts[(2 * IT + i) * NT + tid], a.w_out, c[i], in[i] && a.w_out, 1.f);
    }
#pragma unroll
    for (int k = 0; k < NW; ++k)
#pragma unroll
      for (int j = 0; j < V2; ++j) gw[k][i][j] = both(0.f);
  }
  auto load = [&](const Walk& at, int stage) {
    const bool live = at.live();
    const int64_t off = static_cast<int64_t>(at.grp) * a.cols;
    const int64_t dense = (static_cast<int64_t>(at.row) * a.groups + at.grp) * a.cols;
    Slot* s = slots + stage * L::STREAMS * IT * NT + tid;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const bool ok = live && in[i];
      raw_async<T, kVec>(s + i * NT, a.y, at.row * a.y_row + off + c[i], ok);
      raw_async<T, kVec>(s + (IT + i) * NT, a.z, at.row * a.z_row + off + c[i], ok && gate);
      raw_async<T, kVec>(s + (2 * IT + i) * NT, a.dx_out, dense + c[i], ok && a.dx_out);
      if (FULL) raw_async<T, kVec>(s + (3 * IT + i) * NT, a.x, at.row * a.x_row + off + c[i], ok && residual && norm_out);
      if (FULL) raw_async<T, kVec>(s + (4 * IT + i) * NT, a.dn_out, dense + c[i], ok && norm_out && a.dn_out);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto weight = [&](const void* from, int k, int i) {
    Slot v;
    if (L::weights) v = wts[(k * IT + i) * NT + tid];
    else load_or<T, kVec>(v, from, c[i], in[i] && from, 1.f);
    return v;
  };
  Walk ahead = w;
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    load(ahead, k);
    ahead.next();
  }
  int odd = 0, stage = 0;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * RPB; base < w.total; base += w.step) {
    asm volatile("cp.async.wait_group %0;" :: "n"(NS - 1) : "memory");
    const Slot* s = slots + stage * L::STREAMS * IT * NT + tid;
    const bool live = w.live();
    const int64_t dense = (static_cast<int64_t>(w.row) * a.groups + w.grp) * a.cols;
    float r1 = 1.f;
    if (a.norm_in) {
      float2 q = both(0.f);
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const Slot y = s[i * NT];
#pragma unroll
        for (int j = 0; j < V2; ++j) q = fma2(y.pair(j), y.pair(j), q);
      }
      float s1[1] = {q.x + q.y};
      row_sum<TPR, 1>(s1, red[odd]);
      r1 = rsqrtf(s1[0] * inv + a.eps);
    }
    // b = a act(z) and x' (kept, with the sigmoids), and the two sums of the outgoing norm
    float2 sg[IT][V2], b[FULL ? IT : 1][V2], cx[FULL ? IT : 1][V2];
    float r2 = 0.f, m2 = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i) sigm_vec<T, kVec>(a.gate, s[(IT + i) * NT], sg[i]);
    if (FULL) {
      float2 q0 = both(0.f), q1 = both(0.f);
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const Slot y = s[i * NT], z = s[(IT + i) * NT], x = s[(3 * IT + i) * NT], n = s[(4 * IT + i) * NT];
        const Slot wi = weight(a.w_in, 0, i), sc = weight(a.scale, 1, i), wo = weight(a.w_out, 2, i);
#pragma unroll
        for (int j = 0; j < V2; ++j) {
          const float2 f = act2(a.gate, z.pair(j), sg[i][j]);
          b[FULL ? i : 0][j] = mul2(mul2(mul2(y.pair(j), both(r1)), wi.pair(j)), f);
          if (norm_out) {
            float2 cc = b[FULL ? i : 0][j];
            if (residual) cc = fma2(sc.pair(j), cc, x.pair(j));
            cx[FULL ? i : 0][j] = cc;
            q0 = fma2(cc, cc, q0);
            q1 = fma2(mul2(n.pair(j), wo.pair(j)), cc, q1);
          }
        }
      }
      if (norm_out) {
        float s2[2] = {q0.x + q0.y, q1.x + q1.y};
        row_sum<TPR, 2>(s2, red[2 + odd]);
        r2 = rsqrtf(s2[0] * inv + a.eps);
        m2 = cube_times(r2, s2[1] * inv);
      }
    }
    float2 h[IT][V2], q3 = both(0.f);
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      float2 dc[V2], dz[V2];
      const bool ok = live && in[i];
      {
        const Slot d = s[(2 * IT + i) * NT];
#pragma unroll
        for (int j = 0; j < V2; ++j) dc[j] = d.pair(j);
      }
      if (norm_out) {
        const Slot n = s[(4 * IT + i) * NT], wo = weight(a.w_out, 2, i);
#pragma unroll
        for (int j = 0; j < V2; ++j) {
          const float2 nr = mul2(n.pair(j), both(r2)), cc = cx[FULL ? i : 0][j];
          dc[j] = add2(dc[j], fma2(nr, wo.pair(j), mul2(cc, both(-m2))));
          gw[NW - 1][i][j] = fma2(nr, cc, gw[NW - 1][i][j]);
        }
      }
      if (FULL && ok && a.dx) store_vec<T, kVec>(static_cast<T*>(a.dx) + dense + c[i], dc);
      if (residual) {
        const Slot sc = weight(a.scale, 1, i);
#pragma unroll
        for (int j = 0; j < V2; ++j) {
          gw[NW / 2][i][j] = fma2(dc[j], b[FULL ? i : 0][j], gw[NW / 2][i][j]);
          dc[j] = mul2(dc[j], sc.pair(j));
        }
      }
      const Slot y = s[i * NT], z = s[(IT + i) * NT], wi = weight(a.w_in, 0, i);
#pragma unroll
      for (int j = 0; j < V2; ++j) {
        const float2 yv = y.pair(j), wv = wi.pair(j), yr = mul2(yv, both(r1));
        const float2 f = act2(a.gate, z.pair(j), sg[i][j]), df = dact2(a.gate, f, sg[i][j]);
        dz[j] = mul2(mul2(dc[j], mul2(yr, wv)), df);
        const float2 da = mul2(dc[j], f);
        gw[0][i][j] = fma2(da, yr, gw[0][i][j]);
        h[i][j] = mul2(da, wv);                        // gradient of the normalised y
        q3 = fma2(h[i][j], yv, q3);
      }
      if (ok && a.dz) store_vec<T, kVec>(static_cast<T*>(a.dz) + dense + c[i], dz);
    }
    float m1 = 0.f;
    if (a.norm_in) {
      float s3[1] = {q3.x + q3.y};
      row_sum<TPR, 1>(s3, red[4 + odd]);
      m1 = cube_times(r1, s3[0] * inv);
    }
    if (a.dy) {
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const Slot y = s[i * NT];
#pragma unroll
        for (int j = 0; j < V2; ++j) h[i][j] = fma2(h[i][j], both(r1), mul2(y.pair(j), both(-m1)));
        if (live && in[i]) store_vec<T, kVec>(static_cast<T*>(a.dy) + dense + c[i], h[i]);
      }
    }
    odd ^= 1;
    w.next();
    load(ahead, stage);                               // this row's slots are free: only this thread read them
    ahead.next();
    stage = stage + 1 == NS ? 0 : stage + 1;
  }
  if (!a.partial) return;
#pragma unroll
  for (int k = 0; k < NW; ++k) {
    float* out = a.partial + (static_cast<int64_t>(k) * gridDim.x + blockIdx.x) * a.cols;
    if constexpr (RPB == 1) {
#pragma unroll
      for (int i = 0; i < IT; ++i)
        if (in[i]) store_vec<float, kVec>(out + c[i], gw[k][i]);
    } else {
      float* fold = reinterpret_cast<float*>(smem_raw);                  // [RPB][cols]: at most 8 KB
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      __syncthreads();
#pragma unroll
      for (int i = 0; i < IT; ++i)
        if (in[i]) store_vec<float, kVec>(fold + sub * a.cols + c[i], gw[k][i]);
      __syncthreads();
      for (int x = threadIdx.x; x < a.cols; x += NT) {
        float s = 0.f;
        for (int r = 0; r < RPB; ++r) s += fold[r * a.cols + x];
        out[x] = s;
      }
    }
  }
}

// dw[w][c] = sum over CTAs of partial[w][cta][c], each of 32 groups of CTAs in
// order and then the groups in order: 32 columns a block.
__global__ void __launch_bounds__(1024) norm_reduce_kernel(const float* partial, int ctas, int cols, float* d0,
                                                           float* d1, float* d2) {
  __shared__ float sm[32][33];
  const int w = blockIdx.y;
  float* out = w == 0 ? d0 : w == 1 ? d1 : d2;
  if (!out) return;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
  float s = 0.f;
  if (c < cols) {
    const float* p = partial + static_cast<int64_t>(w) * ctas * cols + c;
#pragma unroll 8
    for (int i = g; i < ctas; i += 32) s += p[static_cast<int64_t>(i) * cols];
  }
  sm[g][threadIdx.x & 31] = s;
  __syncthreads();
  // column g of the block: its 32 partial sums lie across the warp
  s = sm[threadIdx.x & 31][g];
#pragma unroll
  for (int k = 1; k < 32; k <<= 1) s += __shfl_xor_sync(kFull, s, k);
  if ((threadIdx.x & 31) == 0 && blockIdx.x * 32 + g < cols) out[blockIdx.x * 32 + g] = s;
}

int check_launch() { return cudaGetLastError() == cudaSuccess ? 0 : RNN_CUDA_ERROR; }

// Threads a row and vectors a thread: one vector up to ``most`` threads, then
// two, then twice the threads (cols <= 8192).
struct Shape {
  int vec, tpr, it;
};
Shape shape_of(int cols, int vec, int most) {
  const int v = cols / vec;
  int t = 8;
  while (t < v && t < most) t *= 2;
  if (v <= t) return {vec, t, 1};
  return v <= 2 * most ? Shape{vec, most, 2} : Shape{vec, 2 * most, 2};
}
bool full(const NormArgs& a) { return a.residual || a.norm_out; }
Shape fwd_shape(const NormArgs& a) { return shape_of(a.cols, 8, 256); }
Shape bwd_shape(const NormArgs& a) { return shape_of(a.cols, 8, 256); }
int block_of(Shape s) { return s.tpr > kBlock ? s.tpr : kBlock; }
// CTAs of a walk: about ``threads`` resident on each SM, each with rows to keep
// its loads running ahead (and, backward, to amortise its partial sums).
int walk_ctas(const NormArgs& a, Shape s, int threads) {
  const int rpb = block_of(s) / s.tpr;
  const int64_t need = (static_cast<int64_t>(a.rows) * a.groups + rpb - 1) / rpb;
  const int per_sm = threads / block_of(s);
  const int64_t most = static_cast<int64_t>(a.num_sms) * (per_sm > 1 ? per_sm : 1);
  return static_cast<int>(need < most ? need : most);
}
int fwd_ctas(const NormArgs& a) { return walk_ctas(a, fwd_shape(a), full(a) ? 768 : 1024); }
int bwd_ctas(const NormArgs& a) { return walk_ctas(a, bwd_shape(a), 768); }

template <typename T, int V, int TPR, int IT, bool FULL>
int fwd(const NormArgs& a, cudaStream_t s) {
  constexpr int NT = TPR > kBlock ? TPR : kBlock;
  norm_fwd_kernel<T, V, TPR, IT, FULL><<<fwd_ctas(a), NT, 0, s>>>(a);
  return check_launch();
}
template <typename T, int V, int TPR, int IT, bool FULL>
int bwd(const NormArgs& a, cudaStream_t s) {
  constexpr int NT = TPR > kBlock ? TPR : kBlock, RPB = NT / TPR;
  constexpr int smem = BwdSmem<T, V, TPR, IT, FULL>::bytes;
  static_assert(smem <= 227 * 1024 && (RPB == 1 || smem >= kBlock * V * 4), "the rows and the folded sums fit");
  if (cudaFuncSetAttribute(norm_bwd_kernel<T, V, TPR, IT, FULL>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
      cudaSuccess)
    return RNN_CUDA_ERROR;
  norm_bwd_kernel<T, V, TPR, IT, FULL><<<bwd_ctas(a), NT, smem, s>>>(a);
  return check_launch();
}

// Vectors of 8, up to 256 threads a row.
#define RNN_NORM_SHAPES8(CALL, T, FULL)                                             \
  switch (sh.tpr) {                                                                 \
    case 8: return CALL<T, 8, 8, 1, FULL>(a, s);                                    \
    case 16: return CALL<T, 8, 16, 1, FULL>(a, s);                                  \
    case 32: return CALL<T, 8, 32, 1, FULL>(a, s);                                  \
    case 64: return CALL<T, 8, 64, 1, FULL>(a, s);                                  \
    case 128: return CALL<T, 8, 128, 1, FULL>(a, s);                                \
    case 256: return sh.it == 1 ? CALL<T, 8, 256, 1, FULL>(a, s) : CALL<T, 8, 256, 2, FULL>(a, s); \
    default: return CALL<T, 8, 512, 2, FULL>(a, s);                                 \
  }
template <typename T>
int fwd_t(const NormArgs& a, cudaStream_t s) {
  const Shape sh = fwd_shape(a);
  if (full(a)) RNN_NORM_SHAPES8(fwd, T, true)
  RNN_NORM_SHAPES8(fwd, T, false)
}
template <typename T>
int bwd_t(const NormArgs& a, cudaStream_t s) {
  const Shape sh = bwd_shape(a);
  if (full(a)) RNN_NORM_SHAPES8(bwd, T, true)
  RNN_NORM_SHAPES8(bwd, T, false)
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
  const dim3 grid((a.cols + 31) / 32, full(a) ? 3 : 1);
  norm_reduce_kernel<<<grid, 1024, 0, s>>>(a.partial, bwd_ctas(a), a.cols, a.dw_in, a.dscale, a.dw_out);
  rc = check_launch();
  if (!rc) *launches = 2;
  return rc;
}

}  // namespace rnn
