// delta_simt.cu - the gated delta rule in fp32 arithmetic, for every storage
// type and width: the token-by-token recurrence (which is also the serving
// step), its reverse, and the chunk kernel that turns both states into the
// gradients.
#include "common.cuh"
#include "delta.h"
#include "pair.cuh"

namespace rnn {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kWarps = 4;      // warps of a recurrence CTA

// Sums N values (N a power of two, at most 32) over the warp, each step
// exchanging half of what is left, so N values cost about N + log2(32 / N)
// shuffles instead of 5 N.  The sum of value i ends in every lane whose top
// log2 N bits, read from bit 4 down, spell i.
template <int N>
__device__ __forceinline__ float warp_sum_many(float (&v)[N], int lane) {
  int w = 16;
#pragma unroll
  for (int n = N; n > 1; n >>= 1, w >>= 1) {
    const bool up = lane & w;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float keep = up ? v[i + n / 2] : v[i];
      const float give = up ? v[i] : v[i + n / 2];
      v[i] = keep + __shfl_xor_sync(kFull, give, w);
    }
  }
  float x = v[0];
#pragma unroll
  for (; w; w >>= 1) x += __shfl_xor_sync(kFull, x, w);
  return x;
}
// The lane that holds value i of warp_sum_many<N>.
template <int N>
__device__ __forceinline__ constexpr int sum_lane(int i) {
  return i * (32 / N);
}

// VPL consecutive elements as fp32 (zero beyond the row).
template <typename T, int VPL>
__device__ __forceinline__ void load_vec(const T* p, bool in, float (&v)[VPL]) {
  if (!in) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = 0.f;
    return;
  }
  if constexpr (VPL % 4 == 0) {
#pragma unroll
    for (int i = 0; i < VPL; i += 4) {
      float t[4];
      Vec4<T>::load(p + i, t);
      v[i] = t[0]; v[i + 1] = t[1]; v[i + 2] = t[2]; v[i + 3] = t[3];
    }
  } else if constexpr (VPL == 2 && sizeof(T) == 4) {
    const float2 t = *reinterpret_cast<const float2*>(p);
    v[0] = t.x; v[1] = t.y;
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = to_f<T>(p[i]);
  }
}

template <int VPL>
__device__ __forceinline__ void store_state(float* p, const float (&v)[VPL]) {
  if constexpr (VPL % 4 == 0) {
#pragma unroll
    for (int i = 0; i < VPL; i += 4) Vec4<float>::store(p + i, {v[i], v[i + 1], v[i + 2], v[i + 3]});
  } else if constexpr (VPL == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
  } else {
    p[0] = v[0];
  }
}

__device__ __forceinline__ void copy16(void* dst, const void* src, bool ok) {
  const int n = ok ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(smem_u32(dst)), "l"(src), "r"(n) : "memory");
}

// Tokens on their way to a recurrence CTA: kAhead of them a stage, two stages
// (at most 37 KB).  A token's chain of dependent arithmetic is shorter than one
// trip to memory, so what it reads has to be asked for many tokens earlier.
template <typename T, int VPL, int R>
struct TokenStage {
  static constexpr int kAhead = sizeof(T) * VPL > 16 ? 8 : 16;
  T k[kAhead][32 * VPL], q[kAhead][32 * VPL], x[kAhead][kWarps * R];   // x: v, or do
  float al[kAhead], bl[kAhead], beta[kAhead];                          // e^g in two parts (bl: fp32)
};
// The state of an fp32 sequence is S + L, its decay al + bl: S is rounded once a
// token, and over a memory of a thousand tokens those roundings would add up to
// thirty times one, so L keeps what S lost and bl what al lost.  Outputs and sums
// take S alone, within half a last place.  Gradients against 64 bits, 513 tokens of
// slow decay: up to 2.2e-6 without, 3.6e-7 with.  bf16 storage does without: its
// outputs' own rounding is 2^-9.
//
// e^g - al, where al - 1 is exact; below one half a state is forgotten before its
// roundings add up.
__device__ __forceinline__ float decay_rest(float g, float al) {
  return al >= 0.5f && al <= 2.f ? expm1f(g) - (al - 1.f) : 0.f;
}
// al L + bl S of a row, while the token's u is not yet known.
template <int V>
__device__ __forceinline__ void carry_early(const float (&S)[V], float (&L)[V], float al, float bl) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const float2 l = fma2(both(al), make_float2(L[j], L[j + 1]), mul2(both(bl), make_float2(S[j], S[j + 1])));
      L[j] = l.x;
      L[j + 1] = l.y;
    }
  } else {
    L[0] = fmaf(al, L[0], bl * S[0]);
  }
}
// S + L <- al S + (L + u k).
template <int V>
__device__ __forceinline__ void carry_step(float (&S)[V], float (&L)[V], float al, float u, const float (&k)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const float2 s = make_float2(S[j], S[j + 1]);
      const float2 t = fma2(both(u), make_float2(k[j], k[j + 1]), make_float2(L[j], L[j + 1])), h = fma2(both(al), s, t);
      const float2 l = add2(fma2(both(al), s, make_float2(-h.x, -h.y)), t);
      S[j] = h.x;
      S[j + 1] = h.y;
      L[j] = l.x;
      L[j + 1] = l.y;
    }
  } else {
    const float t = fmaf(u, k[0], L[0]), h = fmaf(al, S[0], t);
    L[0] = fmaf(al, S[0], -h) + t;
    S[0] = h;
  }
}
// A lane's part of a . b, and y = x + f a (two elements an instruction: worth it
// where instructions count, with eight rows a warp; with two rows the recurrence of
// 1024 rows of 64 took 164 us so and 158 without).
template <int V>
__device__ __forceinline__ float dot_part(const float (&a)[V], const float (&b)[V]) {
  if constexpr (V % 2 == 0) {
    float2 s = mul2(make_float2(a[0], a[1]), make_float2(b[0], b[1]));
#pragma unroll
    for (int j = 2; j < V; j += 2) s = fma2(make_float2(a[j], a[j + 1]), make_float2(b[j], b[j + 1]), s);
    return s.x + s.y;
  } else {
    return a[0] * b[0];
  }
}
template <int V>
__device__ __forceinline__ void add_times(float (&y)[V], const float (&x)[V], float f, const float (&a)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 2) {
      const float2 s = fma2(both(f), make_float2(a[j], a[j + 1]), make_float2(x[j], x[j + 1]));
      y[j] = s.x;
      y[j + 1] = s.y;
    }
  } else {
    y[0] = fmaf(f, a[0], x[0]);
  }
}
struct TokenSource {
  const void *k, *q, *x;       // of this CTA's heads and value columns, token 0
  const void *g, *beta;
  int64_t k_step, q_step, x_step, g_step, beta_step;   // elements from token to token
  int dk, cols;                // valid columns of k / q and of x
};
// Asks for tokens t0, t0 + dir, ... (those in [0, len)) into st; the scalars of
// this thread's token come back in gb.
template <typename T, int VPL, int R>
__device__ __forceinline__ float2 stage_fetch(TokenStage<T, VPL, R>& st, const TokenSource& s, int t0, int dir, int len) {
  constexpr int E = 16 / sizeof(T), kAhead = TokenStage<T, VPL, R>::kAhead;
  const int per = s.dk / E;
  for (int i = threadIdx.x; i < kAhead * per; i += kWarps * 32) {
    const int n = i / per, c = (i - n * per) * E, t = t0 + dir * n;
    const bool ok = t >= 0 && t < len;
    copy16(&st.k[n][c], static_cast<const T*>(s.k) + (ok ? t * s.k_step + c : 0), ok);
    copy16(&st.q[n][c], static_cast<const T*>(s.q) + (ok ? t * s.q_step + c : 0), ok);
  }
  constexpr int XP = kWarps * R / E;
  for (int i = threadIdx.x; i < kAhead * XP; i += kWarps * 32) {
    const int n = i / XP, c = (i % XP) * E, t = t0 + dir * n;
    const bool ok = t >= 0 && t < len && c < s.cols;
    copy16(&st.x[n][c], static_cast<const T*>(s.x) + (ok ? t * s.x_step + c : 0), ok);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  float2 gb = make_float2(0.f, 0.f);
  const int t = t0 + dir * static_cast<int>(threadIdx.x);
  if (threadIdx.x < kAhead && t >= 0 && t < len) {
    gb.x = to_f<T>(static_cast<const T*>(s.g)[t * s.g_step]);
    gb.y = to_f<T>(static_cast<const T*>(s.beta)[t * s.beta_step]);
  }
  return gb;
}
// Lets the tokens asked for last be read by the CTA.
template <typename T, int VPL, int R>
__device__ __forceinline__ void stage_ready(TokenStage<T, VPL, R>& st, float2 gb) {
  if (threadIdx.x < TokenStage<T, VPL, R>::kAhead) {
    st.al[threadIdx.x] = expf(gb.x);
    if (sizeof(T) == 4) st.bl[threadIdx.x] = decay_rest(gb.x, st.al[threadIdx.x]);
    st.beta[threadIdx.x] = gb.y;
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
}

// The recurrence.  A warp owns R rows of one head's state (row = one value
// column, all of Dk across the lanes, VPL elements each); rows are independent,
// so there is nothing to exchange but the two dot products S k and S q inside
// the warp.  Both are taken of the old state: S_t q = a (S q) + u (k . q).
// One token costs the chain exp -> dot -> shuffles -> update.  AHEAD: tokens come
// through shared memory a stage early (sequences); otherwise each is loaded one
// token early (the serving step, where the state is what takes time).  CARRY: with
// the parts lost to rounding.  Bound by that chain: 0.31 us a token at 1024 rows of
// 64 in fp32 (0.29 without CARRY; 0.56 when each token was loaded one token early);
// the reverse 0.29.
template <typename T, int VPL, int R, bool AHEAD, bool CARRY>
__global__ void __launch_bounds__(kWarps * 32) delta_recur_kernel(const DeltaRecurArgs r) {
  static_assert(AHEAD || !CARRY, "a few tokens' roundings do not add up");
  constexpr int kAhead = TokenStage<T, VPL, R>::kAhead;
  __shared__ __align__(16) TokenStage<T, VPL, R> st[AHEAD ? 2 : 1];
  const DeltaArgs& a = r.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = (a.Dv + kWarps * R - 1) / (kWarps * R);
  const int bid = blockIdx.x;
  const int grp = bid % groups, h = bid / groups % a.Hv, b = bid / groups / a.Hv;
  const int dv0 = (grp * kWarps + warp) * R;
  const int hk = h / (a.Hv / a.Hk);
  const int dk0 = lane * VPL;
  const bool mine = dv0 < a.Dv, in = mine && dk0 < a.Dk;
  int len = a.len ? a.len[b] : a.T;
  int64_t slot = b;
  bool live = true;
  if (r.slots) {
    slot = r.slots[b];
    live = slot >= 0 && slot < r.num_slots;
  } else if (r.num_slots >= 0 && b >= r.num_slots) {
    live = false;
  }
  if (!live) len = 0;
  const int64_t head_elems = static_cast<int64_t>(a.Dv) * a.Dk;
  const int64_t s_off = (slot * a.Hv + h) * head_elems;
  const int64_t ts = a.bfirst ? 1 : a.B, row0 = a.row(b, 0);      // rows from token to token

  const int64_t o_row = static_cast<int64_t>(a.Hv) * a.Dv;
  T* o = static_cast<T*>(r.o) + row0 * o_row + static_cast<int64_t>(h) * a.Dv + dv0;
  TokenSource src;
  src.k = static_cast<const T*>(a.k) + row0 * a.k_row + static_cast<int64_t>(hk) * a.Dk;
  src.q = static_cast<const T*>(a.q) + row0 * a.q_row + static_cast<int64_t>(hk) * a.Dk;
  src.x = static_cast<const T*>(a.v) + row0 * a.v_row + static_cast<int64_t>(h) * a.Dv + grp * kWarps * R;
  src.g = static_cast<const T*>(a.g) + row0 * a.g_row + h;
  src.beta = static_cast<const T*>(a.beta) + row0 * a.beta_row + h;
  src.k_step = ts * a.k_row; src.q_step = ts * a.q_row; src.x_step = ts * a.v_row;
  src.g_step = ts * a.g_row; src.beta_step = ts * a.beta_row;
  src.dk = a.Dk;
  src.cols = a.Dv - grp * kWarps * R;
  const bool vin = lane < R && dv0 + lane < a.Dv;   // this lane loads / stores value row dv0 + lane

  float2 gb = make_float2(0.f, 0.f);
  if (AHEAD && len > 0) gb = stage_fetch<T, VPL, R>(st[0], src, 0, 1, len);
  float S[R][VPL];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const bool ok = in && live && r.s_in != nullptr && dv0 + i < a.Dv;
    load_vec<float, VPL>(r.s_in + s_off + static_cast<int64_t>(dv0 + i) * a.Dk + dk0, ok, S[i]);
  }
  float L[CARRY ? R : 1][VPL];
#pragma unroll
  for (int i = 0; i < (CARRY ? R : 1); ++i)
#pragma unroll
    for (int j = 0; j < VPL; ++j) L[i][j] = 0.f;
  float kc[VPL], qc[VPL], vc = 0.f, al = 0.f, bl = 0.f, bc = 0.f;
  float kn[VPL], qn[VPL], vn = 0.f, gn = 0.f, bn = 0.f;
  auto direct = [&](int t) {
    load_vec<T, VPL>(static_cast<const T*>(src.k) + t * src.k_step + dk0, in, kn);
    load_vec<T, VPL>(static_cast<const T*>(src.q) + t * src.q_step + dk0, in, qn);
    vn = vin ? to_f<T>(static_cast<const T*>(src.x)[t * src.x_step + warp * R + lane]) : 0.f;
    gn = to_f<T>(static_cast<const T*>(src.g)[t * src.g_step]);
    bn = to_f<T>(static_cast<const T*>(src.beta)[t * src.beta_step]);
  };
  if (!AHEAD && len > 0) direct(0);
  const int64_t bh = static_cast<int64_t>(b) * a.Hv + h;
  const int nc = (a.T + kSimtChunk - 1) / kSimtChunk;
  T* ot = o + lane;                         // this token's output and e
  float* et = r.e + (bh * a.T * a.Dv + dv0 + lane);
  for (int t = 0; t < len; ++t) {
    if (AHEAD) {
      const int n = t % kAhead;
      if (n == 0) {
        stage_ready<T, VPL, R>(st[(t / kAhead) & 1], gb);      // and the other stage is free
        if (t + kAhead < len) gb = stage_fetch<T, VPL, R>(st[(t / kAhead + 1) & 1], src, t + kAhead, 1, len);
      }
      const TokenStage<T, VPL, R>& s = st[(t / kAhead) & 1];
      load_vec<T, VPL>(&s.k[n][dk0], in, kc);
      load_vec<T, VPL>(&s.q[n][dk0], in, qc);
      vc = vin ? to_f<T>(s.x[n][warp * R + lane]) : 0.f;
      al = s.al[n];
      if (CARRY) bl = s.bl[n];
      bc = s.beta[n];
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j) { kc[j] = kn[j]; qc[j] = qn[j]; }
      vc = vn; bc = bn;
      al = expf(gn);
      if (t + 1 < len) direct(t + 1);
    }
    if (r.ckpt && t % kSimtChunk == 0 && in) {
      float* c = r.ckpt + (bh * nc + t / kSimtChunk) * head_elems + dk0;
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (dv0 + i < a.Dv) store_state<VPL>(c + static_cast<int64_t>(dv0 + i) * a.Dk, S[i]);
    }
    float d[2 * R], kq = 0.f;
    if constexpr (R == 8 && CARRY) {
      kq = dot_part<VPL>(kc, qc);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        d[i] = dot_part<VPL>(S[i], kc);
        d[R + i] = dot_part<VPL>(S[i], qc);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2 * R; ++i) d[i] = 0.f;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        kq = fmaf(kc[j], qc[j], kq);
#pragma unroll
        for (int i = 0; i < R; ++i) {
          d[i] = fmaf(S[i][j], kc[j], d[i]);
          d[R + i] = fmaf(S[i][j], qc[j], d[R + i]);
        }
      }
    }
    if constexpr (CARRY) {
#pragma unroll
      for (int i = 0; i < R; ++i) carry_early<VPL>(S[i], L[i], al, bl);
    }
    const float sum = warp_sum_many<2 * R>(d, lane);
#pragma unroll
    for (int w = 16; w; w >>= 1) kq += __shfl_xor_sync(kFull, kq, w);
    // lane i < R finishes value row dv0 + i
    const int src_lane = lane < R ? lane : 0;
    const float sk = __shfl_sync(kFull, sum, sum_lane<2 * R>(1) * src_lane);
    const float sq = __shfl_sync(kFull, sum, sum_lane<2 * R>(1) * (R + src_lane));
    const float e = vc - al * sk;
    const float u = bc * e;
    if (vin) {
      *ot = from_f<T>(a.scale * fmaf(al, sq, u * kq));
      if (r.e) *et = e;
    }
    ot += ts * o_row;
    et += a.Dv;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float ui = __shfl_sync(kFull, u, i);
      if constexpr (CARRY) {
        carry_step<VPL>(S[i], L[i], al, ui, kc);
      } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j) S[i][j] = fmaf(al, S[i][j], ui * kc[j]);      // one rounding of the state's size
      }
    }
  }
  for (int t = len; t < a.T; ++t)
    if (vin) o[t * ts * o_row + lane] = from_f<T>(0.f);
  // a skipped sequence has no slot to write; one without tokens keeps its state
  if (r.s_out && live && in && !(len == 0 && r.s_out == r.s_in)) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (dv0 + i < a.Dv) store_state<VPL>(r.s_out + s_off + static_cast<int64_t>(dv0 + i) * a.Dk + dk0, S[i]);
  }
}

// The serving step over many states: all it does is move them, 8 Dk Dv bytes a
// head against 6 Dk Dv operations, so what counts is bytes on their way.  A CTA
// walks units of 32 state rows with a stride; a unit (contiguous, 128 Dk bytes) is
// fetched by one bulk copy kUnits units early, its token inputs one unit early.
// Warp w computes rows 8 w .. 8 w + 7 and writes them back from registers.
// 256 sequences of 32 heads of 128 x 128 (1.08 GB): 173 us, 6.2 TB/s; loads into
// registers without the pipeline took 203 (8 rows a warp) to 213 us (4).
constexpr int kUnitRows = 32;
constexpr uint64_t kStepTimeoutNs = 2000000000ull;     // of a wait for a unit's copy

template <int VPL>
struct StepSmem {
  float S[kUnits][kUnitRows * 32 * VPL];
  uint64_t full[kUnits];
};

template <typename T, int VPL>
__global__ void __launch_bounds__(kWarps * 32) delta_step_kernel(const DeltaRecurArgs r) {
  constexpr int R = kUnitRows / kWarps;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  StepSmem<VPL>& sm = *reinterpret_cast<StepSmem<VPL>*>(smem_raw);
  const DeltaArgs& a = r.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = (a.Dv + kUnitRows - 1) / kUnitRows, per = a.Hv / a.Hk;
  const int units = groups * a.Hv * a.B, stride = gridDim.x;
  const int dk0 = lane * VPL;
  const bool in = dk0 < a.Dk;
  const int64_t ts = a.bfirst ? 1 : a.B, o_row = static_cast<int64_t>(a.Hv) * a.Dv;

  struct Unit {
    int b, h, dv0, rows, len;
    float* S;
  };
  auto at = [&](int u) {
    Unit x;
    const int bh = u / groups;
    x.dv0 = (u - bh * groups) * kUnitRows;
    x.b = bh / a.Hv;
    x.h = bh - x.b * a.Hv;
    x.rows = min(kUnitRows, a.Dv - x.dv0);
    const int64_t slot = r.slots ? r.slots[x.b] : x.b;
    const bool live = slot >= 0 && slot < r.num_slots;
    x.len = live ? (a.len ? a.len[x.b] : a.T) : 0;
    x.S = r.s_out + ((slot * a.Hv + x.h) * a.Dv + x.dv0) * a.Dk;
    return x;
  };
  // by thread 0, once nobody reads the stage; a unit without tokens only turns the barrier's phase
  auto fetch = [&](int u, int stage) {
    const Unit x = at(u);
    const uint32_t bytes = x.len ? x.rows * a.Dk * 4 : 0;
    mbar_arrive_expect_tx(&sm.full[stage], bytes);
    if (bytes) {
      fence_proxy_async_smem();
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                   :: "r"(smem_u32(sm.S[stage])), "l"(x.S), "r"(bytes), "r"(smem_u32(&sm.full[stage])) : "memory");
    }
  };
  float kn[VPL], qn[VPL], vn = 0.f, gn = 0.f, bn = 0.f;
  const int vrow = warp * R + lane;           // of the unit, lanes below R
  auto token = [&](const Unit& x, int t) {
    const int64_t row = a.row(x.b, t);
    const int hk = x.h / per;
    load_vec<T, VPL>(static_cast<const T*>(a.k) + row * a.k_row + hk * a.Dk + dk0, in, kn);
    load_vec<T, VPL>(static_cast<const T*>(a.q) + row * a.q_row + hk * a.Dk + dk0, in, qn);
    vn = lane < R && vrow < x.rows ? to_f<T>(static_cast<const T*>(a.v)[row * a.v_row + static_cast<int64_t>(x.h) * a.Dv + x.dv0 + vrow]) : 0.f;
    gn = to_f<T>(static_cast<const T*>(a.g)[row * a.g_row + x.h]);
    bn = to_f<T>(static_cast<const T*>(a.beta)[row * a.beta_row + x.h]);
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < kUnits; ++i) mbar_init(&sm.full[i], 1);
    fence_mbar_init();
    for (int i = 0; i < kUnits; ++i)
      if (static_cast<int64_t>(blockIdx.x) + i * stride < units) fetch(blockIdx.x + i * stride, i);
  }
  __syncthreads();
  Unit cur{}, nxt = at(min(static_cast<int>(blockIdx.x), units - 1));
  if (nxt.len) token(nxt, 0);
  int turn = 0;
  for (int64_t u = blockIdx.x; u < units; u += stride, ++turn) {
    cur = nxt;
    const int stage = step_fill(turn).stage;
    const bool late = !mbar_wait(&sm.full[stage], step_fill(turn).parity, kStepTimeoutNs);
    float S[R][VPL];
#pragma unroll
    for (int i = 0; i < R; ++i)
      load_vec<float, VPL>(&sm.S[stage][(warp * R + i) * a.Dk + dk0], in && cur.len && warp * R + i < cur.rows, S[i]);
    if (__syncthreads_or(late)) {
      // copies that are still under way keep the CTA for as long again, each
      if (threadIdx.x == 0) {
        atomicCAS(r.status, 0u, static_cast<unsigned int>(RNN_TIMEOUT));
        const int turns = (units - 1 - static_cast<int>(blockIdx.x)) / stride + 1;
        for (int t = turn; t <= step_last_fill(turn, turns); ++t)
          mbar_wait(&sm.full[step_fill(t).stage], step_fill(t).parity, kStepTimeoutNs);
      }
      return;
    }
    if (threadIdx.x == 0 && u + static_cast<int64_t>(kUnits) * stride < units) fetch(static_cast<int>(u) + kUnits * stride, stage);
    float kc[VPL], qc[VPL], vc, gc, bc;
    auto take = [&]() {
#pragma unroll
      for (int j = 0; j < VPL; ++j) { kc[j] = kn[j]; qc[j] = qn[j]; }
      vc = vn; gc = gn; bc = bn;
    };
    auto next_unit = [&]() {
      if (u + stride < units) {
        nxt = at(static_cast<int>(u) + stride);
        if (nxt.len) token(nxt, 0);
      }
    };
    T* o = static_cast<T*>(r.o) + a.row(cur.b, 0) * o_row + static_cast<int64_t>(cur.h) * a.Dv + cur.dv0 + vrow;
    const bool vin = lane < R && vrow < cur.rows;
    for (int t = 0; t < cur.len; ++t) {
      take();
      if (t + 1 < cur.len) token(cur, t + 1);
      else next_unit();
      const float al = expf(gc);
      float d[2 * R], kq = 0.f;
#pragma unroll
      for (int i = 0; i < 2 * R; ++i) d[i] = 0.f;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        kq = fmaf(kc[j], qc[j], kq);
#pragma unroll
        for (int i = 0; i < R; ++i) {
          d[i] = fmaf(S[i][j], kc[j], d[i]);
          d[R + i] = fmaf(S[i][j], qc[j], d[R + i]);
        }
      }
      const float sum = warp_sum_many<2 * R>(d, lane);
#pragma unroll
      for (int w = 16; w; w >>= 1) kq += __shfl_xor_sync(kFull, kq, w);
      const int src_lane = lane < R ? lane : 0;
      const float sk = __shfl_sync(kFull, sum, sum_lane<2 * R>(1) * src_lane);
      const float sq = __shfl_sync(kFull, sum, sum_lane<2 * R>(1) * (R + src_lane));
      const float uu = bc * (vc - al * sk);
      if (vin) o[t * ts * o_row] = from_f<T>(a.scale * fmaf(al, sq, uu * kq));
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float ui = __shfl_sync(kFull, uu, i);
#pragma unroll
        for (int j = 0; j < VPL; ++j) S[i][j] = fmaf(al, S[i][j], ui * kc[j]);      // one rounding of the state's size
      }
    }
    for (int t = cur.len; t < a.T; ++t)
      if (vin) o[t * ts * o_row] = from_f<T>(0.f);
    if (!cur.len) next_unit();
    if (in && cur.len) {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (warp * R + i < cur.rows) store_state<VPL>(cur.S + static_cast<int64_t>(warp * R + i) * a.Dk + dk0, S[i]);
    }
  }
}

// The reverse recurrence of the state gradient, same ownership:
//   dS += scale do_t q_t^T;  y_t = dS k_t;  dS -= beta_t y_t k_t^T;  dS *= a_t.
template <typename T, int VPL, int R>
__global__ void __launch_bounds__(kWarps * 32) delta_recur_bwd_kernel(const DeltaRecurBwdArgs r) {
  constexpr int kAhead = TokenStage<T, VPL, R>::kAhead;
  __shared__ __align__(16) TokenStage<T, VPL, R> st[2];
  const DeltaArgs& a = r.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int groups = (a.Dv + kWarps * R - 1) / (kWarps * R);
  const int bid = blockIdx.x;
  const int grp = bid % groups, h = bid / groups % a.Hv, b = bid / groups / a.Hv;
  const int dv0 = (grp * kWarps + warp) * R;
  const int hk = h / (a.Hv / a.Hk);
  const int dk0 = lane * VPL;
  const bool in = dv0 < a.Dv && dk0 < a.Dk;
  const int len = a.len ? a.len[b] : a.T;
  const int64_t bh = static_cast<int64_t>(b) * a.Hv + h;
  const int64_t head_elems = static_cast<int64_t>(a.Dv) * a.Dk;
  const int64_t ts = a.bfirst ? 1 : a.B, row0 = a.row(b, 0), o_row = static_cast<int64_t>(a.Hv) * a.Dv;
  TokenSource src;
  src.k = static_cast<const T*>(a.k) + row0 * a.k_row + static_cast<int64_t>(hk) * a.Dk;
  src.q = static_cast<const T*>(a.q) + row0 * a.q_row + static_cast<int64_t>(hk) * a.Dk;
  src.x = static_cast<const T*>(r.dout) + row0 * o_row + static_cast<int64_t>(h) * a.Dv + grp * kWarps * R;
  src.g = static_cast<const T*>(a.g) + row0 * a.g_row + h;
  src.beta = static_cast<const T*>(a.beta) + row0 * a.beta_row + h;
  src.k_step = ts * a.k_row; src.q_step = ts * a.q_row; src.x_step = ts * o_row;
  src.g_step = ts * a.g_row; src.beta_step = ts * a.beta_row;
  src.dk = a.Dk;
  src.cols = a.Dv - grp * kWarps * R;
  const bool vin = lane < R && dv0 + lane < a.Dv;
  const int nc = (a.T + kSimtChunk - 1) / kSimtChunk;

  float2 gb = make_float2(0.f, 0.f);
  if (len > 0) gb = stage_fetch<T, VPL, R>(st[0], src, len - 1, -1, len);
  float dS[R][VPL];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const bool ok = in && r.dsT != nullptr && dv0 + i < a.Dv;
    load_vec<float, VPL>(r.dsT + bh * head_elems + static_cast<int64_t>(dv0 + i) * a.Dk + dk0, ok, dS[i]);
  }
  constexpr bool CARRY = sizeof(T) == 4;
  float L[CARRY ? R : 1][VPL];
#pragma unroll
  for (int i = 0; i < (CARRY ? R : 1); ++i)
#pragma unroll
    for (int j = 0; j < VPL; ++j) L[i][j] = 0.f;
  float* yt = r.y + ((bh * a.T + len - 1) * a.Dv + dv0 + lane);
  for (int it = 0; it < len; ++it) {
    const int t = len - 1 - it, n = it % kAhead;
    if (n == 0) {
      stage_ready<T, VPL, R>(st[(it / kAhead) & 1], gb);
      if (it + kAhead < len) gb = stage_fetch<T, VPL, R>(st[(it / kAhead + 1) & 1], src, t - kAhead, -1, len);
    }
    const TokenStage<T, VPL, R>& s = st[(it / kAhead) & 1];
    float kc[VPL], qc[VPL];
    load_vec<T, VPL>(&s.k[n][dk0], in, kc);
    load_vec<T, VPL>(&s.q[n][dk0], in, qc);
    const float dc = vin ? to_f<T>(s.x[n][warp * R + lane]) : 0.f, al = s.al[n], bl = CARRY ? s.bl[n] : 0.f, bc = s.beta[n];
    if ((t % kSimtChunk == kSimtChunk - 1 || it == 0) && in) {
      float* c = r.ckpt + (bh * nc + t / kSimtChunk) * head_elems + dk0;
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (dv0 + i < a.Dv) store_state<VPL>(c + static_cast<int64_t>(dv0 + i) * a.Dk, dS[i]);
    }
    float d[R], dd[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      dd[i] = a.scale * __shfl_sync(kFull, dc, i);
      if constexpr (CARRY && R == 8) {
        float x[VPL];
        add_times<VPL>(x, dS[i], dd[i], qc);
        d[i] = dot_part<VPL>(x, kc);
      } else {
        d[i] = 0.f;
#pragma unroll
        for (int j = 0; j < VPL; ++j) d[i] = fmaf(fmaf(dd[i], qc[j], dS[i][j]), kc[j], d[i]);
      }
    }
    if constexpr (CARRY) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        add_times<VPL>(L[i], L[i], dd[i], qc);
        carry_early<VPL>(dS[i], L[i], al, bl);
      }
    }
    const float sum = warp_sum_many<R>(d, lane);
    const float y = __shfl_sync(kFull, sum, sum_lane<R>(1) * (lane < R ? lane : 0));
    if (vin) *yt = y;
    yt -= a.Dv;
    const float de = bc * y;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float ei = __shfl_sync(kFull, de, i);
      if constexpr (CARRY) {
        carry_step<VPL>(dS[i], L[i], al, -al * ei, kc);
      } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j) dS[i][j] = fmaf(al, dS[i][j], al * fmaf(dd[i], qc[j], -ei * kc[j]));
      }
    }
  }
  if (r.ds0 && in) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (dv0 + i < a.Dv) store_state<VPL>(r.ds0 + bh * head_elems + static_cast<int64_t>(dv0 + i) * a.Dk + dk0, dS[i]);
  }
}

// Gradients of one chunk of C = 32 tokens, one key head and all value heads
// that share it, from the state before the chunk (S0), the state gradient after
// it (dS1), e and y.  With G the cumulative decay inside the chunk and
// D_ij = exp(G_i - G_j) for j <= i:
//   N = Y E^T, Pm = dO E^T
//   mP_ij = scale D_ij beta_j Pm_ij (j <= i),  mA_ij = -D_ij beta_i beta_j N_ij (j < i)
//   dq = scale e^G dO S0 + mP K
//   dk = -e^G beta Y S0 + e^{G_C - G} beta E dS1 + mP^T Q + mA K + mA^T K
//   dv = beta Y,  dbeta = diag N
//   dG_i = sums over row i minus column i of (mP * Q K^T + mA * K K^T), plus the
//          products of q and k with the terms through S0, minus k with the
//          term through dS1;  dg = suffix sums of dG plus <S1, dS1>.
// The decay gradient uses the pair sums, not q . dq - k . dk of whole rows, so
// that a pair on one side of a token cancels exactly instead of to rounding.
// Thread (i, l) of 256 owns token i and key columns l, l + 8, ...; the value
// columns pass in slices of 16, the next one on its way meanwhile.  Bound by
// shared memory reads, one for each multiply-add or two: 64 us for 68 chunks of
// two heads of 64 x 128 (110 before slices were fetched early).
constexpr int kCb = kSimtChunk;      // tokens
constexpr int kSlice = 16;           // value columns a pass

template <int DKM>
struct ChunkBwdSmem {
  static constexpr int P = DKM + 8;  // row pitch: four tokens of a warp fall on different banks
  float K[kCb][P], Q[kCb][P], dK[kCb][P], dQ[kCb][P];
  float S0[kSlice][P], dS[kSlice][P];
  float E[kCb][kSlice + 1], Y[kCb][kSlice + 1], dO[kCb][kSlice + 1];
  float mP[kCb][kCb + 1], mA[kCb][kCb + 1], X[kCb][kCb + 1];
  float Gh[kCb], Gl[kCb], eG[kCb], eE[kCb], beta[kCb], dG[kCb], w[kCb];
  float red[8];
};

template <typename T, int DKM>
__global__ void __launch_bounds__(256) delta_chunk_bwd_kernel(const DeltaChunkBwdArgs r) {
  constexpr int M = DKM / 8;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  ChunkBwdSmem<DKM>& sm = *reinterpret_cast<ChunkBwdSmem<DKM>*>(smem_raw);
  const DeltaArgs& a = r.a;
  const int tid = threadIdx.x, i = tid >> 3, l = tid & 7, lane = tid & 31;
  const int nc = (a.T + kCb - 1) / kCb;
  const int64_t bid = blockIdx.x;
  const int c = static_cast<int>(bid % nc);
  const int hk = static_cast<int>(bid / nc % a.Hk), b = static_cast<int>(bid / nc / a.Hk);
  const int t0 = c * kCb;
  const int len = a.len ? a.len[b] : a.T;
  const int nt = min(kCb, len - t0);            // valid tokens here, may be <= 0
  const int span = min(kCb, a.T - t0);          // rows that exist
  const int per = a.Hv / a.Hk;
  const int64_t qk_row = static_cast<int64_t>(a.Hk) * a.Dk, v_row = static_cast<int64_t>(a.Hv) * a.Dv;
  const int64_t head_elems = static_cast<int64_t>(a.Dv) * a.Dk;
  const int64_t trow = a.row(b, t0 + i < a.T ? t0 + i : 0);   // this thread's token

  for (int x = tid; x < kCb * a.Dk; x += 256) {
    const int ti = x / a.Dk, d = x - ti * a.Dk;
    const bool ok = ti < nt;
    const int64_t row = a.row(b, t0 + (ok ? ti : 0));
    sm.K[ti][d] = ok ? to_f<T>(static_cast<const T*>(a.k)[row * a.k_row + hk * a.Dk + d]) : 0.f;
    sm.Q[ti][d] = ok ? to_f<T>(static_cast<const T*>(a.q)[row * a.q_row + hk * a.Dk + d]) : 0.f;
    sm.dK[ti][d] = 0.f;
    sm.dQ[ti][d] = 0.f;
  }
  __syncthreads();
  float kk[4], qk[4];
#pragma unroll
  for (int jj = 0; jj < 4; ++jj) kk[jj] = qk[jj] = 0.f;
  for (int d = 0; d < a.Dk; ++d) {
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      const float kj = sm.K[l + 8 * jj][d];
      kk[jj] = fmaf(sm.K[i][d], kj, kk[jj]);
      qk[jj] = fmaf(sm.Q[i][d], kj, qk[jj]);
    }
  }

  for (int hh = 0; hh < per && nt > 0; ++hh) {
    const int h = hk * per + hh;
    const int64_t bh = static_cast<int64_t>(b) * a.Hv + h;
    if (tid < 32) {
      const bool ok = tid < nt;
      const int64_t row = a.row(b, t0 + (ok ? tid : 0));
      const float gg = ok ? to_f<T>(static_cast<const T*>(a.g)[row * a.g_row + h]) : 0.f;
      TwoF G = {gg < kDecayFloor ? kDecayFloor : gg, 0.f};
#pragma unroll
      for (int w = 1; w < 32; w <<= 1) {
        const TwoF up = {__shfl_up_sync(kFull, G.h, w), __shfl_up_sync(kFull, G.l, w)};
        if (tid >= w) G = two_add(up, G);
      }
      sm.Gh[tid] = G.h;
      sm.Gl[tid] = G.l;
      sm.eG[tid] = expf(G.h + G.l);
      sm.eE[tid] = expf((__shfl_sync(kFull, G.h, 31) - G.h) + (__shfl_sync(kFull, G.l, 31) - G.l));
      sm.beta[tid] = ok ? to_f<T>(static_cast<const T*>(a.beta)[row * a.beta_row + h]) : 0.f;
    }
    float N[4], Pm[4], dq1[M], dk1[M], dk3[M], frob = 0.f;
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) N[jj] = Pm[jj] = 0.f;
#pragma unroll
    for (int m = 0; m < M; ++m) dq1[m] = dk1[m] = dk3[m] = 0.f;
    // a slice waits in registers while the one before it is multiplied
    constexpr int NV = kCb * kSlice / 256, NS = kSlice * DKM / 256;
    float re[NV], ry[NV], ro[NV], rs[NS], rd[NS];
    auto fetch = [&](int v0) {
#pragma unroll
      for (int p = 0; p < NV; ++p) {
        const int x = tid + p * 256, ti = x / kSlice, d = x % kSlice;
        const bool ok = ti < nt && v0 + d < a.Dv;
        const int64_t at = ok ? (bh * a.T + t0 + ti) * a.Dv + v0 + d : 0;
        const int64_t row = a.row(b, t0 + (ok ? ti : 0));
        ry[p] = ok ? r.y[at] : 0.f;
        re[p] = ok ? r.e[at] : 0.f;
        ro[p] = ok ? to_f<T>(static_cast<const T*>(r.dout)[row * v_row + static_cast<int64_t>(h) * a.Dv + v0 + d]) : 0.f;
      }
#pragma unroll
      for (int p = 0; p < NS; ++p) {
        const int x = tid + p * 256, d = x / DKM, kx = x % DKM;
        const bool ok = v0 + d < a.Dv && kx < a.Dk;
        const int64_t at = ok ? (bh * nc + c) * head_elems + static_cast<int64_t>(v0 + d) * a.Dk + kx : 0;
        rs[p] = ok ? r.s0[at] : 0.f;
        rd[p] = ok ? r.ds1[at] : 0.f;
      }
    };
    fetch(0);
    for (int v0 = 0; v0 < a.Dv; v0 += kSlice) {
      __syncthreads();
#pragma unroll
      for (int p = 0; p < NV; ++p) {
        const int x = tid + p * 256, ti = x / kSlice, d = x % kSlice;
        sm.E[ti][d] = re[p];
        sm.Y[ti][d] = ry[p];
        sm.dO[ti][d] = ro[p];
        if (ti < nt && v0 + d < a.Dv)
          static_cast<T*>(r.dv)[a.row(b, t0 + ti) * v_row + static_cast<int64_t>(h) * a.Dv + v0 + d] = from_f<T>(sm.beta[ti] * ry[p]);
      }
#pragma unroll
      for (int p = 0; p < NS; ++p) {
        const int x = tid + p * 256, d = x / DKM, kx = x % DKM;
        sm.S0[d][kx] = rs[p];
        sm.dS[d][kx] = rd[p];
        frob = fmaf(rs[p], rd[p], frob);
      }
      __syncthreads();
      if (v0 + kSlice < a.Dv) fetch(v0 + kSlice);
      for (int d = 0; d < kSlice; ++d) {
        const float y = sm.Y[i][d], e = sm.E[i][d], dO = sm.dO[i][d];
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const float ej = sm.E[l + 8 * jj][d];
          N[jj] = fmaf(y, ej, N[jj]);
          Pm[jj] = fmaf(dO, ej, Pm[jj]);
        }
#pragma unroll
        for (int m = 0; m < M; ++m) {
          const float s0 = sm.S0[d][l + 8 * m], ds = sm.dS[d][l + 8 * m];
          dq1[m] = fmaf(dO, s0, dq1[m]);
          dk1[m] = fmaf(y, s0, dk1[m]);
          dk3[m] = fmaf(e, ds, dk3[m]);
        }
      }
    }
    // columns beyond Dk: keys and queries there are not loaded
    const float bi = sm.beta[i], eG = sm.eG[i];
    float own = 0.f, thru = 0.f;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const bool ok = l + 8 * m < a.Dk;
      dq1[m] = ok ? dq1[m] * a.scale * eG : 0.f;
      dk1[m] = ok ? -dk1[m] * eG * bi : 0.f;
      dk3[m] = ok ? dk3[m] * sm.eE[i] * bi : 0.f;
      const float qv = ok ? sm.Q[i][l + 8 * m] : 0.f, kv = ok ? sm.K[i][l + 8 * m] : 0.f;
      own = fmaf(qv, dq1[m], fmaf(kv, dk1[m], own));
      thru = fmaf(kv, dk3[m], thru);
    }
#pragma unroll
    for (int w = 1; w < 8; w <<= 1) {
      own += __shfl_xor_sync(kFull, own, w);
      thru += __shfl_xor_sync(kFull, thru, w);
    }
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) frob += __shfl_xor_sync(kFull, frob, w);
    if (lane == 0) sm.red[tid >> 5] = frob;
    float rows = 0.f;
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      const int j = l + 8 * jj;
      const float D = j <= i ? expf((sm.Gh[i] - sm.Gh[j]) + (sm.Gl[i] - sm.Gl[j])) : 0.f;
      const float mp = D * a.scale * sm.beta[j] * Pm[jj];
      const float ma = j < i ? -D * bi * sm.beta[j] * N[jj] : 0.f;
      sm.mP[i][j] = mp;
      sm.mA[i][j] = ma;
      const float x = mp * qk[jj] + ma * kk[jj];
      sm.X[i][j] = x;
      rows += x;
      if (j == i && i < nt) static_cast<T*>(r.dbeta)[trow * a.Hv + h] = from_f<T>(N[jj]);
    }
#pragma unroll
    for (int w = 1; w < 8; w <<= 1) rows += __shfl_xor_sync(kFull, rows, w);
    __syncthreads();
    float cols = 0.f;
    for (int j = l; j < kCb; j += 8) cols += sm.X[j][i];
#pragma unroll
    for (int w = 1; w < 8; w <<= 1) cols += __shfl_xor_sync(kFull, cols, w);
    if (l == 0) {
      sm.dG[i] = rows - cols + own - thru;
      sm.w[i] = thru;
    }
#pragma unroll
    for (int m = 0; m < M; ++m) {
      const int d = l + 8 * m;
      if (d >= a.Dk) continue;
      float dq = dq1[m], dk = dk1[m] + dk3[m];
      for (int j = 0; j < kCb; ++j) {
        dq = fmaf(sm.mP[i][j], sm.K[j][d], dq);
        dk = fmaf(sm.mP[j][i], sm.Q[j][d], dk);
        dk = fmaf(sm.mA[i][j] + sm.mA[j][i], sm.K[j][d], dk);
      }
      sm.dQ[i][d] += dq;
      sm.dK[i][d] += dk;
    }
    __syncthreads();
    if (tid < 32) {
      float x = sm.dG[tid], w = sm.w[tid], f = tid < 8 ? sm.red[tid] : 0.f;
#pragma unroll
      for (int s = 1; s < 32; s <<= 1) {
        const float dn = __shfl_down_sync(kFull, x, s);
        if (tid + s < 32) x += dn;
        w += __shfl_xor_sync(kFull, w, s);
        f += __shfl_xor_sync(kFull, f, s);
      }
      x += w + sm.eG[kCb - 1] * f;
      if (tid < nt) static_cast<T*>(r.dg)[a.row(b, t0 + tid) * a.Hv + h] = from_f<T>(x);
    }
    __syncthreads();
  }
  // gradients of masked tokens are zero
  for (int ti = max(nt, 0); ti < span; ++ti) {
    const int64_t row = a.row(b, t0 + ti);
    for (int hh = 0; hh < per; ++hh) {
      const int h = hk * per + hh;
      for (int d = tid; d < a.Dv; d += 256)
        static_cast<T*>(r.dv)[row * v_row + static_cast<int64_t>(h) * a.Dv + d] = from_f<T>(0.f);
      if (tid == 0) {
        static_cast<T*>(r.dg)[row * a.Hv + h] = from_f<T>(0.f);
        static_cast<T*>(r.dbeta)[row * a.Hv + h] = from_f<T>(0.f);
      }
    }
  }
  for (int x = tid; x < span * a.Dk; x += 256) {
    const int ti = x / a.Dk, d = x - ti * a.Dk;
    const int64_t at = a.row(b, t0 + ti) * qk_row + hk * a.Dk + d;
    // (a NaN in a valid token makes the sums of masked rows NaN as well)
    static_cast<T*>(r.dq)[at] = from_f<T>(ti < nt ? sm.dQ[ti][d] : 0.f);
    static_cast<T*>(r.dk)[at] = from_f<T>(ti < nt ? sm.dK[ti][d] : 0.f);
  }
}

int check_launch() { return cudaGetLastError() == cudaSuccess ? 0 : RNN_CUDA_ERROR; }

int vpl_of(int Dk) { return Dk <= 32 ? 1 : Dk <= 64 ? 2 : Dk <= 128 ? 4 : 8; }

// Where four rows a warp would leave schedulers without one, two: a token's
// chain is then shorter (fp32, 513 tokens of 128, with two and four rows a warp:
// 1024 rows 173 and 200 us, 2048 rows 194 and 201, 4096 rows 260 and 234).
bool few_rows(const DeltaArgs& a, int num_sms) {
  return static_cast<int64_t>(a.B) * a.Hv * a.Dv <= 16ll * num_sms;
}

// Where warps are many, what counts is instructions, and eight rows a warp share a
// token's (fp32, 256 tokens, forward and reverse: 65536 rows of 128 927 + 920 us
// against 1106 + 1015 with four rows, 8192 rows of 64 121 + 113 against 137 + 120;
// 4096 rows of 32 105 + 86 against 89 + 77).
bool many_rows(const DeltaArgs& a, int num_sms) {
  return static_cast<int64_t>(a.B) * a.Hv * a.Dv >= 48ll * num_sms;
}

// Sequences of at least this many tokens are staged (bf16, 4096 rows of 128, staged
// and not: 4 tokens 6.7 and 7.6 us, 8 tokens 7.3 and 10.4, 32 tokens 17 and 29;
// 98304 rows: 4 tokens 38.5 and 37.5, 8 tokens 56 and 58).
constexpr int kAheadFrom = 8;

template <typename T, int VPL, int R, bool AHEAD, bool CARRY>
int recur(const DeltaRecurArgs& r, cudaStream_t s) {
  const int64_t groups = (r.a.Dv + kWarps * R - 1) / (kWarps * R);
  delta_recur_kernel<T, VPL, R, AHEAD, CARRY><<<static_cast<unsigned>(groups * r.a.Hv * r.a.B), kWarps * 32, 0, s>>>(r);
  return check_launch();
}
template <typename T, int VPL>
int recur_v(const DeltaRecurArgs& r, cudaStream_t s) {
  constexpr bool f32 = sizeof(T) == 4;
  if (r.a.T >= kAheadFrom) {
    if constexpr (f32 && VPL <= 4) {
      if (many_rows(r.a, r.num_sms)) return recur<T, VPL, 8, true, true>(r, s);
    }
    return few_rows(r.a, r.num_sms) ? recur<T, VPL, 2, true, f32>(r, s) : recur<T, VPL, 4, true, f32>(r, s);
  }
  if constexpr (VPL <= 4) {
    // A step over more units than three CTAs an SM take in two turns.  With more
    // than two tokens the chain of a unit is longer than its transfer and the
    // recurrence's larger number of warps wins (128 x 128, pipeline and recurrence:
    // 256 sequences x 32 heads, one token 175 and 232 us, two 245 and 284, three 318
    // and 325, four 393 and 371; 48 x 16, one 21.7 and 22.1, two 28.0 and 27.2, three
    // 36.0 and 32.3).
    const int64_t units = static_cast<int64_t>((r.a.Dv + kUnitRows - 1) / kUnitRows) * r.a.Hv * r.a.B;
    if (r.status && r.a.T <= 2 && units >= 6 * r.num_sms && units + 3ll * kUnits * r.num_sms < (1ll << 31)) {
      const int smem = sizeof(StepSmem<VPL>);
      if (cudaFuncSetAttribute(delta_step_kernel<T, VPL>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return RNN_CUDA_ERROR;
      delta_step_kernel<T, VPL><<<3 * r.num_sms, kWarps * 32, smem, s>>>(r);
      return check_launch();
    }
  }
  if constexpr (VPL <= 4) {
    // several tokens for many states: bound by issue, where eight rows share a
    // token's work (48 sequences x 16 heads, four tokens: 25.6 against 27.6 us)
    if (static_cast<int64_t>(r.a.B) * r.a.Hv * r.a.Dv >= 256ll * r.num_sms && r.a.T > 1) return recur<T, VPL, 8, false, false>(r, s);
  }
  return recur<T, VPL, 4, false, false>(r, s);
}
template <typename T>
int recur_t(const DeltaRecurArgs& r, cudaStream_t s) {
  switch (vpl_of(r.a.Dk)) {
    case 1: return recur_v<T, 1>(r, s);
    case 2: return recur_v<T, 2>(r, s);
    case 4: return recur_v<T, 4>(r, s);
    default: return recur_v<T, 8>(r, s);
  }
}
template <typename T, int VPL, int R>
int recur_bwd(const DeltaRecurBwdArgs& r, cudaStream_t s) {
  const int64_t groups = (r.a.Dv + kWarps * R - 1) / (kWarps * R);
  delta_recur_bwd_kernel<T, VPL, R><<<static_cast<unsigned>(groups * r.a.Hv * r.a.B), kWarps * 32, 0, s>>>(r);
  return check_launch();
}
template <typename T, int VPL>
int recur_bwd_v(const DeltaRecurBwdArgs& r, cudaStream_t s) {
  if constexpr (sizeof(T) == 4 && VPL <= 4) {      // VPL 8 has no registers for eight rows
    if (many_rows(r.a, r.num_sms)) return recur_bwd<T, VPL, 8>(r, s);
  }
  return few_rows(r.a, r.num_sms) ? recur_bwd<T, VPL, 2>(r, s) : recur_bwd<T, VPL, 4>(r, s);
}
template <typename T>
int recur_bwd_t(const DeltaRecurBwdArgs& r, cudaStream_t s) {
  switch (vpl_of(r.a.Dk)) {
    case 1: return recur_bwd_v<T, 1>(r, s);
    case 2: return recur_bwd_v<T, 2>(r, s);
    case 4: return recur_bwd_v<T, 4>(r, s);
    default: return recur_bwd_v<T, 8>(r, s);
  }
}
template <typename T, int DKM>
int chunk_bwd(const DeltaChunkBwdArgs& r, cudaStream_t s) {
  const int smem = sizeof(ChunkBwdSmem<DKM>);
  if (cudaFuncSetAttribute(delta_chunk_bwd_kernel<T, DKM>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
      cudaSuccess)
    return RNN_CUDA_ERROR;
  const int64_t nc = (r.a.T + kCb - 1) / kCb;
  delta_chunk_bwd_kernel<T, DKM><<<static_cast<unsigned>(nc * r.a.Hk * r.a.B), 256, smem, s>>>(r);
  return check_launch();
}
template <typename T>
int chunk_bwd_t(const DeltaChunkBwdArgs& r, cudaStream_t s) {
  return r.a.Dk <= 64 ? chunk_bwd<T, 64>(r, s) : r.a.Dk <= 128 ? chunk_bwd<T, 128>(r, s) : chunk_bwd<T, 256>(r, s);
}

}  // namespace

int launch_delta_recur(const DeltaRecurArgs& r, int is_bf16, cudaStream_t s) {
  return is_bf16 ? recur_t<__nv_bfloat16>(r, s) : recur_t<float>(r, s);
}
int launch_delta_recur_bwd(const DeltaRecurBwdArgs& r, int is_bf16, cudaStream_t s) {
  return is_bf16 ? recur_bwd_t<__nv_bfloat16>(r, s) : recur_bwd_t<float>(r, s);
}
int launch_delta_chunk_bwd(const DeltaChunkBwdArgs& r, int is_bf16, cudaStream_t s) {
  return is_bf16 ? chunk_bwd_t<__nv_bfloat16>(r, s) : chunk_bwd_t<float>(r, s);
}

}  // namespace rnn
