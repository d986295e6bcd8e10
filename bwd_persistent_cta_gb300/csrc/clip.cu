// clip.cu - the norm of many tensors together, and every one scaled by the same
// factor.
//
// The tensors lie end to end in one range of elements, which the CTAs share out
// evenly whatever the tensors' sizes: a CTA finds its first tensor by bisection and
// walks on from there.  One kernel leaves a sum of squares for each CTA, the other adds
// them up, in order, and scales.
#include "clip.h"
#include "common.cuh"
#include "pair.cuh"
#include "vec.cuh"

namespace rnn {

namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;
// Vectors of 16 bytes a thread, in flight at once: the norm's sums take registers of their
// own (252 MB of gradients: 50 us, 5.0 TB/s, with four, 61 with eight; scaling them, in place,
// 81 us, 6.2 TB/s, with eight, 83 with four).
constexpr int kNormVectors = 4, kScaleVectors = 8;

template <int CAP>
struct Pointers {
  const void* in[CAP];
  void* out[CAP];
};

// A launch's share of the list: tensors first .. first + num - 1.
struct Share {
  const int64_t* start;
  const int* dtype;
  int first, num;
  int64_t begin, end;          // elements
};

// The sum of squares of a few values.  Where fp32 would lose it (above 2^100, or so small
// that squares may have gone below the normal range) it is taken again in 64 bits.
template <int N>
__device__ __forceinline__ double squares(const float2 (&v)[N]) {
  float2 q[2] = {both(0.f), both(0.f)};
#pragma unroll
  for (int i = 0; i < N; ++i) q[i & 1] = fma2(v[i], v[i], q[i & 1]);
  const float2 p = add2(q[0], q[1]);
  const float s = p.x + p.y;
  if (s >= 0x1p-80f && s <= 0x1p100f) return s;
  float most = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) most = fmaxf(most, fmaxf(fabsf(v[i].x), fabsf(v[i].y)));
  if (most == 0.f && s == 0.f) return 0.0;               // gradients of rows that were not used
  double d = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i) d += static_cast<double>(v[i].x) * v[i].x + static_cast<double>(v[i].y) * v[i].y;
  return d;
}

// The last tensor that begins at or before element ``at``.
__device__ __forceinline__ int tensor_at(const Share& h, int64_t at) {
  int a = 0, b = h.num;
  while (b - a > 1) {
    const int m = (a + b) / 2;
    if (h.start[h.first + m] <= at) a = m;
    else b = m;
  }
  return a;
}
// Calls f(tensor, from, to) for the parts of the tensors that lie in lo .. hi, from the
// first to the last or the other way round.
template <bool BACK, typename F>
__device__ __forceinline__ void walk(const Share& h, int64_t lo, int64_t hi, F f) {
  for (int i = tensor_at(h, BACK ? hi - 1 : lo); i >= 0 && i < h.num; i += BACK ? -1 : 1) {
    const int64_t s = h.start[h.first + i], e = h.start[h.first + i + 1];
    const int64_t from = s > lo ? s : lo, to = e < hi ? e : hi;
    if (to > from) f(i, from - s, to - s);
    if (BACK ? s <= lo : e >= hi) break;
  }
}

template <typename T>
__device__ __forceinline__ double part_squares(const T* p, int64_t n) {
  // up to the first 16-byte boundary, and behind the last vector, one by one
  int64_t head = ((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T);
  if (head > n) head = n;
  constexpr int V = 16 / sizeof(T);
  const int64_t vecs = (n - head) / V, tail = head + vecs * V;
  double sum = 0.0;
  const int tid = threadIdx.x;
  if (tid < head) {
    const float2 one[1] = {make_float2(to_f(p[tid]), 0.f)};
    sum += squares(one);
  }
  if (tail + tid < n) {
    const float2 one[1] = {make_float2(to_f(p[tail + tid]), 0.f)};
    sum += squares(one);
  }
  constexpr int U = kNormVectors;
  int64_t i = tid;
  for (; i + (U - 1) * kThreads < vecs; i += U * kThreads) {
    Raw<T, V> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u].load(p + head + (i + u * kThreads) * V);
    float2 v[U * V / 2];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int j = 0; j < V / 2; ++j) v[u * V / 2 + j] = r[u].pair(j);
    sum += squares(v);
  }
  for (; i < vecs; i += kThreads) {
    Raw<T, V> r;
    r.load(p + head + i * V);
    float2 v[V / 2];
#pragma unroll
    for (int j = 0; j < V / 2; ++j) v[j] = r.pair(j);
    sum += squares(v);
  }
  return sum;
}

__device__ __forceinline__ double block_sum(double v, double* sm) {
#pragma unroll
  for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(kFull, v, m);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  for (int w = 0; w < kThreads / 32; ++w) v += sm[w];
  return v;
}

__device__ __forceinline__ void slice(const Share& h, int64_t* lo, int64_t* hi) {
  const int64_t per = ((h.end - h.begin + gridDim.x - 1) / gridDim.x + 7) & ~7LL;
  *lo = h.begin + per * blockIdx.x;
  *hi = *lo + per < h.end ? *lo + per : h.end;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) clip_norm_kernel(const __grid_constant__ Pointers<CAP> ptr, const Share h, double* partial) {
  __shared__ double sm[kThreads / 32];
  int64_t lo, hi;
  slice(h, &lo, &hi);
  double sum = 0.0;
  if (lo < hi)
    walk<false>(h, lo, hi, [&](int i, int64_t from, int64_t to) {
      if (h.dtype[h.first + i] == RNN_F32) sum += part_squares(static_cast<const float*>(ptr.in[i]) + from, to - from);
      else sum += part_squares(static_cast<const __nv_bfloat16*>(ptr.in[i]) + from, to - from);
    });
  sum = block_sum(sum, sm);
  if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// What every element is multiplied by: ``by``, then ``then`` twice.
struct Factor {
  float by, then;
  __device__ __forceinline__ bool one() const { return by == 1.f && then == 1.f; }
  __device__ __forceinline__ float2 of(float2 v) const { return mul2(mul2(mul2(v, both(by)), both(then)), both(then)); }
  __device__ __forceinline__ float of(float v) const { return v * by * then * then; }
};
// The norm and the factor, from the partial sums of all launches.  Both stay in 64 bits until
// they are done with: the sum cannot overflow there, so a norm that is not finite means a NaN
// or infinity among the gradients, while finite ones may have a norm that fp32 cannot hold.
// A factor below the normal numbers would lose bits: powers of two, exact, are multiplied
// behind it.
__device__ __forceinline__ Factor clip_factor(const double* partial, int parts, float max_norm, float eps, float* norm, double* sm) {
  double v = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) v += partial[i];
  v = block_sum(v, sm);
  __shared__ Factor f;
  // one thread: the root and the quotient by all 256 took 7 us of a large list's 495
  if (threadIdx.x == 0) {
    const double n = sqrt(v), d = n + eps;
    if (norm && blockIdx.x == 0) *norm = static_cast<float>(n);
    f = {1.f, 1.f};
    if (isfinite(n) && d > max_norm) {
      const double m = max_norm / d;           // 2^-298 at least: 2^42 elements
      if (m >= 0x1p-100) f.by = static_cast<float>(m);
      else if (m >= 0x1p-200) f = {static_cast<float>(m * 0x1p100), 0x1p-50f};
      else f = {static_cast<float>(m * 0x1p200), 0x1p-100f};
    }
  }
  __syncthreads();
  return f;
}

// From the end of the part to its beginning: what the norm's kernel read last is still in
// L2 (the last 126 MB of a long list), and outputs are stored past it.
template <typename T>
__device__ __forceinline__ void part_scale(const T* p, T* o, int64_t n, const Factor f) {
  constexpr int V = 16 / sizeof(T), U = kScaleVectors;
  int64_t head = ((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T);
  if (head > n) head = n;
  // where the output lies otherwise on its boundaries, element by element
  const bool same = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) == 0;
  const int64_t vecs = same ? (n - head) / V : 0, tail = head + vecs * V;
  const int tid = threadIdx.x;
  for (int64_t i = tail + tid; i < n; i += kThreads) o[i] = from_f<T>(f.of(to_f(p[i])));
  auto put = [&](const Raw<T, V>& r, int64_t i) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      const float2 v = f.of(r.pair(j));
      if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162 h = __float22bfloat162_rn(v);
        w[j] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[2 * j] = __float_as_uint(v.x);
        w[2 * j + 1] = __float_as_uint(v.y);
      }
    }
    __stcs(reinterpret_cast<uint4*>(o + head + i * V), make_uint4(w[0], w[1], w[2], w[3]));
  };
  int64_t i = vecs - 1 - tid;
  for (; i - (U - 1) * kThreads >= 0; i -= U * kThreads) {
    Raw<T, V> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u].load(p + head + (i - u * kThreads) * V);
#pragma unroll
    for (int u = 0; u < U; ++u) put(r[u], i - u * kThreads);
  }
  for (; i >= 0; i -= kThreads) {
    Raw<T, V> r;
    r.load(p + head + i * V);
    put(r, i);
  }
  if (tid < head) o[tid] = from_f<T>(f.of(to_f(p[tid])));
}

// Which tensors a launch scales.
enum { kAll, kApart, kInPlace };

template <int CAP>
__global__ void __launch_bounds__(kThreads) clip_scale_kernel(const __grid_constant__ Pointers<CAP> ptr, const Share h, const double* partial,
                                                              int parts, float max_norm, float eps, float* norm, int which) {
  __shared__ double sm[kThreads / 32];
  const Factor f = clip_factor(partial, parts, max_norm, eps, norm, sm);
  int64_t lo, hi;
  slice(h, &lo, &hi);
  if (lo >= hi) return;
  walk<true>(h, lo, hi, [&](int i, int64_t from, int64_t to) {
    const bool inplace = ptr.in[i] == ptr.out[i];
    // a factor of one leaves every element as it is: nothing to write in place
    if (inplace ? f.one() || which == kApart : which == kInPlace) return;
    if (h.dtype[h.first + i] == RNN_F32)
      part_scale(static_cast<const float*>(ptr.in[i]) + from, static_cast<float*>(ptr.out[i]) + from, to - from, f);
    else
      part_scale(static_cast<const __nv_bfloat16*>(ptr.in[i]) + from, static_cast<__nv_bfloat16*>(ptr.out[i]) + from, to - from, f);
  });
}

__global__ void __launch_bounds__(kThreads) clip_root_kernel(const double* partial, int parts, float* norm) {
  __shared__ double sm[kThreads / 32];
  clip_factor(partial, parts, 0.f, 0.f, norm, sm);
}

int check_launch() { return cudaGetLastError() == cudaSuccess ? 0 : RNN_CUDA_ERROR; }

int most_ctas(int num_sms) { return num_sms * (2048 / kThreads); }

template <int CAP>
int group(const ClipArgs& c, const Share& h, int ctas, bool scale, int which, double* mine, int parts, bool first, cudaStream_t s) {
  Pointers<CAP> p;
  for (int i = 0; i < h.num; ++i) {
    p.in[i] = c.grads[h.first + i];
    p.out[i] = c.out ? c.out[h.first + i] : const_cast<void*>(c.grads[h.first + i]);
  }
  if (scale) clip_scale_kernel<CAP><<<ctas, kThreads, 0, s>>>(p, h, c.partial, parts, c.max_norm, c.eps, first ? c.norm : nullptr, which);
  else clip_norm_kernel<CAP><<<ctas, kThreads, 0, s>>>(p, h, mine);
  return check_launch();
}

}  // namespace

size_t clip_workspace_bytes(int num, int num_sms) {
  const size_t groups = (num + kClipGroup - 1) / kClipGroup;
  return groups * most_ctas(num_sms) * sizeof(double);
}

int launch_clip(const ClipArgs& c, cudaStream_t s, int* launches) {
  *launches = 0;
  const int groups = (c.num + kClipGroup - 1) / kClipGroup;
  int rc = 0, parts = 0;
  for (int pass = 0; pass < (c.scale ? c.split ? 3 : 2 : 1); ++pass) {
    int at = 0;
    for (int g = 0; g < groups; ++g) {
      Share h{c.start, c.dtype, g * kClipGroup, 0, 0, 0};
      h.num = c.num - h.first < kClipGroup ? c.num - h.first : kClipGroup;
      h.begin = c.host_start[h.first];
      h.end = c.host_start[h.first + h.num];
      // at least 2048 elements a CTA
      const int64_t want = (h.end - h.begin + 2047) / 2048;
      const int most = most_ctas(c.num_sms), ctas = want < 1 ? 1 : want < most ? static_cast<int>(want) : most;
      const bool scale = pass > 0, first = pass == 1 && g == 0;
      const int which = c.split ? pass == 1 ? kApart : kInPlace : kAll;
      rc = h.num <= 100 ? group<100>(c, h, ctas, scale, which, c.partial + at, parts, first, s)
                        : group<kClipGroup>(c, h, ctas, scale, which, c.partial + at, parts, first, s);
      if (rc) return rc;
      ++*launches;
      at += ctas;
    }
    parts = at;
  }
  if (!c.scale) {
    clip_root_kernel<<<1, kThreads, 0, s>>>(c.partial, parts, c.norm);
    if ((rc = check_launch())) return rc;
    ++*launches;
  }
  return 0;
}

}  // namespace rnn
