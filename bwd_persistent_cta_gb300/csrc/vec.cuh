// vec.cuh - a thread's V consecutive elements: loads, pairs of fp32 values, stores.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace rnn {

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

}  // namespace rnn
