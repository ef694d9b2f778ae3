// Device helpers shared by the layer operators (causal convolution, selective
// scan, single-token steps, block norm): vector loads and stores of bf16 /
// fp32 rows as fp32 registers, and the softplus / sigmoid / exp2 they use.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

namespace ssd {
namespace lm {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// V consecutive elements as raw storage: one 16- or 8-byte access where V
// elements are that wide (the address is then that aligned: see vec_ok),
// two for 8 floats, else one element.
template <typename T, int V>
struct Raw;
template <>
struct Raw<__nv_bfloat16, 8> {
  uint4 u;
};
template <>
struct Raw<__nv_bfloat16, 4> {
  uint2 u;
};
template <>
struct Raw<float, 4> {
  uint4 u;
};
template <>
struct Raw<float, 8> {
  uint4 u, v;
};
template <typename T>
struct Raw<T, 1> {
  T u;
};

template <typename T, int V>
__device__ __forceinline__ Raw<T, V> ld_raw(const T* p) {
  return *reinterpret_cast<const Raw<T, V>*>(p);
}
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> zero_raw() {
  Raw<T, V> r;
  if constexpr (V == 1) {
    r.u = from_f<T>(0.f);
  } else if constexpr (sizeof(r.u) == 8) {
    r.u = make_uint2(0, 0);
  } else {
    r.u = make_uint4(0, 0, 0, 0);
    if constexpr (sizeof(r) == 32) r.v = make_uint4(0, 0, 0, 0);
  }
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void unpack(const Raw<T, V>& r, float (&f)[V]) {
  const T* e = reinterpret_cast<const T*>(&r);
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = to_f(e[i]);
}
template <typename T, int V>
__device__ __forceinline__ Raw<T, V> pack(const float (&f)[V]) {
  Raw<T, V> r;
  T* e = reinterpret_cast<T*>(&r);
#pragma unroll
  for (int i = 0; i < V; ++i) e[i] = from_f<T>(f[i]);
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void st_raw(T* p, const Raw<T, V>& r) {
  *reinterpret_cast<Raw<T, V>*>(p) = r;
}

// Whether rows of `stride` elements of `esize` bytes starting at p can be
// accessed in vectors of v elements.
__host__ __device__ inline bool vec_ok(const void* p, int64_t stride, int esize, int v) {
  const int64_t bytes = (int64_t)v * esize < 16 ? (int64_t)v * esize : 16;
  return (reinterpret_cast<uintptr_t>(p) % bytes) == 0 && (stride * esize) % bytes == 0;
}

__device__ __forceinline__ float ex2(float v) {  // 2^v (MUFU, ~2 ulp; 0 below 2^-126)
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// 1 / (1 + e^-v): e^-v = inf for v < -88 gives exactly 0.
__device__ __forceinline__ float sigmoid(float v) {
  return __fdividef(1.f, 1.f + ex2(-v * kLog2e));
}

// softplus(v) = log(1 + e^v), v itself above 20.  With e = e^-|v| it is
// max(v, 0) + log(1 + e), and log(1 + e) = 2 atanh(s), s = e / (2 + e) <= 1/3:
// the series 2 s (1 + s^2/3 + s^4/5 + ...) up to s^14 / 15 leaves less than
// s^16 / 17 < 2e-9 of it.  Steps are typically 1e-3 to 1e-1, where 1 + e in fp32
// would round away what the logarithm needs; this form keeps ~5e-7 relative.
__device__ __forceinline__ float softplus(float v) {
  const float e = ex2(-fabsf(v) * kLog2e);
  const float s = __fdividef(e, 2.f + e), q = s * s;
  float p = 1.f / 15.f;
  p = fmaf(p, q, 1.f / 13.f);
  p = fmaf(p, q, 1.f / 11.f);
  p = fmaf(p, q, 1.f / 9.f);
  p = fmaf(p, q, 1.f / 7.f);
  p = fmaf(p, q, 1.f / 5.f);
  p = fmaf(p, q, 1.f / 3.f);
  p = fmaf(p, q, 1.f);
  return v > 20.f ? v : fmaxf(v, 0.f) + 2.f * s * p;
}

}  // namespace lm
}  // namespace ssd
