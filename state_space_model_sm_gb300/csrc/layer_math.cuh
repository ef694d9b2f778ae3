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

__device__ __forceinline__ float rcp(float v) {  // 1 / v (MUFU, 1 ulp; 0 for inf)
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// 1 / (1 + e^-v): e^-v = inf for v < -88 gives exactly 0.
__device__ __forceinline__ float sigmoid(float v) { return rcp(1.f + ex2(-v * kLog2e)); }

// softplus(v) = log(1 + e^v).  With e = e^-|v| it is max(v, 0) + log(1 + e), and
// log(1 + e) = 2 atanh(s), s = e / (2 + e) <= 1/3.  atanh(s) / s as a polynomial in
// q = s^2 on [0, 1/9], interpolated at the Chebyshev nodes: degree 4 is within
// 8e-9.  Steps are typically 1e-3 to 1e-1, where 1 + e in fp32 would round away
// what the logarithm needs; this form is within 5e-7 + 1e-7 max(-v, 0) of the value
// (the second part from the rounding of v log2(e), which e^-|v| passes on); above 20
// it is v, as e vanishes against v, and below -87 0, as e is not a normal number.
constexpr float kAtanh1 = 0.3333316147327423f, kAtanh2 = 0.20012298226356506f,
                kAtanh3 = 0.13982579112052917f, kAtanh4 = 0.14078889787197113f;
__device__ __forceinline__ float softplus(float v) {
  const float e = ex2(-fabsf(v) * kLog2e);
  const float s = e * rcp(2.f + e), q = s * s;
  float p = fmaf(kAtanh4, q, kAtanh3);
  p = fmaf(p, q, kAtanh2);
  p = fmaf(p, q, kAtanh1);
  p = fmaf(p, q, 1.f);
  return fmaf(s + s, p, fmaxf(v, 0.f));
}

// Pairs, for the packed fp32 instructions (one issue for two operations).
__device__ __forceinline__ float2 f2(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  return __ffma2_rn(a, b, c);
}
__device__ __forceinline__ float2 ex2_2(float2 v) { return make_float2(ex2(v.x), ex2(v.y)); }
__device__ __forceinline__ float2 rcp_2(float2 v) { return make_float2(rcp(v.x), rcp(v.y)); }
__device__ __forceinline__ float2 sigmoid2(float2 v) {
  return rcp_2(add2(f2(1.f), ex2_2(mul2(v, f2(-kLog2e)))));
}
__device__ __forceinline__ float2 softplus2(float2 v) {
  const float2 e = ex2_2(mul2(make_float2(fabsf(v.x), fabsf(v.y)), f2(-kLog2e)));
  const float2 s = mul2(e, rcp_2(add2(f2(2.f), e))), q = mul2(s, s);
  float2 p = fma2(f2(kAtanh4), q, f2(kAtanh3));
  p = fma2(p, q, f2(kAtanh2));
  p = fma2(p, q, f2(kAtanh1));
  p = fma2(p, q, f2(1.f));
  return fma2(add2(s, s), p, make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}

// The decay e^(delta A) of a step, from a2 = A log2(e).  Measured over its range,
// the instruction's 2^v lies 2e-8 low on average (a third of an ulp); over the
// hundreds of steps that a slow state remembers the product of decays would
// drift by that many times 2e-8 (gradients of A by 1e-6, three times what
// correctly rounded exponentials give).  A constant in the exponent takes the mean
// out; at delta = 0 the result is exactly 1.
constexpr float kDecayMean = 2.9e-8f;
__device__ __forceinline__ float decay(float delta, float a2) {
  return ex2(fmaf(delta, a2, kDecayMean));
}
__device__ __forceinline__ float2 decay2(float delta, float2 a2) {
  return ex2_2(fma2(f2(delta), a2, f2(kDecayMean)));
}

// The same for single values, for code over either.
__device__ __forceinline__ float mul2(float a, float b) { return a * b; }
__device__ __forceinline__ float add2(float a, float b) { return a + b; }
__device__ __forceinline__ float fma2(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float sigmoid2(float v) { return sigmoid(v); }

// Two adjacent elements as one access where wide (their address is then
// aligned to both), else as two; `two` says whether there is a second one.
template <typename T>
struct alignas(2 * sizeof(T)) Two {
  T a, b;
};
template <typename T>
__device__ __forceinline__ Two<T> ld_two(const T* p, bool two, bool wide) {
  if (wide) return *reinterpret_cast<const Two<T>*>(p);
  Two<T> r;
  r.a = p[0];
  r.b = p[two ? 1 : 0];
  return r;
}
__device__ __forceinline__ float2 unpack2(const Two<float>& r) { return make_float2(r.a, r.b); }
__device__ __forceinline__ float2 unpack2(const Two<__nv_bfloat16>& r) {
  return __bfloat1622float2(__halves2bfloat162(r.a, r.b));
}
template <typename T>
__device__ __forceinline__ void st_two(T* p, float2 v, bool two, bool wide) {
  if (wide) {
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float2*>(p) = v;
    else
      *reinterpret_cast<__nv_bfloat162*>(p) = __float22bfloat162_rn(v);
  } else {
    p[0] = from_f<T>(v.x);
    if (two) p[1] = from_f<T>(v.y);
  }
}

// Asynchronous copies of 4, 8 or 16 bytes into shared memory.
template <int BYTES>
__device__ __forceinline__ void cp_async(void* dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(BYTES)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_wait() {  // until at most N groups are in flight
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace lm
}  // namespace ssd
