// What the attention kernels share: exponentials in units of log 2, the tanh cap,
// and pairs of 16-bit numbers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cstdint>

#include "ptx.cuh"

namespace tki {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

template <typename E>
struct Pack;
template <>
struct Pack<__nv_bfloat16> {
  static constexpr uint32_t type = 1;
  static __device__ __forceinline__ uint32_t two(float x, float y) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
template <>
struct Pack<__half> {
  static constexpr uint32_t type = 0;
  static __device__ __forceinline__ uint32_t two(float x, float y) {
    const __half2 v = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};

__device__ __forceinline__ float exp2_fast(float x) {  // 2 ulp
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A capped logit c tanh(z / c), z = x scale, in units of log 2, good to 5 2^-23 of
// itself whatever the cap. With u = z / c: c (1 - 2 / (1 + e^2u)) from |u| = kBent on;
// below, where that difference cancels (its error is one of c, however small z is),
// z (1 + u^2 P(u^2)), P a fit of (tanh(u) / u - 1) / u^2 to 2^-24 of the result.
// Two logits at a time: one by one, 2048 rows x 512 shared entries take 171 us
// in place of 154, 1024 rows with 128 heads 146 in place of 117.
constexpr float kBent = 0.5f;
// Two numbers at a time.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ uint64_t twice(float x) { return pair(x, x); }
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ float2 both(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ float reciprocal(float x) {  // 1 ulp
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// x is two products, u = x scale / cap.
__device__ __forceinline__ float2 capped_low(uint64_t x, uint64_t u, float scale_log2e) {
  const uint64_t u2 = mul2(u, u);
  uint64_t p = fma2(twice(1.7999219e-2f), u2, twice(-5.3391054e-2f));
  p = fma2(p, u2, twice(1.3330513e-1f));
  p = fma2(p, u2, twice(-3.3333310e-1f));
  return both(mul2(mul2(x, twice(scale_log2e)), fma2(p, u2, twice(1.0f))));
}
__device__ __forceinline__ float2 capped_high(uint64_t u, float cap_log2e) {
  const float2 a = both(mul2(u, twice(2.0f * kLog2e)));
  const float2 e = both(add2(pair(exp2_fast(a.x), exp2_fast(a.y)), twice(1.0f)));
  return both(mul2(fma2(twice(-2.0f), pair(reciprocal(e.x), reciprocal(e.y)), twice(1.0f)), twice(cap_log2e)));
}

__device__ __forceinline__ bool is_low(float x) { return x == __int_as_float(0xff800000); }

__device__ __forceinline__ float4 ld_dsmem_f4(uint32_t addr) {
  const uint4 v = ld_dsmem_v4(addr);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}

// In FP32, the largest number where it has none: a product of zero stays zero.
inline float finite(double x) {
  const double most = FLT_MAX;
  return static_cast<float>(x > most ? most : x < -most ? -most : x);
}

}  // namespace tki
