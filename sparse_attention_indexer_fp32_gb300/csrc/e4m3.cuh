// E4M3 numbers: four bits of precision, largest 448, smallest normal 2^-6,
// steps of 2^-9 below; no infinities, one NaN (0x7f) of either sign.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

namespace tki {

// Two numbers rounded to nearest, past 448 to 448; the first in the low byte.
__device__ __forceinline__ uint32_t e4m3_two(float low, float high) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(high), "f"(low));
  return r;
}
// The two numbers of 16 bits, exactly.
__device__ __forceinline__ float2 e4m3_both(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The larger ones of two pairs of 16-bit numbers without a sign.
__device__ __forceinline__ uint32_t max_two(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

}  // namespace tki
