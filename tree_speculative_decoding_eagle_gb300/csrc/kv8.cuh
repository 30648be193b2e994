// The 8-bit cache's numbers: e4m3 with a power-of-two scale for each block.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace eagle {

constexpr int kScaleMin = -64, kScaleMax = 64;  // exponents of a block's scale

// The least e with amax <= 448 * 2^e = 1.75 * 2^(e+8), clamped; amax >= 0 finite.
__device__ __forceinline__ int block_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kScaleMin), kScaleMax);
}
__device__ __forceinline__ float exponent_scale(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }
// Exponent of a stored scale: of the power of two below it, clamped.
__device__ __forceinline__ int scale_exponent(float s) {
  const int e = static_cast<int>((__float_as_uint(s) >> 23) & 0xffu) - 127;
  return min(max(e, kScaleMin), kScaleMax);
}

// Two floats to two e4m3 numbers (lo in the low byte), to nearest even,
// saturating; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 numbers (low 16 bits) to packed f16, exactly.
__device__ __forceinline__ uint32_t e4m3_to_half2(uint32_t pair) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(pair)));
  return r;
}

// Largest magnitude of eight packed bf16 numbers.
__device__ __forceinline__ float amax8(const uint4 &v) {
  const uint4 a = make_uint4(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu);
  return vec_max<__nv_bfloat16>(a);
}

}  // namespace eagle
