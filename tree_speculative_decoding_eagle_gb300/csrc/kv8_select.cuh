// What the kernels of the page selection share.
#pragma once

#include "kv8.cuh"

namespace eagle {

struct SelectArgs {
  const __nv_bfloat16 *q;
  const uint8_t *bounds;
  const float *k_scale;
  const int32_t *block_table, *kv_len;
  float *scores;  // workspace [B * n * Hkv, stride]
  int32_t *sel;
  float *sel_score;
  int32_t *status;
  int B, n, Hq, Hkv, G, log_g;  // 2^log_g: heads of a KV head, padded
  int log_page, max_pages, num_pages, stride, top, first, last;
};

// Pages of a request's prefix.
__device__ __forceinline__ int live_pages(const SelectArgs &a, int b) {
  const int64_t L = min(static_cast<int64_t>(max(a.kv_len[b], 0)), static_cast<int64_t>(a.max_pages) << a.log_page);
  return static_cast<int>((L + (1 << a.log_page) - 1) >> a.log_page);
}
__device__ __forceinline__ float finite_or_zero(float x) { return fabsf(x) <= 3.402823466e38f ? x : 0.f; }
// Two of a row's numbers as whole numbers in f16.
__device__ __forceinline__ uint32_t whole_half2(uint32_t w, float f) {
  const float lo = rintf(finite_or_zero(bf16_lo(w)) * f), hi = rintf(finite_or_zero(bf16_hi(w)) * f);
  const __half2 h = __floats2half2_rn(fminf(fmaxf(lo, -128.f), 128.f), fminf(fmaxf(hi, -128.f), 128.f));
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t half2_max0(uint32_t w) {
  const __half2 h = __hmax2(*reinterpret_cast<const __half2 *>(&w), __float2half2_rn(0.f));
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t half2_min0(uint32_t w) {
  const __half2 h = __hmin2(*reinterpret_cast<const __half2 *>(&w), __float2half2_rn(0.f));
  return *reinterpret_cast<const uint32_t *>(&h);
}
// The exponent e of a row with amax / 2^e in [64, 128).
__device__ __forceinline__ int whole_exponent(float amax) {
  return amax > 0.f ? min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 6, -32), 32) : 0;
}
// Largest magnitude of eight packed numbers that are finite.
__device__ __forceinline__ float finite_amax8(const uint4 &x) {
  float f[8], amax = 0.f;
  VecTraits<__nv_bfloat16>::unpack(x, f);
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(finite_or_zero(f[e])));
  return amax;
}

}  // namespace eagle
