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
// The exponent e of a row with amax / 2^e in [64, 128).
__device__ __forceinline__ int whole_exponent(float amax) {
  return amax > 0.f ? min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 6, -32), 32) : 0;
}
// Eight packed numbers, the ones that are not finite as zeros.
__device__ __forceinline__ uint4 finite8(uint4 x) {
  uint32_t *w = &x.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] &= ~__vcmpeq2(w[i] & 0x7f807f80u, 0x7f807f80u);
  return x;
}

}  // namespace eagle
