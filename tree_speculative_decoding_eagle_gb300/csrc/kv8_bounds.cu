// The bounds of a page's keys: for each page, head and column the least and the
// greatest e4m3 number over the page's rows, rounded outwards to halves.
//
// e4m3 numbers below 8 that are multiples of 1/2 are e4m3 numbers, and all from 4
// on are multiples of 1/2, so the rounded bounds are held in e4m3 exactly, in units
// of the page's scale.  What the rounding is for: a selection's sums of products
// with whole numbers are then multiples of 1/2 below 2^23, exact in float32 in any
// order (kv8_select.cu).  It widens a bound by less than half a unit of a page
// whose largest number lies in (224, 448].
//
// What bounds it: HBM for prompts (one byte read an element), latency for single
// tokens.  A warp takes a page of a head: a lane looks after 16 neighbouring columns
// of every fourth (or eighth) row, 16 bytes a request with up to eight requests
// in flight, as f16 pairs (e4m3 to f16 is exact, and f16 has packed minima and maxima);
// the lanes of a column then hand their results down, halving the columns that a
// lane still looks after at each step.
// Measured, on the device: 16 prompts of 4096 tokens, 8 heads of 128, 15.0 us (67 MB
// read, 69 MB in all, 69 % of the copy rate); one more token of each of 64 requests, 8
// heads of 64, pages of 64, 5.5 us.
#include "kv8.cuh"

namespace eagle {

constexpr int kBoundWarps = 4;

struct BoundArgs {
  const uint8_t *k_pages;
  const int32_t *block_table, *from_len, *kv_len;
  uint8_t *bounds;
  int32_t *status;
  int Hkv, log_page, max_pages, num_pages;
};

__device__ __forceinline__ __half2 as_half2(uint32_t w) { return *reinterpret_cast<const __half2 *>(&w); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<const uint32_t *>(&h); }
// Two f16 numbers that are e4m3 numbers to their codes (lo in the low byte).
__device__ __forceinline__ uint32_t half2_to_e4m3(uint32_t w) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(w));
  return r;
}

template <int DH>
__global__ void __launch_bounds__(kBoundWarps * 32, 8) kv8_bounds_kernel(BoundArgs a) {
  constexpr int LANES = DH / 16, ROWS = 32 / LANES;  // lanes a row, rows a request
  constexpr int AHEAD = 32 / ROWS;                   // requests in flight: 32 rows
  const int b = blockIdx.y, lane = threadIdx.x & 31, col = lane % LANES, sub = lane / LANES;
  const int P = 1 << a.log_page;
  pdl_wait();
  pdl_trigger();
  const int from = max(a.from_len[b], 0);
  const int L = static_cast<int>(min(static_cast<int64_t>(a.kv_len[b]), static_cast<int64_t>(a.max_pages) << a.log_page));
  if (L <= from) return;
  const int first = from >> a.log_page, pages = ((L - 1) >> a.log_page) - first + 1;
  const int64_t units = static_cast<int64_t>(pages) * a.Hkv;
  for (int64_t u = static_cast<int64_t>(blockIdx.x) * kBoundWarps + (threadIdx.x >> 5); u < units;
       u += static_cast<int64_t>(gridDim.x) * kBoundWarps) {
    const int lp = first + static_cast<int>(u / a.Hkv), g = static_cast<int>(u % a.Hkv);
    const int page = a.block_table[static_cast<int64_t>(b) * a.max_pages + lp];
    if (page < 0 || page >= a.num_pages) {
      if (lane == 0) report(a.status, EAGLE_ERR_INVALID);
      continue;
    }
    const int rows = min(P, L - (lp << a.log_page));
    const int64_t block = static_cast<int64_t>(page) * a.Hkv + g;
    const uint8_t *src = a.k_pages + (block << a.log_page) * DH + col * 16;
    uint32_t hi[8], lo[8];  // columns 2i, 2i + 1 of the lane's 16
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      hi[i] = 0xfc00fc00u;  // -inf
      lo[i] = 0x7c007c00u;
    }
    for (int r0 = 0; r0 < rows; r0 += ROWS * AHEAD) {
      uint4 x[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i)  // in the last request, past the last row: that row again
        if (r0 + i * ROWS < rows) x[i] = ld_stream16(src + static_cast<int64_t>(min(r0 + i * ROWS + sub, rows - 1)) * DH);
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (r0 + i * ROWS >= rows) break;
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t v = e4m3_to_half2(j & 1 ? w[j / 2] >> 16 : w[j / 2] & 0xffffu);
          hi[j] = as_u32(__hmax2_nan(as_half2(hi[j]), as_half2(v)));
          lo[j] = as_u32(__hmin2_nan(as_half2(lo[j]), as_half2(v)));
        }
      }
    }
    // Lanes sub and sub ^ 1, ^ 2 (and ^ 4) share the columns: each step a lane keeps
    // half of those it has and hands the other half over.
    int c0 = 0;  // the first pair that this lane still looks after
#pragma unroll
    for (int o = 1, keep = 4; o < ROWS; o *= 2, keep /= 2) {
      const bool upper = sub & o;
#pragma unroll
      for (int i = 0; i < keep; ++i) {
        const uint32_t gh = upper ? hi[i] : hi[i + keep], gl = upper ? lo[i] : lo[i + keep];
        const uint32_t mh = upper ? hi[i + keep] : hi[i], ml = upper ? lo[i + keep] : lo[i];
        hi[i] = as_u32(__hmax2_nan(as_half2(mh), as_half2(__shfl_xor_sync(0xffffffffu, gh, o * LANES))));
        lo[i] = as_u32(__hmin2_nan(as_half2(ml), as_half2(__shfl_xor_sync(0xffffffffu, gl, o * LANES))));
      }
      if (upper) c0 += keep;
    }
    constexpr int KEPT = 8 / ROWS;  // pairs a lane ends up with: two (DH = 128) or one
    const __half2 two = __float2half2_rn(2.f), half = __float2half2_rn(0.5f);
    uint16_t *dst = reinterpret_cast<uint16_t *>(a.bounds + block * 2 * DH) + col * 8 + c0;
#pragma unroll
    for (int i = 0; i < KEPT; ++i) {
      // a NaN among the rows: as wide as it can be
      const uint32_t bad = __vcmpgtu2(hi[i] & 0x7fff7fffu, 0x7c007c00u);
      const uint32_t l = as_u32(__hmul2(h2floor(__hmul2(as_half2(lo[i]), two)), half));
      const uint32_t h = as_u32(__hmul2(h2ceil(__hmul2(as_half2(hi[i]), two)), half));
      dst[i] = static_cast<uint16_t>(half2_to_e4m3((l & ~bad) | (0xdf00df00u & bad)));           // -448
      dst[DH / 2 + i] = static_cast<uint16_t>(half2_to_e4m3((h & ~bad) | (0x5f005f00u & bad)));
    }
  }
}

cudaError_t launch_kv8_bounds(const uint8_t *k_pages, const int32_t *block_table, int max_pages, int page_size,
                              int num_pages, const int32_t *from_len, const int32_t *kv_len, int B, int Hkv, int dh,
                              uint8_t *bounds, int32_t *status, int num_sms, cudaStream_t st) {
  int log_page = 0;
  while ((1 << log_page) < page_size) ++log_page;
  const BoundArgs a = {k_pages, block_table, from_len, kv_len, bounds, status, Hkv, log_page, max_pages, num_pages};
  // Which pages are touched is known on the device alone: each request has CTAs for
  // its share of sixteen an SM, at most one warp for each page and head.
  const int64_t most = (static_cast<int64_t>(max_pages) * Hkv + kBoundWarps - 1) / kBoundWarps;
  const int64_t share = (16ll * num_sms + B - 1) / B;
  const dim3 grid(static_cast<unsigned>(share < most ? share : most), B);
  return dh == 128 ? launch_chained(kv8_bounds_kernel<128>, grid, dim3(kBoundWarps * 32), 0, st, a)
                   : launch_chained(kv8_bounds_kernel<64>, grid, dim3(kBoundWarps * 32), 0, st, a);
}

}  // namespace eagle
