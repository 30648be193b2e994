// What the two kernels of the attention over the 8-bit cache share: their
// arguments, the powers of two, and the merge of a KV split.
#pragma once

#include "kv8.cuh"
#include "sm100.cuh"
#include "tmap.cuh"

namespace eagle {

constexpr int kMaxClusterSplits8 = 8;  // KV splits that one cluster merges
constexpr float kBias = 6.f;      // P' = 2^(kBias + ...)

struct Kv8Args {
  const __nv_bfloat16 *q, *k_tree, *v_tree;
  const float *k_scale, *v_scale;
  const int32_t *block_table, *kv_len;
  const uint64_t *mask;
  int B, n, Hq, Hkv, G, W, S;
  int page_size, log_page, page_box, max_pages, num_pages;
  float scale_log2;  // softmax scale times log2(e)
  __nv_bfloat16 *out;
  float *lse;
  int32_t *status;
  // KV split (S > 1): one workspace slot per CTA, [slot_rows][DH] fp32 O rows
  // then [slot_rows] (m, l) pairs, the slots of a (b, g, M-group) consecutive
  float *part;
  int slot_rows;
};

// 2^e in float32 for any int e that a sum of exponents can give, kept away
// from 0 and infinity (0 * inf must not arise from finite inputs).
__device__ __forceinline__ float pow2_clamped(int e) { return exponent_scale(min(max(e, -120), 120)); }

// The exponent e with amax / 2^e in [2^8, 2^9), where an e4m3 block's numbers
// end too: a bf16 number keeps its 8 bits in f16 down to 2^-25 of amax.
__device__ __forceinline__ int half_exponent(float amax) {
  if (amax == 0.f) return 0;
  return max(static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 8, -100);
}
__device__ __forceinline__ uint32_t bf16x2_to_half2(uint32_t w, float f) {
  const __half2 h = __floats2half2_rn(bf16_lo(w) * f, bf16_hi(w) * f);
  return *reinterpret_cast<const uint32_t *>(&h);
}
// Largest magnitude of eight packed bf16 numbers.
__device__ __forceinline__ float amax8(const uint4 &v) {
  const uint4 a = make_uint4(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu);
  return vec_max<__nv_bfloat16>(a);
}

// Columns 4c..4c+3 of query row rho of (b, g): out = o / l, lse from (m, l).
template <int DH>
__device__ __forceinline__ void kv8_write_out(const Kv8Args &a, int bg, int rho, int c, float4 o, float m, float l) {
  const float inv = l == 0.f ? 0.f : 1.f / l;  // a NaN stays one
  const int i = rho / a.G, h = (bg % a.Hkv) * a.G + rho % a.G;
  const int64_t orow = (static_cast<int64_t>(bg / a.Hkv) * a.n + i) * a.Hq + h;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv), hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  uint2 packed;
  packed.x = *reinterpret_cast<const uint32_t *>(&lo);
  packed.y = *reinterpret_cast<const uint32_t *>(&hi);
  reinterpret_cast<uint2 *>(a.out + orow * DH)[c] = packed;
  if (c == 0 && a.lse) a.lse[orow] = l == 0.f ? -INFINITY : (m - kBias + log2f(l)) * kLn2;
}

// out and lse of row rr, columns 4c..4c+3, of a (b, g, M-group) from its S
// slots: out = sum_s w_s O_s / sum_s w_s l_s with w_s = 2^(m_s - max m).
// Eight splits' values are in flight at a time.
template <int DH>
__device__ __forceinline__ void kv8_merge_item(const Kv8Args &a, int bg, int mg, int MT, int rr, int c) {
  constexpr int NV = DH / 4;
  const int64_t slot_floats = static_cast<int64_t>(a.slot_rows) * (DH + 2);
  const float *slots = a.part + (static_cast<int64_t>(bg) * gridDim.y + mg) * a.S * slot_floats;
  float M = -INFINITY, Ls = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 0; s0 < a.S; s0 += 8) {
    float2 ml[8];
    float4 po[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int s = s0 + u;
      if (s < a.S) {
        ml[u] = __ldcg(reinterpret_cast<const float2 *>(slots + s * slot_floats + static_cast<int64_t>(a.slot_rows) * DH) + rr);
        po[u] = __ldcg(reinterpret_cast<const float4 *>(slots + s * slot_floats) + rr * NV + c);
      } else {
        ml[u] = make_float2(-INFINITY, 0.f);
        po[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    float Mn = M;
#pragma unroll
    for (int u = 0; u < 8; ++u) Mn = fmaxf(Mn, ml[u].x);
    const float w0 = M > -INFINITY ? ex2_approx(M - Mn) : 0.f;
    M = Mn;
    Ls *= w0;
    o.x *= w0; o.y *= w0; o.z *= w0; o.w *= w0;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float w = ml[u].x > -INFINITY ? ex2_approx(ml[u].x - M) : 0.f;
      Ls = fmaf(w, ml[u].y, Ls);
      if (w != 0.f) {
        o.x = fmaf(w, po[u].x, o.x); o.y = fmaf(w, po[u].y, o.y);
        o.z = fmaf(w, po[u].z, o.z); o.w = fmaf(w, po[u].w, o.w);
      }
    }
  }
  const int rho = mg * MT * 128 + rr;
  kv8_write_out<DH>(a, bg, rho, c, o, M, Ls);
}

// The merge of a split launch of several waves: one thread per (row, 4 columns).
template <int DH>
__global__ void __launch_bounds__(256) tree_attn_kv8_merge_kernel(Kv8Args a, int MT) {
  constexpr int NV = DH / 4;
  const int mg = blockIdx.y, bg = blockIdx.z;
  const int nr = max(0, min(a.n * a.G - mg * MT * 128, MT * 128));
  const int item = blockIdx.x * blockDim.x + threadIdx.x;
  pdl_wait();  // the partial results come from the attention kernel
  if (item < nr * NV) kv8_merge_item<DH>(a, bg, mg, MT, item / NV, item % NV);
}

// A pool [num_pages * Hkv, page_size, dh] of bytes in boxes of page_box rows,
// plain or with the swizzle of a row's width.  Three dimensions, so no
// coordinate passes 32 bits however long the pool.
inline bool make_pool_map(CUtensorMap *map, const void *base, int64_t blocks, int page_size, int dh, int page_box,
                          bool swizzle) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(dh), static_cast<cuuint64_t>(page_size), static_cast<cuuint64_t>(blocks)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(dh), static_cast<cuuint64_t>(dh) * page_size};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(dh), static_cast<cuuint32_t>(page_box), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE : (dh == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B),
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace eagle
