// Stage 3 over the 8-bit paged cache: tree-masked attention whose prefix keys
// and values are e4m3 numbers with a power-of-two scale for each page and head.
//
// One warp per (sequence, node, query head): the lanes share the head's
// columns, keys come one at a time, the softmax is the running one (maximum,
// sum, rescaled accumulator) in float32.
#include "kv8.cuh"

namespace eagle {

struct Kv8Args {
  const __nv_bfloat16 *q, *k_tree, *v_tree;
  const uint8_t *k_pages, *v_pages;
  const float *k_scale, *v_scale;
  const int32_t *block_table, *kv_len;
  const uint64_t *mask;
  int B, n, Hq, Hkv, G, W, log_page, max_pages, num_pages;
  float scale_log2;
  __nv_bfloat16 *out;
  float *lse;
  int32_t *status;
};

template <int DH>
__global__ void __launch_bounds__(128) tree_attn_kv8_row_kernel(Kv8Args a) {
  constexpr int C = DH / 32;  // columns a lane
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  pdl_wait();
  if (row >= static_cast<int64_t>(a.B) * a.n * a.Hq) return;
  const int h = static_cast<int>(row % a.Hq), i = static_cast<int>(row / a.Hq % a.n);
  const int b = static_cast<int>(row / a.Hq / a.n), g = h / a.G;
  const int P = 1 << a.log_page;
  const int L = static_cast<int>(min(static_cast<int64_t>(max(a.kv_len[b], 0)), static_cast<int64_t>(a.max_pages) << a.log_page));
  float q[C], o[C];
  for (int c = 0; c < C; ++c) {
    q[c] = __bfloat162float(a.q[row * DH + lane * C + c]) * a.scale_log2;
    o[c] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const auto take = [&](const float (&k)[C], const float (&v)[C]) {
    float s = 0.f;
    for (int c = 0; c < C; ++c) s = fmaf(q[c], k[c], s);
    s = warp_sum(s);
    const float mn = fmaxf(m, s), alpha = exp2f(m - mn), p = exp2f(s - mn);
    l = l * alpha + p;
    for (int c = 0; c < C; ++c) o[c] = fmaf(p, v[c], o[c] * alpha);
    m = mn;
  };
  for (int p0 = 0; p0 < L; p0 += P) {
    int page = a.block_table[static_cast<int64_t>(b) * a.max_pages + (p0 >> a.log_page)];
    if (page < 0 || page >= a.num_pages) {
      report(a.status, EAGLE_ERR_INVALID);
      page = 0;
    }
    const int64_t at = static_cast<int64_t>(page) * a.Hkv + g;
    const float ks = exponent_scale(scale_exponent(a.k_scale[at])), vs = exponent_scale(scale_exponent(a.v_scale[at]));
    const int64_t base = (at << a.log_page) * DH + lane * C;
    for (int r = 0; r < min(P, L - p0); ++r) {
      float k[C], v[C];
      for (int c = 0; c < C; ++c) {
        const uint32_t kc = e4m3_to_half2(a.k_pages[base + static_cast<int64_t>(r) * DH + c]);
        const uint32_t vc = e4m3_to_half2(a.v_pages[base + static_cast<int64_t>(r) * DH + c]);
        k[c] = __low2float(*reinterpret_cast<const __half2 *>(&kc)) * ks;
        v[c] = __low2float(*reinterpret_cast<const __half2 *>(&vc)) * vs;
      }
      take(k, v);
    }
  }
  const uint64_t *mrow = a.mask + (static_cast<int64_t>(b) * a.n + i) * a.W;
  for (int j = 0; j < a.n; ++j) {
    if (!((mrow[j >> 6] >> (j & 63)) & 1ull)) continue;
    const int64_t at = ((static_cast<int64_t>(b) * a.Hkv + g) * a.n + j) * DH + lane * C;
    float k[C], v[C];
    for (int c = 0; c < C; ++c) {
      k[c] = __bfloat162float(a.k_tree[at + c]);
      v[c] = __bfloat162float(a.v_tree[at + c]);
    }
    take(k, v);
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int c = 0; c < C; ++c) a.out[row * DH + lane * C + c] = __float2bfloat16(o[c] * inv);
  if (a.lse && lane == 0) a.lse[row] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

size_t attn_kv8_workspace_bytes(int, int, int, int, int, int, int) { return 0; }

cudaError_t launch_tree_attn_kv8(const void *q, const uint8_t *k_pages, const uint8_t *v_pages, const float *k_scale,
                                 const float *v_scale, const int32_t *block_table, int max_pages, int page_size,
                                 int num_pages, const int32_t *kv_len, const void *k_tree, const void *v_tree,
                                 const uint64_t *mask, int B, int n, int Hq, int Hkv, int dh, float scale, void *out,
                                 float *lse, void *, int32_t *status, int, cudaStream_t st) {
  int lp = 0;
  while ((1 << lp) < page_size) ++lp;
  Kv8Args a = {reinterpret_cast<const __nv_bfloat16 *>(q), reinterpret_cast<const __nv_bfloat16 *>(k_tree),
               reinterpret_cast<const __nv_bfloat16 *>(v_tree), k_pages, v_pages, k_scale, v_scale, block_table,
               kv_len, mask, B, n, Hq, Hkv, Hq / Hkv, (n + 63) / 64, lp, max_pages, num_pages, scale * kLog2e,
               reinterpret_cast<__nv_bfloat16 *>(out), lse, status};
  const int64_t rows = static_cast<int64_t>(B) * n * Hq;
  const dim3 grid(static_cast<unsigned>((rows + 3) / 4));
  return dh == 64 ? launch_chained(tree_attn_kv8_row_kernel<64>, grid, dim3(128), 0, st, a)
                  : launch_chained(tree_attn_kv8_row_kernel<128>, grid, dim3(128), 0, st, a);
}

}  // namespace eagle
