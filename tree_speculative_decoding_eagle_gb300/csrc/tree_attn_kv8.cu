// Stage 3 over the 8-bit paged cache: which kernel runs, and with what
// (tree_attn_kv8_kernel.cuh for many query rows a KV head, tree_attn_kv8_few.cu for
// few).
#include "tree_attn_kv8_kernel.cuh"

namespace eagle {

// tree_attn_kv8_few.cu
size_t attn_kv8_few_workspace_bytes(int B, int n, int Hq, int Hkv, int dh, int Lmax, int num_sms);
cudaError_t launch_tree_attn_kv8_few(Kv8Args a, const void *k_pages, const void *v_pages, int dh, void *ws, int num_sms,
                                     cudaStream_t st);

// Query rows of a KV head up to which the few-row kernel runs: its warp-level
// MMAs cost a row tile of 16 what the bytes cost at two tiles.  Measured (us,
// few-row kernel / this one): 20 rows, dh 64, 64 heads of U[1024, 4096] keys 25.1 /
// 25.6; 30 rows, dh 128, 320 such heads 138 / 112 (149 / 170 when the bound was set:
// at dh 128 with many heads it now belongs between 16 and 32).  With more row tiles
// the few-row kernel took 208 us at 51 rows, dh 128, 320 heads, against 127, and 145
// at 56 rows, dh 64, 256 heads of 4096 keys, against 94.
constexpr int kFewRows = 32;

size_t attn_kv8_workspace_bytes(int B, int n, int Hq, int Hkv, int dh, int Lmax, int num_sms) {
  if (n * (Hq / Hkv) <= kFewRows) return attn_kv8_few_workspace_bytes(B, n, Hq, Hkv, dh, Lmax, num_sms);
  const Kv8Plan p = kv8_plan(B, n, Hq, Hkv, dh, Lmax, num_sms);
  if (p.S <= 1) return 0;
  return static_cast<size_t>(B) * Hkv * p.mgroups * p.S * kv8_slot_rows(p, n * (Hq / Hkv)) * (dh + 2) * sizeof(float);
}

cudaError_t launch_tree_attn_kv8(const void *q, const uint8_t *k_pages, const uint8_t *v_pages, const float *k_scale,
                                 const float *v_scale, const int32_t *block_table, int max_pages, int page_size,
                                 int num_pages, const int32_t *kv_len, const void *k_tree, const void *v_tree,
                                 const uint64_t *mask, int B, int n, int Hq, int Hkv, int dh, float scale, void *out,
                                 float *lse, void *ws, int32_t *status, int num_sms, cudaStream_t st) {
  Kv8Args a;
  a.q = reinterpret_cast<const __nv_bfloat16 *>(q);
  a.k_tree = reinterpret_cast<const __nv_bfloat16 *>(k_tree);
  a.v_tree = reinterpret_cast<const __nv_bfloat16 *>(v_tree);
  a.k_scale = k_scale; a.v_scale = v_scale;
  a.block_table = block_table; a.kv_len = kv_len; a.mask = mask;
  a.B = B; a.n = n; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv; a.W = (n + 63) / 64;
  a.page_size = page_size; a.max_pages = max_pages; a.num_pages = num_pages;
  a.log_page = 0;
  while ((1 << a.log_page) < page_size) ++a.log_page;
  a.scale_log2 = scale * kLog2e;
  a.out = reinterpret_cast<__nv_bfloat16 *>(out);
  a.lse = lse; a.status = status;
  if (n * a.G <= kFewRows) return launch_tree_attn_kv8_few(a, k_pages, v_pages, dh, ws, num_sms, st);
  const Kv8Plan p = kv8_plan(B, n, Hq, Hkv, dh, max_pages * page_size, num_sms);
  return launch_kv8<false>(a, k_pages, v_pages, dh, p, ws, st);
}

}  // namespace eagle
