// C ABI of the library: argument validation, workspace sizing and dispatch
// to the stage kernels.  Every entry point returns an eagle_status and never
// throws, allocates or synchronises.
#include <cuda_runtime.h>

#include <limits>

#include "common.cuh"

namespace eagle {
// draft_topk.cu
size_t draft_workspace_bytes(int B, int D, int k, int V, int vec, int num_sms);
cudaError_t launch_draft_topk(const void *logits, int dtype, int B, int D, int k, int V, int64_t ld,
                              int32_t *tok, float *conf, float *stats, void *ws, int32_t *status,
                              int num_sms, cudaStream_t st);
// tree_build.cu
cudaError_t launch_tree_build(const int32_t *tok, const float *conf, int B, int D, int k, int m, int flags,
                              const int32_t *root_tok, int32_t *node_tok, int32_t *node_parent,
                              int32_t *node_depth, float *node_score, int32_t *node_src,
                              int32_t *node_row, uint64_t *mask, int32_t *status, cudaStream_t st);
cudaError_t launch_tree_mask(const int32_t *parent, int B, int n, uint64_t *mask, cudaStream_t st);
// verify_draft.cu
cudaError_t launch_verify_draft(const void *target, const void *draft, int dtype, int64_t ld_t, int64_t ld_d,
                                const int32_t *node_tok, const int32_t *node_parent, const int32_t *node_row,
                                int B, int m, int D, int k, int V, float temperature, const float *uniforms,
                                int32_t *accept_len, int32_t *path_nodes, int32_t *out_tokens, int32_t *status,
                                cudaStream_t st);
// tree_attn_tc.cu (paged prefix)
cudaError_t launch_tree_attn_tc_paged(const void *q, const void *k_pages, const void *v_pages,
                                      const int32_t *block_table, int max_pages, int page_size, int num_pages,
                                      const int32_t *kv_len, const void *k_tree, const void *v_tree,
                                      const uint64_t *mask, int B, int n, int Hq, int Hkv, int dh, float scale,
                                      void *out, float *lse, void *ws, int32_t *status, int num_sms,
                                      cudaStream_t st);
// kv_commit.cu
cudaError_t launch_kv_commit(const void *k_tree, const void *v_tree, int dtype, int B, int n, int Hkv, int dh,
                             const int32_t *accept_len, const int32_t *path_nodes, int D, void *k_cache,
                             void *v_cache, int Lmax, const int32_t *block_table, int max_pages, int page_size,
                             int num_pages, int32_t *kv_len, int32_t *slot_mapping, int32_t *status,
                             cudaStream_t st);
// static_tree.cu
cudaError_t launch_static_tree(const int32_t *tok, const float *conf, int B, int D, int k, const int32_t *parent,
                               const int32_t *rank, int n, const int32_t *root_tok, int32_t *node_tok,
                               int32_t *node_parent, int32_t *node_depth, float *node_score, int32_t *node_src,
                               int32_t *node_row, uint64_t *mask, int32_t *status, cudaStream_t st);
size_t tree_smem_bytes(int D, int k, int m, int flags);
// tree_attn_simt.cu / tree_attn_tc.cu
size_t attn_simt_workspace_bytes(int B, int n, int Hq, int dh, int Lmax, int num_sms);
cudaError_t launch_tree_attn_simt(const void *q, const void *k_cache, const void *v_cache,
                                  const int32_t *kv_len, const void *k_tree, const void *v_tree,
                                  const uint64_t *mask, int dtype, int B, int n, int Hq, int Hkv,
                                  int dh, int Lmax, float scale, void *out, float *lse, void *ws,
                                  int num_sms, cudaStream_t st);
size_t attn_tc_workspace_bytes(int B, int n, int Hq, int Hkv, int dh, int Lmax, int num_sms);
int attn_tc_kernel_count(int B, int n, int Hq, int Hkv, int dh, int Lmax, int num_sms);
cudaError_t launch_tree_attn_tc(const void *q, const void *k_cache, const void *v_cache, const int32_t *kv_len,
                                const void *k_tree, const void *v_tree, const uint64_t *mask, int B, int n,
                                int Hq, int Hkv, int dh, int Lmax, float scale, void *out, float *lse, void *ws,
                                int32_t *status, int num_sms, cudaStream_t st);
// qk_norm_rope.cu
cudaError_t launch_qk_norm_rope(const void *q, const void *k, const void *v, int dtype, int B, int n, int Hq, int Hkv,
                                int dh, int64_t ld_q, int64_t ld_k, int64_t ld_v, const void *q_weight,
                                const void *k_weight, float weight_offset, float eps, const double *inv_freq,
                                int rot_dim, int interleaved, float factor, const int32_t *pos_base,
                                const int32_t *pos_off, int shift, void *q_out, void *k_tree, void *v_tree, int num_sms,
                                cudaStream_t st);
// kv8_bounds.cu
cudaError_t launch_kv8_bounds(const uint8_t *k_pages, const int32_t *block_table, int max_pages, int page_size,
                              int num_pages, const int32_t *from_len, const int32_t *kv_len, int B, int Hkv, int dh,
                              uint8_t *bounds, int32_t *status, int num_sms, cudaStream_t st);
// kv8_select.cu
size_t kv8_select_workspace_bytes(int B, int n, int Hkv, int max_pages);
cudaError_t launch_kv8_select(const void *q, const uint8_t *bounds, const float *k_scale, const int32_t *block_table,
                              int max_pages, int page_size, int num_pages, const int32_t *kv_len, int B, int n, int Hq,
                              int Hkv, int dh, int top, int first, int last, int32_t *sel, float *score, void *ws,
                              int32_t *status, int num_sms, cudaStream_t st);
// tree_attn_kv8_pages.cu
size_t attn_kv8_pages_workspace_bytes(int B, int n, int Hq, int Hkv, int dh, int top, int max_pages, int page_size, int num_sms);
cudaError_t launch_tree_attn_kv8_pages(const void *q, const uint8_t *k_pages, const uint8_t *v_pages, const float *k_scale,
                                       const float *v_scale, const int32_t *block_table, int max_pages, int page_size,
                                       int num_pages, const int32_t *kv_len, const void *k_tree, const void *v_tree,
                                       const uint64_t *mask, const int32_t *sel, int top, int B, int n, int Hq, int Hkv,
                                       int dh, float scale, void *out, float *lse, void *ws, int32_t *status, int num_sms,
                                       cudaStream_t st);
// verify.cu
size_t verify_workspace_bytes(int B, int m, int V);
cudaError_t launch_verify(const void *target, int dtype, int64_t ld, const int32_t *node_tok,
                          const int32_t *node_parent, int B, int m, int D, int V, int mode,
                          float temperature, const float *u, int32_t *accept_len,
                          int32_t *path_nodes, int32_t *out_tokens, int32_t *status, void *ws,
                          int num_sms, cudaStream_t st);

// page_map.cu
cudaError_t launch_page_map(const int32_t *kv_len, const int32_t *new_len, int B, int page_size, int max_pages,
                            int num_pages, int32_t *block_table, int32_t *page_count, const int32_t *free_pages,
                            int32_t *free_count, int32_t *slot_map, int T, int32_t *new_start, int32_t *granted,
                            int32_t *status, cudaStream_t st);
cudaError_t launch_page_release(const int32_t *keep_len, int B, int page_size, int max_pages, int num_pages,
                                int32_t *block_table, int32_t *page_count, int32_t *free_pages, int32_t *free_count,
                                int32_t *status, cudaStream_t st);
// rope.cu
cudaError_t launch_rope(const void *q, const void *k, const void *v, int dtype, int B, int n, int Hq, int Hkv, int dh,
                        int64_t ld_q, int64_t ld_k, int64_t ld_v, const double *inv_freq, int rot_dim,
                        int interleaved, float factor, const int32_t *pos_base, const int32_t *pos_off, int shift,
                        void *q_out, void *k_tree, void *v_tree, cudaStream_t st);
void rope_freqs(int rot_dim, double theta, int kind, double stretch, int orig_len, double low, double high,
                double *inv_freq, float *factor);
// kv8_write.cu
cudaError_t launch_kv8_append(const void *k, const void *v, int dtype, int T, int Hkv, int dh, int64_t token_stride,
                              int64_t head_stride, const int32_t *slot_map, uint8_t *k_pages, uint8_t *v_pages,
                              float *k_scale, float *v_scale, int page_size, int num_pages, int32_t *status,
                              int num_sms, cudaStream_t st);
cudaError_t launch_kv8_commit(const void *k_tree, const void *v_tree, int dtype, int B, int n, int Hkv, int dh, bool root,
                              const int32_t *accept_len, const int32_t *path_nodes, int D, uint8_t *k_pages,
                              uint8_t *v_pages, float *k_scale, float *v_scale, const int32_t *block_table,
                              int max_pages, int page_size, int num_pages, int32_t *kv_len, int32_t *slot_mapping,
                              int32_t *status, cudaStream_t st);
// tree_attn_kv8.cu
size_t attn_kv8_workspace_bytes(int B, int n, int Hq, int Hkv, int dh, int Lmax, int num_sms);
cudaError_t launch_tree_attn_kv8(const void *q, const uint8_t *k_pages, const uint8_t *v_pages, const float *k_scale,
                                 const float *v_scale, const int32_t *block_table, int max_pages, int page_size,
                                 int num_pages, const int32_t *kv_len, const void *k_tree, const void *v_tree,
                                 const uint64_t *mask, int B, int n, int Hq, int Hkv, int dh, float scale, void *out,
                                 float *lse, void *ws, int32_t *status, int num_sms, cudaStream_t st);

// SM count of the current device (queried once per device).
int current_num_sms() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (cached[dev] == 0) {
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || sms <= 0)
      sms = 148;
    cached[dev] = sms;
  }
  return cached[dev];
}

static inline int elem_size(int dtype) { return dtype == EAGLE_BF16 ? 2 : 4; }
static inline bool valid_dtype(int dtype) { return dtype == EAGLE_F32 || dtype == EAGLE_BF16; }
static inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
static inline int from_cuda(cudaError_t e) { return e == cudaSuccess ? EAGLE_OK : EAGLE_ERR_CUDA; }

}  // namespace eagle

using namespace eagle;

extern "C" {

const char *eagle_status_string(int code) {
  switch (code) {
    case EAGLE_OK: return "ok";
    case EAGLE_ERR_INVALID: return "invalid argument";
    case EAGLE_ERR_UNSUPPORTED: return "unsupported configuration";
    case EAGLE_ERR_CUDA: return "CUDA error";
    case EAGLE_ERR_WORKSPACE: return "workspace too small";
    case EAGLE_ERR_TIMEOUT: return "device wait timed out";
    case EAGLE_ERR_PAGES: return "too few free pages";
    default: return "unknown status";
  }
}

int eagle_version(void) { return 100; }

size_t eagle_draft_topk_workspace_size(int B, int D, int k, int V) {
  if (B < 1 || D < 1 || k < 1 || V < 1) return 0;
  // the split count depends on the vector width; take the larger of the two
  size_t a = draft_workspace_bytes(B, D, k, V, 8, current_num_sms());
  size_t b = draft_workspace_bytes(B, D, k, V, 4, current_num_sms());
  return a > b ? a : b;
}

int eagle_draft_topk(const void *logits, int dtype, int B, int D, int k, int V, int64_t ld,
                     int32_t *tok, float *conf, float *stats, int32_t *status, void *workspace,
                     size_t workspace_bytes, eagle_stream_t stream) {
  if (!logits || !tok || !conf || !valid_dtype(dtype)) return EAGLE_ERR_INVALID;
  if (B < 1 || D < 1 || k < 1 || k > 32 || V < 1 || k > V || ld < V) return EAGLE_ERR_INVALID;
  const int es = elem_size(dtype);
  if ((static_cast<int64_t>(V) * es) % 16 || (ld * es) % 16 || !aligned16(logits)) return EAGLE_ERR_INVALID;
  if (static_cast<int64_t>(B) * (1 + (D - 1) * k) > 65535) return EAGLE_ERR_UNSUPPORTED;
  const int sms = current_num_sms();
  const size_t need = draft_workspace_bytes(B, D, k, V, 16 / es, sms);
  if (workspace_bytes < need || (need && !workspace)) return EAGLE_ERR_WORKSPACE;
  return from_cuda(launch_draft_topk(logits, dtype, B, D, k, V, ld, tok, conf, stats, workspace,
                                     status, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int eagle_tree_build_variant(const int32_t *tok, const float *conf, int B, int D, int k, int m, int flags,
                             const int32_t *root_tok, int32_t *node_tok, int32_t *node_parent,
                             int32_t *node_depth, float *node_score, int32_t *node_src, int32_t *node_row,
                             uint64_t *mask, int32_t *status, eagle_stream_t stream) {
  if (!tok || !conf || !node_tok || !node_parent) return EAGLE_ERR_INVALID;
  if (B < 1 || D < 1 || k < 1 || k > 32 || m < 1) return EAGLE_ERR_INVALID;
  if (flags & ~(EAGLE_TREE_CONFIDENCE_ONLY | EAGLE_TREE_NO_RERANK)) return EAGLE_ERR_INVALID;
  const int64_t NC = k + static_cast<int64_t>(D - 1) * k * k;
  if (NC > 4095 || m > NC) return EAGLE_ERR_INVALID;
  if ((flags & EAGLE_TREE_NO_RERANK) && m > static_cast<int64_t>(D) * k) return EAGLE_ERR_INVALID;
  if (tree_smem_bytes(D, k, m, flags) > 227 * 1024) return EAGLE_ERR_UNSUPPORTED;  // one CTA's shared memory
  return from_cuda(launch_tree_build(tok, conf, B, D, k, m, flags, root_tok, node_tok, node_parent,
                                     node_depth, node_score, node_src, node_row, mask, status,
                                     reinterpret_cast<cudaStream_t>(stream)));
}

int eagle_tree_build(const int32_t *tok, const float *conf, int B, int D, int k, int m,
                     const int32_t *root_tok, int32_t *node_tok, int32_t *node_parent,
                     int32_t *node_depth, float *node_score, int32_t *node_src, int32_t *node_row,
                     uint64_t *mask, int32_t *status, eagle_stream_t stream) {
  return eagle_tree_build_variant(tok, conf, B, D, k, m, 0, root_tok, node_tok, node_parent, node_depth,
                                  node_score, node_src, node_row, mask, status, stream);
}

int eagle_static_tree(const int32_t *tok, const float *conf, int B, int D, int k, const int32_t *tree_parent,
                      const int32_t *tree_rank, int n, const int32_t *root_tok, int32_t *node_tok,
                      int32_t *node_parent, int32_t *node_depth, float *node_score, int32_t *node_src,
                      int32_t *node_row, uint64_t *mask, int32_t *status, eagle_stream_t stream) {
  if (!tok || !conf || !tree_parent || !tree_rank || !node_tok || !node_parent) return EAGLE_ERR_INVALID;
  if (B < 1 || D < 1 || D > 32 || k < 1 || k > 32 || n < 1 || n > 1024) return EAGLE_ERR_INVALID;
  return from_cuda(launch_static_tree(tok, conf, B, D, k, tree_parent, tree_rank, n, root_tok, node_tok,
                                      node_parent, node_depth, node_score, node_src, node_row, mask, status,
                                      reinterpret_cast<cudaStream_t>(stream)));
}

int eagle_tree_mask(const int32_t *node_parent, int B, int n, uint64_t *mask, eagle_stream_t stream) {
  if (!node_parent || !mask || B < 1 || n < 1 || n > 4096) return EAGLE_ERR_INVALID;
  return from_cuda(launch_tree_mask(node_parent, B, n, mask, reinterpret_cast<cudaStream_t>(stream)));
}

size_t eagle_tree_attn_workspace_size(int dtype, int B, int n, int Hq, int Hkv, int dh, int Lmax) {
  if (B < 1 || n < 1 || Hq < 1 || Hkv < 1 || dh < 1 || Lmax < 0) return 0;
  if (dtype == EAGLE_BF16) return attn_tc_workspace_bytes(B, n, Hq, Hkv, dh, Lmax, current_num_sms());
  return attn_simt_workspace_bytes(B, n, Hq, dh, Lmax, current_num_sms());
}

int eagle_tree_attn_kernel_count(int dtype, int B, int n, int Hq, int Hkv, int dh, int Lmax) {
  if (!valid_dtype(dtype) || B < 1 || n < 1 || Hq < 1 || Hkv < 1 || dh < 1 || Lmax < 0) return 0;
  if (dtype == EAGLE_BF16) return attn_tc_kernel_count(B, n, Hq, Hkv, dh, Lmax, current_num_sms());
  // fp32: a split prefix adds the combine kernel (it asks for a workspace)
  return attn_simt_workspace_bytes(B, n, Hq, dh, Lmax, current_num_sms()) > 0 ? 2 : 1;
}

int eagle_tree_attn(const void *q, const void *k_cache, const void *v_cache, const int32_t *kv_len,
                    const void *k_tree, const void *v_tree, const uint64_t *mask, int dtype, int B,
                    int n, int Hq, int Hkv, int dh, int Lmax, float scale, void *out, float *lse,
                    int32_t *status, void *workspace, size_t workspace_bytes, eagle_stream_t stream) {
  if (!q || !k_cache || !v_cache || !kv_len || !k_tree || !v_tree || !mask || !out) return EAGLE_ERR_INVALID;
  if (!valid_dtype(dtype) || B < 1 || n < 1 || n > 4096 || Hq < 1 || Hkv < 1 || Hq % Hkv || Lmax < 0)
    return EAGLE_ERR_INVALID;
  if (dh != 64 && dh != 128) return EAGLE_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(B) * Hkv > 65535) return EAGLE_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_tree) ||
      !aligned16(v_tree) || !aligned16(out))
    return EAGLE_ERR_INVALID;
  const int sms = current_num_sms();
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == EAGLE_BF16) {
    const size_t need = attn_tc_workspace_bytes(B, n, Hq, Hkv, dh, Lmax, sms);
    if (workspace_bytes < need || (need && !workspace)) return EAGLE_ERR_WORKSPACE;
    return from_cuda(launch_tree_attn_tc(q, k_cache, v_cache, kv_len, k_tree, v_tree, mask, B, n, Hq, Hkv, dh,
                                         Lmax, scale, out, lse, workspace, status, sms, st));
  }
  const size_t need = attn_simt_workspace_bytes(B, n, Hq, dh, Lmax, sms);
  if (workspace_bytes < need || (need && !workspace)) return EAGLE_ERR_WORKSPACE;
  return from_cuda(launch_tree_attn_simt(q, k_cache, v_cache, kv_len, k_tree, v_tree, mask, dtype, B, n, Hq,
                                         Hkv, dh, Lmax, scale, out, lse, workspace, sms, st));
}

static bool valid_pages(int max_pages, int page_size, int num_pages) {
  return max_pages >= 1 && num_pages >= 1 && page_size >= 16 && page_size <= 4096 &&
         (page_size & (page_size - 1)) == 0 && static_cast<int64_t>(max_pages) * page_size <= (1 << 24);
}

size_t eagle_tree_attn_paged_workspace_size(int dtype, int B, int n, int Hq, int Hkv, int dh, int max_pages,
                                            int page_size) {
  if (dtype != EAGLE_BF16 || B < 1 || n < 1 || Hq < 1 || Hkv < 1 || dh < 1 || max_pages < 1 || page_size < 1)
    return 0;
  return attn_tc_workspace_bytes(B, n, Hq, Hkv, dh, max_pages * page_size, current_num_sms());
}

int eagle_tree_attn_paged(const void *q, const void *k_pages, const void *v_pages, const int32_t *block_table,
                          int max_pages, int page_size, int num_pages, const int32_t *kv_len, const void *k_tree,
                          const void *v_tree, const uint64_t *mask, int dtype, int B, int n, int Hq, int Hkv,
                          int dh, float scale, void *out, float *lse, int32_t *status, void *workspace,
                          size_t workspace_bytes, eagle_stream_t stream) {
  if (!q || !k_pages || !v_pages || !block_table || !kv_len || !k_tree || !v_tree || !mask || !out)
    return EAGLE_ERR_INVALID;
  if (!valid_dtype(dtype) || B < 1 || n < 1 || n > 4096 || Hq < 1 || Hkv < 1 || Hq % Hkv ||
      !valid_pages(max_pages, page_size, num_pages))
    return EAGLE_ERR_INVALID;
  if (dtype != EAGLE_BF16 || (dh != 64 && dh != 128)) return EAGLE_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(B) * Hkv > 65535) return EAGLE_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_tree) || !aligned16(v_tree) ||
      !aligned16(out))
    return EAGLE_ERR_INVALID;
  const int sms = current_num_sms();
  const size_t need = attn_tc_workspace_bytes(B, n, Hq, Hkv, dh, max_pages * page_size, sms);
  if (workspace_bytes < need || (need && !workspace)) return EAGLE_ERR_WORKSPACE;
  return from_cuda(launch_tree_attn_tc_paged(q, k_pages, v_pages, block_table, max_pages, page_size, num_pages,
                                             kv_len, k_tree, v_tree, mask, B, n, Hq, Hkv, dh, scale, out, lse,
                                             workspace, status, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int eagle_kv_commit(const void *k_tree, const void *v_tree, int dtype, int B, int n, int Hkv, int dh,
                    const int32_t *accept_len, const int32_t *path_nodes, int D, void *k_cache, void *v_cache,
                    int Lmax, const int32_t *block_table, int max_pages, int page_size, int num_pages,
                    int32_t *kv_len, int32_t *slot_mapping, int32_t *status, eagle_stream_t stream) {
  if (!k_tree || !v_tree || !accept_len || !path_nodes || !k_cache || !v_cache || !kv_len) return EAGLE_ERR_INVALID;
  if (!valid_dtype(dtype) || B < 1 || n < 1 || n > 4096 || Hkv < 1 || dh < 1 || D < 1 || D > 64)
    return EAGLE_ERR_INVALID;
  if ((dh * elem_size(dtype)) % 16) return EAGLE_ERR_INVALID;
  if (block_table ? !valid_pages(max_pages, page_size, num_pages) : Lmax < 1) return EAGLE_ERR_INVALID;
  if (!aligned16(k_tree) || !aligned16(v_tree) || !aligned16(k_cache) || !aligned16(v_cache))
    return EAGLE_ERR_INVALID;
  return from_cuda(launch_kv_commit(k_tree, v_tree, dtype, B, n, Hkv, dh, accept_len, path_nodes, D, k_cache,
                                    v_cache, Lmax, block_table, max_pages, page_size, num_pages, kv_len,
                                    slot_mapping, status, reinterpret_cast<cudaStream_t>(stream)));
}

size_t eagle_verify_workspace_size(int B, int m, int V) {
  if (B < 1 || m < 0 || V < 1) return 0;
  return verify_workspace_bytes(B, m, V);
}

int eagle_verify(const void *target, int dtype, int64_t ld, const int32_t *node_tok,
                 const int32_t *node_parent, int B, int m, int D, int V, int mode, float temperature,
                 const float *uniforms, int32_t *accept_len, int32_t *path_nodes,
                 int32_t *out_tokens, int32_t *status, void *workspace, size_t workspace_bytes,
                 eagle_stream_t stream) {
  if (!target || !node_tok || !node_parent || !accept_len || !path_nodes || !out_tokens)
    return EAGLE_ERR_INVALID;
  if (!valid_dtype(dtype) || B < 1 || m < 0 || m + 1 > 4096 || D < 1 || V < 1 || ld < V)
    return EAGLE_ERR_INVALID;
  if (mode != EAGLE_GREEDY && mode != EAGLE_SAMPLE) return EAGLE_ERR_INVALID;
  if (mode == EAGLE_SAMPLE && (!uniforms || !(temperature > 0.f))) return EAGLE_ERR_INVALID;
  const int es = elem_size(dtype);
  if ((static_cast<int64_t>(V) * es) % 16 || (ld * es) % 16 || !aligned16(target)) return EAGLE_ERR_INVALID;
  const size_t need = verify_workspace_bytes(B, m, V);
  if (workspace_bytes < need || !workspace) return EAGLE_ERR_WORKSPACE;
  return from_cuda(launch_verify(target, dtype, ld, node_tok, node_parent, B, m, D, V, mode,
                                 temperature, uniforms, accept_len, path_nodes, out_tokens, status,
                                 workspace, current_num_sms(), reinterpret_cast<cudaStream_t>(stream)));
}

int eagle_verify_draft(const void *target, const void *draft, int dtype, int64_t ld_t, int64_t ld_d,
                       const int32_t *node_tok, const int32_t *node_parent, const int32_t *node_row, int B,
                       int m, int D, int k, int V, float temperature, const float *uniforms,
                       int32_t *accept_len, int32_t *path_nodes, int32_t *out_tokens, int32_t *status,
                       eagle_stream_t stream) {
  if (!target || !draft || !node_tok || !node_parent || !node_row || !uniforms || !accept_len || !path_nodes ||
      !out_tokens)
    return EAGLE_ERR_INVALID;
  if (!valid_dtype(dtype) || B < 1 || m < 0 || m + 1 > 4096 || D < 1 || k < 1 || k > 32 || V < 1)
    return EAGLE_ERR_INVALID;
  if (ld_t < V || ld_d < V || !(temperature > 0.f)) return EAGLE_ERR_INVALID;
  const int es = elem_size(dtype);
  if ((static_cast<int64_t>(V) * es) % 16 || (ld_t * es) % 16 || (ld_d * es) % 16 || !aligned16(target) ||
      !aligned16(draft))
    return EAGLE_ERR_INVALID;
  if (B > 65535) return EAGLE_ERR_UNSUPPORTED;  // sequences index the grid's y dimension
  return from_cuda(launch_verify_draft(target, draft, dtype, ld_t, ld_d, node_tok, node_parent, node_row, B, m,
                                       D, k, V, temperature, uniforms, accept_len, path_nodes, out_tokens, status,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

constexpr int kMaxTokens = 1 << 30;  // of one call: token indexes stay clear of 2^31

// Page pools addressed by 32-bit slots.
static bool valid_slots(int max_pages, int page_size, int num_pages) {
  return valid_pages(max_pages, page_size, num_pages) && static_cast<int64_t>(num_pages) * page_size <= INT32_MAX;
}

static int map_pages(const int32_t *kv_len, const int32_t *new_len, int B, int page_size, int max_pages, int num_pages,
                     int32_t *block_table, int32_t *page_count, const int32_t *free_pages, int32_t *free_count,
                     int32_t *slot_map, int T, int32_t *new_start, int32_t *granted, int32_t *status,
                     eagle_stream_t stream) {
  if (!kv_len || !new_len || !block_table || !page_count || !free_pages || !free_count) return EAGLE_ERR_INVALID;
  if (B < 1 || T < 0 || T > kMaxTokens || (!slot_map && T) || !valid_slots(max_pages, page_size, num_pages))
    return EAGLE_ERR_INVALID;
  if (B > 4096) return EAGLE_ERR_UNSUPPORTED;  // one CTA's shared memory holds every request's sums
  return from_cuda(launch_page_map(kv_len, new_len, B, page_size, max_pages, num_pages, block_table, page_count,
                                   free_pages, free_count, slot_map, T, new_start, granted, status,
                                   reinterpret_cast<cudaStream_t>(stream)));
}

int eagle_page_map(const int32_t *kv_len, const int32_t *new_len, int B, int page_size, int max_pages, int num_pages,
                   int32_t *block_table, int32_t *page_count, const int32_t *free_pages, int32_t *free_count,
                   int32_t *slot_map, int T, int32_t *new_start, int32_t *status, eagle_stream_t stream) {
  return map_pages(kv_len, new_len, B, page_size, max_pages, num_pages, block_table, page_count, free_pages, free_count,
                   slot_map, T, new_start, nullptr, status, stream);
}

int eagle_page_reserve(const int32_t *kv_len, const int32_t *new_len, int B, int page_size, int max_pages,
                       int num_pages, int32_t *block_table, int32_t *page_count, const int32_t *free_pages,
                       int32_t *free_count, int32_t *slot_map, int T, int32_t *new_start, int32_t *granted,
                       int32_t *status, eagle_stream_t stream) {
  if (!granted) return EAGLE_ERR_INVALID;
  return map_pages(kv_len, new_len, B, page_size, max_pages, num_pages, block_table, page_count, free_pages, free_count,
                   slot_map, T, new_start, granted, status, stream);
}

int eagle_page_release(const int32_t *keep_len, int B, int page_size, int max_pages, int num_pages,
                       int32_t *block_table, int32_t *page_count, int32_t *free_pages, int32_t *free_count,
                       int32_t *status, eagle_stream_t stream) {
  if (!keep_len || !block_table || !page_count || !free_pages || !free_count) return EAGLE_ERR_INVALID;
  if (B < 1 || !valid_slots(max_pages, page_size, num_pages)) return EAGLE_ERR_INVALID;
  if (B > 4096) return EAGLE_ERR_UNSUPPORTED;
  return from_cuda(launch_page_release(keep_len, B, page_size, max_pages, num_pages, block_table, page_count,
                                       free_pages, free_count, status, reinterpret_cast<cudaStream_t>(stream)));
}

// Shared by eagle_rope and eagle_qk_norm_rope.
static int check_rope(const void *q, const void *k, const void *v, int dtype, int B, int n, int Hq, int Hkv, int dh,
                      int64_t ld_q, int64_t ld_k, int64_t ld_v, const double *inv_freq, int rot_dim, const void *q_out,
                      const void *k_tree, const void *v_tree) {
  if (!q || !k || !inv_freq || !q_out || !k_tree || (v && !v_tree) || !valid_dtype(dtype)) return EAGLE_ERR_INVALID;
  if (B < 1 || n < 1 || Hq < 1 || Hkv < 1 || dh < 1 || rot_dim < 2 || rot_dim % 2 || rot_dim > dh)
    return EAGLE_ERR_INVALID;
  if (static_cast<int64_t>(B) * n > (1 << 24) || dh > 512 || static_cast<int64_t>(Hq) + 2ll * Hkv > (1 << 16))
    return EAGLE_ERR_UNSUPPORTED;
  const int es = elem_size(dtype);
  if ((dh * es) % 16 || (ld_q * es) % 16 || (ld_k * es) % 16 || (v && (ld_v * es) % 16)) return EAGLE_ERR_INVALID;
  if (ld_q < static_cast<int64_t>(Hq) * dh || ld_k < static_cast<int64_t>(Hkv) * dh ||
      (v && ld_v < static_cast<int64_t>(Hkv) * dh))
    return EAGLE_ERR_INVALID;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_tree) ||
      !aligned16(v_tree))
    return EAGLE_ERR_INVALID;
  if (q_out == q && ld_q != static_cast<int64_t>(Hq) * dh) return EAGLE_ERR_INVALID;
  return EAGLE_OK;
}

int eagle_rope(const void *q, const void *k, const void *v, int dtype, int B, int n, int Hq, int Hkv, int dh,
               int64_t ld_q, int64_t ld_k, int64_t ld_v, const double *inv_freq, int rot_dim, int interleaved,
               float factor, const int32_t *pos_base, const int32_t *pos_off, int shift, void *q_out, void *k_tree,
               void *v_tree, eagle_stream_t stream) {
  const int rc = check_rope(q, k, v, dtype, B, n, Hq, Hkv, dh, ld_q, ld_k, ld_v, inv_freq, rot_dim, q_out, k_tree, v_tree);
  if (rc != EAGLE_OK) return rc;
  return from_cuda(launch_rope(q, k, v, dtype, B, n, Hq, Hkv, dh, ld_q, ld_k, ld_v, inv_freq, rot_dim, interleaved,
                               factor, pos_base, pos_off, shift, q_out, k_tree, v_tree,
                               reinterpret_cast<cudaStream_t>(stream)));
}

int eagle_qk_norm_rope(const void *q, const void *k, const void *v, int dtype, int B, int n, int Hq, int Hkv, int dh,
                       int64_t ld_q, int64_t ld_k, int64_t ld_v, const void *q_weight, const void *k_weight,
                       float weight_offset, float eps, const double *inv_freq, int rot_dim, int interleaved,
                       float factor, const int32_t *pos_base, const int32_t *pos_off, int shift, void *q_out,
                       void *k_tree, void *v_tree, eagle_stream_t stream) {
  const int rc = check_rope(q, k, v, dtype, B, n, Hq, Hkv, dh, ld_q, ld_k, ld_v, inv_freq, rot_dim, q_out, k_tree, v_tree);
  if (rc != EAGLE_OK) return rc;
  constexpr float kMax = std::numeric_limits<float>::max();  // no NaN, no infinity
  if (!(eps > 0.f && eps <= kMax) || !(weight_offset >= -kMax && weight_offset <= kMax)) return EAGLE_ERR_INVALID;
  if (!aligned16(q_weight) || !aligned16(k_weight)) return EAGLE_ERR_INVALID;
  return from_cuda(launch_qk_norm_rope(q, k, v, dtype, B, n, Hq, Hkv, dh, ld_q, ld_k, ld_v, q_weight, k_weight,
                                       weight_offset, eps, inv_freq, rot_dim, interleaved, factor, pos_base, pos_off,
                                       shift, q_out, k_tree, v_tree, current_num_sms(),
                                       reinterpret_cast<cudaStream_t>(stream)));
}

int eagle_rope_freqs(int rot_dim, double theta, int kind, double stretch, int orig_len, double low, double high,
                     double *inv_freq, float *factor) {
  constexpr double kMax = std::numeric_limits<double>::max();  // no NaN, no infinity
  if (!inv_freq || rot_dim < 2 || rot_dim % 2 || !(theta > 1.0 && theta <= kMax) || !(stretch >= 1.0 && stretch <= kMax))
    return EAGLE_ERR_INVALID;
  if (kind < EAGLE_ROPE_PLAIN || kind > EAGLE_ROPE_YARN) return EAGLE_ERR_INVALID;
  if (kind >= EAGLE_ROPE_BANDS && (orig_len < 1 || !(low > 0.0) || !(high > low && high <= kMax))) return EAGLE_ERR_INVALID;
  rope_freqs(rot_dim, theta, kind, stretch, orig_len, low, high, inv_freq, factor);
  return EAGLE_OK;
}

int eagle_kv8_append(const void *k, const void *v, int dtype, int T, int Hkv, int dh, int64_t token_stride,
                     int64_t head_stride, const int32_t *slot_map, uint8_t *k_pages, uint8_t *v_pages,
                     float *k_scale, float *v_scale, int page_size, int num_pages, int32_t *status,
                     eagle_stream_t stream) {
  if (!valid_dtype(dtype) || T < 0 || T > kMaxTokens || Hkv < 1 || dh < 16 || dh % 16 || dh > 512 || token_stride < 0 || head_stride < 0)
    return EAGLE_ERR_INVALID;
  if (!valid_slots(1, page_size, num_pages)) return EAGLE_ERR_INVALID;
  if (Hkv > 32767) return EAGLE_ERR_UNSUPPORTED;
  if (T == 0) return EAGLE_OK;
  if (!k || !v || !slot_map || !k_pages || !v_pages || !k_scale || !v_scale) return EAGLE_ERR_INVALID;
  const int es = elem_size(dtype);
  if ((token_stride * es) % 16 || (head_stride * es) % 16) return EAGLE_ERR_INVALID;
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_pages) || !aligned16(v_pages)) return EAGLE_ERR_INVALID;
  return from_cuda(launch_kv8_append(k, v, dtype, T, Hkv, dh, token_stride, head_stride, slot_map, k_pages, v_pages,
                                     k_scale, v_scale, page_size, num_pages, status, current_num_sms(),
                                     reinterpret_cast<cudaStream_t>(stream)));
}

static int kv8_commit(bool root, const void *k_tree, const void *v_tree, int dtype, int B, int n, int Hkv, int dh,
                      const int32_t *accept_len, const int32_t *path_nodes, int D, uint8_t *k_pages, uint8_t *v_pages,
                      float *k_scale, float *v_scale, const int32_t *block_table, int max_pages, int page_size,
                      int num_pages, int32_t *kv_len, int32_t *slot_mapping, int32_t *status, eagle_stream_t stream) {
  if (!k_tree || !v_tree || !accept_len || !path_nodes || !k_pages || !v_pages || !k_scale || !v_scale ||
      !block_table || !kv_len)
    return EAGLE_ERR_INVALID;
  if (!valid_dtype(dtype) || B < 1 || n < 1 || n > 4096 || Hkv < 1 || dh < 16 || dh % 16 || dh > 512 || D < 1 || D > 64)
    return EAGLE_ERR_INVALID;
  if (!valid_slots(max_pages, page_size, num_pages)) return EAGLE_ERR_INVALID;
  if (Hkv > 32767 || B > 65535) return EAGLE_ERR_UNSUPPORTED;
  if (!aligned16(k_tree) || !aligned16(v_tree) || !aligned16(k_pages) || !aligned16(v_pages))
    return EAGLE_ERR_INVALID;
  return from_cuda(launch_kv8_commit(k_tree, v_tree, dtype, B, n, Hkv, dh, root, accept_len, path_nodes, D, k_pages,
                                     v_pages, k_scale, v_scale, block_table, max_pages, page_size, num_pages, kv_len,
                                     slot_mapping, status, reinterpret_cast<cudaStream_t>(stream)));
}

int eagle_kv8_commit(const void *k_tree, const void *v_tree, int dtype, int B, int n, int Hkv, int dh,
                     const int32_t *accept_len, const int32_t *path_nodes, int D, uint8_t *k_pages, uint8_t *v_pages,
                     float *k_scale, float *v_scale, const int32_t *block_table, int max_pages, int page_size,
                     int num_pages, int32_t *kv_len, int32_t *slot_mapping, int32_t *status, eagle_stream_t stream) {
  return kv8_commit(false, k_tree, v_tree, dtype, B, n, Hkv, dh, accept_len, path_nodes, D, k_pages, v_pages, k_scale,
                    v_scale, block_table, max_pages, page_size, num_pages, kv_len, slot_mapping, status, stream);
}

int eagle_kv8_commit_root(const void *k_tree, const void *v_tree, int dtype, int B, int n, int Hkv, int dh,
                          const int32_t *accept_len, const int32_t *path_nodes, int D, uint8_t *k_pages,
                          uint8_t *v_pages, float *k_scale, float *v_scale, const int32_t *block_table, int max_pages,
                          int page_size, int num_pages, int32_t *kv_len, int32_t *slot_mapping, int32_t *status,
                          eagle_stream_t stream) {
  return kv8_commit(true, k_tree, v_tree, dtype, B, n, Hkv, dh, accept_len, path_nodes, D, k_pages, v_pages, k_scale,
                    v_scale, block_table, max_pages, page_size, num_pages, kv_len, slot_mapping, status, stream);
}

// Query rows of a KV head: their M-groups are a grid dimension, their number an int.
static bool valid_query_rows(int n, int Hq, int Hkv) { return static_cast<int64_t>(n) * (Hq / Hkv) <= (1 << 23); }

size_t eagle_tree_attn_kv8_workspace_size(int dtype, int B, int n, int Hq, int Hkv, int dh, int max_pages,
                                          int page_size) {
  if (dtype != EAGLE_BF16 || B < 1 || n < 1 || n > 4096 || Hq < 1 || Hkv < 1 || Hq % Hkv || (dh != 64 && dh != 128) ||
      !valid_pages(max_pages, page_size, 1) || !valid_query_rows(n, Hq, Hkv))
    return 0;
  return attn_kv8_workspace_bytes(B, n, Hq, Hkv, dh, max_pages * page_size, current_num_sms());
}

int eagle_tree_attn_kv8(const void *q, const uint8_t *k_pages, const uint8_t *v_pages, const float *k_scale,
                        const float *v_scale, const int32_t *block_table, int max_pages, int page_size,
                        int num_pages, const int32_t *kv_len, const void *k_tree, const void *v_tree,
                        const uint64_t *mask, int dtype, int B, int n, int Hq, int Hkv, int dh, float scale,
                        void *out, float *lse, int32_t *status, void *workspace, size_t workspace_bytes,
                        eagle_stream_t stream) {
  if (!q || !k_pages || !v_pages || !k_scale || !v_scale || !block_table || !kv_len || !k_tree || !v_tree || !mask ||
      !out)
    return EAGLE_ERR_INVALID;
  if (!valid_dtype(dtype) || B < 1 || n < 1 || n > 4096 || Hq < 1 || Hkv < 1 || Hq % Hkv || !(scale > 0.f) ||
      !valid_pages(max_pages, page_size, num_pages))
    return EAGLE_ERR_INVALID;
  if (dtype != EAGLE_BF16 || (dh != 64 && dh != 128)) return EAGLE_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(B) * Hkv > 65535 || static_cast<int64_t>(num_pages) * Hkv > INT32_MAX ||
      !valid_query_rows(n, Hq, Hkv))
    return EAGLE_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_tree) || !aligned16(v_tree) ||
      !aligned16(out) || !aligned16(workspace))  // partial results are float4s
    return EAGLE_ERR_INVALID;
  const int sms = current_num_sms();
  const size_t need = attn_kv8_workspace_bytes(B, n, Hq, Hkv, dh, max_pages * page_size, sms);
  if (workspace_bytes < need || (need && !workspace)) return EAGLE_ERR_WORKSPACE;
  return from_cuda(launch_tree_attn_kv8(q, k_pages, v_pages, k_scale, v_scale, block_table, max_pages, page_size,
                                        num_pages, kv_len, k_tree, v_tree, mask, B, n, Hq, Hkv, dh, scale, out, lse,
                                        workspace, status, sms, reinterpret_cast<cudaStream_t>(stream)));
}

int eagle_kv8_bounds(const uint8_t *k_pages, const int32_t *block_table, int max_pages, int page_size, int num_pages,
                     const int32_t *from_len, const int32_t *kv_len, int B, int Hkv, int dh, uint8_t *k_bounds,
                     int32_t *status, eagle_stream_t stream) {
  if (!k_pages || !block_table || !from_len || !kv_len || !k_bounds) return EAGLE_ERR_INVALID;
  if (B < 1 || Hkv < 1 || !valid_pages(max_pages, page_size, num_pages)) return EAGLE_ERR_INVALID;
  if ((dh != 64 && dh != 128) || B > 65535 || static_cast<int64_t>(num_pages) * Hkv > INT32_MAX) return EAGLE_ERR_UNSUPPORTED;
  if (!aligned16(k_pages) || !aligned16(k_bounds)) return EAGLE_ERR_INVALID;
  return from_cuda(launch_kv8_bounds(k_pages, block_table, max_pages, page_size, num_pages, from_len, kv_len, B, Hkv, dh,
                                     k_bounds, status, current_num_sms(), reinterpret_cast<cudaStream_t>(stream)));
}

constexpr int kMaxSelectPages = 16384;  // a request's pages: a row's scores are held by the threads of one CTA

// Nodes by KV heads of a call with selected pages, and heads of a KV head: EAGLE_OK or what is wrong.
static int check_nodes(int B, int n, int Hq, int Hkv, int dh) {
  if (B < 1 || n < 1 || n > 4096 || Hq < 1 || Hkv < 1 || Hq % Hkv) return EAGLE_ERR_INVALID;
  if ((dh != 64 && dh != 128) || Hq / Hkv > 32 || static_cast<int64_t>(B) * Hkv > 65535 ||
      static_cast<int64_t>(B) * n * Hkv > (1 << 24))
    return EAGLE_ERR_UNSUPPORTED;
  return EAGLE_OK;
}

size_t eagle_kv8_select_workspace_size(int dtype, int B, int n, int Hq, int Hkv, int dh, int max_pages, int page_size) {
  if (dtype != EAGLE_BF16 || check_nodes(B, n, Hq, Hkv, dh) != EAGLE_OK || !valid_pages(max_pages, page_size, 1) ||
      max_pages > kMaxSelectPages)
    return 0;
  return kv8_select_workspace_bytes(B, n, Hkv, max_pages);
}

int eagle_kv8_select(const void *q, int dtype, const uint8_t *k_bounds, const float *k_scale, const int32_t *block_table,
                     int max_pages, int page_size, int num_pages, const int32_t *kv_len, int B, int n, int Hq, int Hkv,
                     int dh, int top, int first, int last, int32_t *sel, float *score, int32_t *status, void *workspace,
                     size_t workspace_bytes, eagle_stream_t stream) {
  if (!q || !k_bounds || !k_scale || !block_table || !kv_len || !sel) return EAGLE_ERR_INVALID;
  if (!valid_dtype(dtype) || !valid_pages(max_pages, page_size, num_pages) || top < 1 || first < 0 || last < 0 ||
      first > top || last > top - first)
    return EAGLE_ERR_INVALID;
  const int rc = check_nodes(B, n, Hq, Hkv, dh);
  if (rc != EAGLE_OK) return rc;
  if (dtype != EAGLE_BF16 || max_pages > kMaxSelectPages || top > kMaxSelectPages ||
      static_cast<int64_t>(num_pages) * Hkv > (1 << 30) - 1)  // lines of 128 bytes are numbered in 31 bits
    return EAGLE_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k_bounds) || !aligned16(workspace)) return EAGLE_ERR_INVALID;
  if (!workspace || workspace_bytes < kv8_select_workspace_bytes(B, n, Hkv, max_pages)) return EAGLE_ERR_WORKSPACE;
  return from_cuda(launch_kv8_select(q, k_bounds, k_scale, block_table, max_pages, page_size, num_pages, kv_len, B, n, Hq,
                                     Hkv, dh, top, first, last, sel, score, workspace, status, current_num_sms(),
                                     reinterpret_cast<cudaStream_t>(stream)));
}

// Positions of a list of selected pages, as for a block table.
static bool valid_list(int top, int page_size) { return top >= 1 && static_cast<int64_t>(top) * page_size <= (1 << 24); }

size_t eagle_tree_attn_kv8_pages_workspace_size(int dtype, int B, int n, int Hq, int Hkv, int dh, int top, int max_pages,
                                                int page_size) {
  if (dtype != EAGLE_BF16 || check_nodes(B, n, Hq, Hkv, dh) != EAGLE_OK || !valid_pages(max_pages, page_size, 1) ||
      !valid_list(top, page_size))
    return 0;
  return attn_kv8_pages_workspace_bytes(B, n, Hq, Hkv, dh, top, max_pages, page_size, current_num_sms());
}

int eagle_tree_attn_kv8_pages(const void *q, const uint8_t *k_pages, const uint8_t *v_pages, const float *k_scale,
                              const float *v_scale, const int32_t *block_table, int max_pages, int page_size,
                              int num_pages, const int32_t *kv_len, const void *k_tree, const void *v_tree,
                              const uint64_t *mask, const int32_t *sel, int top, int dtype, int B, int n, int Hq, int Hkv,
                              int dh, float scale, void *out, float *lse, int32_t *status, void *workspace,
                              size_t workspace_bytes, eagle_stream_t stream) {
  if (!q || !k_pages || !v_pages || !k_scale || !v_scale || !block_table || !kv_len || !k_tree || !v_tree || !mask ||
      !sel || !out)
    return EAGLE_ERR_INVALID;
  if (!valid_dtype(dtype) || !(scale > 0.f) || !valid_pages(max_pages, page_size, num_pages) || !valid_list(top, page_size))
    return EAGLE_ERR_INVALID;
  const int rc = check_nodes(B, n, Hq, Hkv, dh);
  if (rc != EAGLE_OK) return rc;
  if (dtype != EAGLE_BF16 || static_cast<int64_t>(num_pages) * Hkv > INT32_MAX) return EAGLE_ERR_UNSUPPORTED;
  if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(k_tree) || !aligned16(v_tree) ||
      !aligned16(out) || !aligned16(workspace))  // partial results are float4s
    return EAGLE_ERR_INVALID;
  const int sms = current_num_sms();
  const size_t need = attn_kv8_pages_workspace_bytes(B, n, Hq, Hkv, dh, top, max_pages, page_size, sms);
  if (workspace_bytes < need || (need && !workspace)) return EAGLE_ERR_WORKSPACE;
  return from_cuda(launch_tree_attn_kv8_pages(q, k_pages, v_pages, k_scale, v_scale, block_table, max_pages, page_size,
                                              num_pages, kv_len, k_tree, v_tree, mask, sel, top, B, n, Hq, Hkv, dh, scale,
                                              out, lse, workspace, status, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
