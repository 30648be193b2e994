/*
 * eagle.h — C ABI of the GB300 (sm_103a) implementation of one EAGLE-2
 * tree-speculative decoding step.
 *
 * The step has four stages, each an entry point below:
 *   eagle_draft_topk  per-row softmax statistics and top-k of the draft logits
 *   eagle_tree_build  global scores, top-k frontier expansion, top-m rerank,
 *                     node order (and, optionally, the attention mask)
 *   eagle_tree_mask   ancestor-only attention mask from parent pointers
 *   eagle_tree_attn   tree-masked attention of the tree nodes over the KV prefix
 *   eagle_verify      greedy or speculative-sampling verification walk
 * and eagle_step runs the four in order (or replays them as one graph).
 * Around them, for a serving loop whose KV cache is paged and held in 8 bits:
 *   eagle_page_map, eagle_page_reserve, eagle_page_release   pages of a free
 *                                        list to requests and back
 *   eagle_rope                           rotary positions of q and k
 *   eagle_qk_norm_rope                   norms of their heads and rotary positions
 *   eagle_kv8_append, eagle_kv8_commit, eagle_kv8_commit_root   keys and values into the 8-bit cache
 *   eagle_tree_attn_kv8                  the tree attention over that cache
 *   eagle_kv8_bounds, eagle_kv8_select, eagle_tree_attn_kv8_pages   the same over the
 *                                        pages that a query's score selects
 *
 * Sources (the pages the method is taken from):
 *   [EAGLE-2] "論文解説: EAGLE-2 - 動的ドラフトツリーによるLLM推論の高速化"
 *             (0h-n0.github.io, paper 2406.16858)
 *   [EAGLE-1] abeam.tech explainer of "EAGLE: Speculative Sampling Requires
 *             Rethinking Feature Uncertainty" (ICML 2024)
 *
 * Conventions for every entry point:
 *   - All array pointers are DEVICE pointers owned by the caller; the library
 *     never allocates, frees or keeps them.  Scratch memory is passed in as
 *     `workspace` (size from the matching *_workspace_size query; a size of
 *     0 means the call needs none).  A workspace needs no initialisation and
 *     keeps no state between calls: a call writes every byte of it that it
 *     reads.  One workspace must not be used by two calls that may overlap
 *     on the GPU.
 *   - Every call is asynchronous on `stream` (NULL = the legacy default
 *     stream).  The return value reports argument and launch errors only:
 *     EAGLE_OK, EAGLE_ERR_INVALID (bad argument, nothing launched),
 *     EAGLE_ERR_UNSUPPORTED (valid but not implemented, nothing launched),
 *     EAGLE_ERR_WORKSPACE (workspace too small), EAGLE_ERR_CUDA (a CUDA error
 *     was reported while launching).
 *   - Errors found on the device (inputs outside the documented domain) are
 *     written to an optional device `status` word as a nonzero eagle_status;
 *     the word is never written on success, so the caller zeroes it first.
 *     No kernel traps or aborts.
 *   - Layouts are dense row-major in the index order given, unless a leading
 *     dimension `ld` (in elements) is given.  Pointers to 16-bit or 32-bit
 *     logits and to attention tensors must be 16-byte aligned.
 */
#ifndef EAGLE_H
#define EAGLE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t. */
typedef struct CUstream_st *eagle_stream_t;

typedef enum {
  EAGLE_OK = 0,
  EAGLE_ERR_INVALID = -1,
  EAGLE_ERR_UNSUPPORTED = -2,
  EAGLE_ERR_CUDA = -3,
  EAGLE_ERR_WORKSPACE = -4,
  EAGLE_ERR_TIMEOUT = -5,
  EAGLE_ERR_PAGES = -6
} eagle_status;

typedef enum { EAGLE_F32 = 0, EAGLE_BF16 = 1 } eagle_dtype;

typedef enum { EAGLE_GREEDY = 0, EAGLE_SAMPLE = 1 } eagle_mode;

/* Human-readable name of a status code (static string, never NULL). */
const char *eagle_status_string(int code);

/* Library version: major * 10000 + minor * 100 + patch. */
int eagle_version(void);

/* ------------------------------------------------------------------------
 * Self test of the bounded device waits (failure detection).
 * The pages describe no failure handling; this call checks the library's
 * own.  Every wait inside the step's kernels (on an mbarrier completed by a
 * copy, an MMA or another CTA of a cluster) gives up after a wall-time
 * limit, and the kernel then reports EAGLE_ERR_TIMEOUT in the status word
 * instead of hanging.  This launches one warp that initialises an mbarrier
 * nothing will ever complete and waits on it with the same helper the
 * kernels use, for `limit_ns` nanoseconds:
 *   which       0: the CTA-local wait; 1: the polling wait used for
 *               barriers that other CTAs of a cluster arrive on; 3: the short
 *               wait of eagle_tree_attn_kv8's roles; 4: the same when another
 *               role has given up already, which ends it before the limit
 *   status      device int32 (required): EAGLE_ERR_TIMEOUT when the wait
 *               gave up as designed, EAGLE_ERR_INVALID if it returned as
 *               though the barrier had completed
 *   elapsed_ns  device uint64 (out; may be NULL): the wall time waited
 * Nothing else is in flight, so the context stays usable afterwards.
 * Limits: 1000 <= limit_ns <= 100000000 (1 us to 100 ms).
 * ------------------------------------------------------------------------ */
int eagle_selftest_wait(uint64_t limit_ns, int which, int32_t *status,
                        uint64_t *elapsed_ns, eagle_stream_t stream);

/* ------------------------------------------------------------------------
 * Stage 1 — draft softmax statistics and top-k.
 * [EAGLE-2] section "ドラフトモデルのキャリブレーション": a draft token's
 * confidence is the probability the draft model assigns it; it approximates
 * the token's acceptance rate.  For each USED row x of the draft logits:
 *   M = max_t x_t,  Z = sum_t exp(x_t - M),
 *   tok[0..k-1] = the k largest logits, in order (ties -> lower token id),
 *   conf[r] = exp(x_tok[r] - M) / Z,  stats = (M, ln Z).
 * Used rows: [b, 0, 0] (the root's distribution) and [b, d, j] for
 * d = 1..D-1, j = 0..k-1 (the j-th expanded node of tree layer d).  Rows
 * [b, 0, 1..k-1] are neither read nor written.
 *
 *   logits  device, dtype `dtype`, row [b, d, j] starts at element
 *           ((b*D + d)*k + j) * ld; 16-byte aligned; V*elemsize and
 *           ld*elemsize multiples of 16 bytes.  Values finite or -inf, at
 *           least k finite per used row, no NaN.
 *   tok     device int32 [B, D, k, k]     (out)
 *   conf    device float [B, D, k, k]     (out)
 *   stats   device float [B, D, k, 2]     (out; may be NULL)
 *   status  device int32 (out; may be NULL): EAGLE_ERR_TIMEOUT if the
 *           bounded wait of a row's merge gave up (the row is then not
 *           written)
 * Workspace: none (the size is 0); a row split over several CTAs merges
 * through the shared memory of their thread-block cluster.
 * Limits: 1 <= k <= 32, k <= V, D >= 1, B >= 1.
 * ------------------------------------------------------------------------ */
size_t eagle_draft_topk_workspace_size(int B, int D, int k, int V);

int eagle_draft_topk(const void *logits, int dtype, int B, int D, int k, int V,
                     int64_t ld, int32_t *tok, float *conf, float *stats,
                     int32_t *status, void *workspace, size_t workspace_bytes,
                     eagle_stream_t stream);

/* ------------------------------------------------------------------------
 * Stage 2 — dynamic draft tree.
 * [EAGLE-2] section "動的ドラフトツリーの構築アルゴリズム": V_i = product of
 * the confidences on the root path (V_i equation); at every depth the k
 * nodes with the largest V are expanded with their own top-k tokens; the m
 * candidates with the largest V are kept; ancestors are added so the set is
 * a connected tree.
 * Computation (exactly): root = gid 0, V = 1.  Depth-1 candidates are the
 * root row's tokens (gids 1..k).  For d = 1..D-1 the k depth-d candidates
 * greatest in the key order (V desc, parent gid asc, token asc) are the
 * expanded set E_d; E_d[j] takes row [d, j]; its children get
 * V = fl32(V_parent * conf) (IEEE float multiply, round to nearest, no
 * flush to zero) and gids numbered depth by depth, by j, then by child rank.
 * The m candidates greatest in key order are kept.  With 0 <= conf <= 1 every
 * ancestor precedes its descendants in key order, so the kept set is
 * already connected (the ancestor step adds nothing).
 * Output order: node 0 = root, nodes 1..m = kept candidates in key order, so
 * parent index < node index.
 *
 *   tok, conf    device int32 / float [B, D, k, k], as written by stage 1
 *                (tokens of one row distinct, 0 <= token < 2^20,
 *                 0 <= conf <= 1)
 *   root_tok     device int32 [B] or NULL (root token reported as -1)
 *   node_tok     device int32 [B, m+1]  (out)
 *   node_parent  device int32 [B, m+1]  (out; root -1)
 *   node_depth   device int32 [B, m+1]  (out; may be NULL)
 *   node_score   device float [B, m+1]  (out; V; may be NULL)
 *   node_src     device int32 [B, m+1]  (out; candidate gid; may be NULL)
 *   node_row     device int32 [B, m+1]  (out; d*k + j if the node was
 *                expanded with row [d, j], root 0, else -1; may be NULL)
 *   mask         device uint64 [B, m+1, W], W = ceil((m+1)/64) (out; may be
 *                NULL) — the same words eagle_tree_mask writes
 *   status       device int32 (out; may be NULL): EAGLE_ERR_INVALID when a
 *                token or confidence is outside its range above.  Repeated
 *                tokens within a row are not checked (stage 1 never writes
 *                them): the tree is then unspecified, but every output
 *                index stays in range and nothing is read or written out of
 *                bounds.
 * Limits: 1 <= k <= 32, D >= 1, 1 <= m <= k + (D-1)k^2 <= 4095.
 * ------------------------------------------------------------------------ */
int eagle_tree_build(const int32_t *tok, const float *conf, int B, int D, int k,
                     int m, const int32_t *root_tok, int32_t *node_tok,
                     int32_t *node_parent, int32_t *node_depth,
                     float *node_score, int32_t *node_src, int32_t *node_row,
                     uint64_t *mask, int32_t *status, eagle_stream_t stream);

/* ------------------------------------------------------------------------
 * Stage 2, ablation variants of the tree build.
 * [EAGLE-2] section "実験結果", ablation table: the method without the global
 * acceptance probability ("confidence only") and without reranking.  Same
 * arguments, outputs and limits as eagle_tree_build, plus `flags`, a bitwise
 * OR of:
 *   EAGLE_TREE_CONFIDENCE_ONLY  rank a candidate by its own confidence c
 *       instead of V (node_score then holds c).  The expansion takes each
 *       layer's k greatest keys as before; the rerank grows the tree
 *       best-first, repeatedly adding the greatest key whose parent is
 *       already in the tree (with V keys this is exactly the top-m set), so
 *       node order is the order of selection and every parent precedes its
 *       children.
 *   EAGLE_TREE_NO_RERANK  no rerank: the tree is the layers' selections
 *       E_1, E_2, ..., E_D (each layer's k greatest keys; E_D chosen the
 *       same way although never expanded), in depth order and rank order
 *       within a depth, truncated to m nodes.  Requires m <= D*k.
 * flags = 0 is eagle_tree_build.  Other bits: EAGLE_ERR_INVALID.
 * ------------------------------------------------------------------------ */
#define EAGLE_TREE_CONFIDENCE_ONLY 1
#define EAGLE_TREE_NO_RERANK 2
int eagle_tree_build_variant(const int32_t *tok, const float *conf, int B, int D,
                             int k, int m, int flags, const int32_t *root_tok,
                             int32_t *node_tok, int32_t *node_parent,
                             int32_t *node_depth, float *node_score,
                             int32_t *node_src, int32_t *node_row,
                             uint64_t *mask, int32_t *status,
                             eagle_stream_t stream);

/* ------------------------------------------------------------------------
 * Stage 2 for the EAGLE-1 static draft tree.
 * [EAGLE-2] sections "背景" and "EAGLE-1からの変更点": EAGLE-1 places its draft
 * tokens on a tree shape fixed in advance and applies it to every input;
 * only the tokens come from the draft.  The shape is an input template:
 *   tree_parent  device int32 [n]: -1 for node 0 (the root), else the parent
 *                index, which must be smaller than the node's own
 *   tree_rank    device int32 [n]: node i is the tree_rank[i]-th of its
 *                parent's top-k draft tokens (0 <= rank < k, distinct among
 *                siblings; entry 0 ignored)
 * Draft rows: the root's distribution is row [0, 0]; the j-th node of depth
 * d >= 1 that has children (in node order) uses row [d, j], so a depth may
 * hold at most k such nodes and none at depth D.  Inputs tok/conf/root_tok
 * and the outputs are those of eagle_tree_build with m = n - 1: node order is
 * the template's, node_src = the template index, node_score = the float32
 * product of the confidences on the root path, node_row = d*k + j for nodes
 * with children (root 0), else -1; mask optional.
 * Device errors: a template that breaks the rules above sets
 * EAGLE_ERR_INVALID in *status (when given) and leaves the outputs unwritten.
 * Limits: 1 <= k <= 32, 1 <= D <= 32, 1 <= n <= 1024.
 * ------------------------------------------------------------------------ */
int eagle_static_tree(const int32_t *tok, const float *conf, int B, int D, int k,
                      const int32_t *tree_parent, const int32_t *tree_rank, int n,
                      const int32_t *root_tok, int32_t *node_tok,
                      int32_t *node_parent, int32_t *node_depth,
                      float *node_score, int32_t *node_src, int32_t *node_row,
                      uint64_t *mask, int32_t *status, eagle_stream_t stream);

/* ------------------------------------------------------------------------
 * Ancestor-only attention mask.
 * [EAGLE-2] section "注意マスクの調整": each token attends only to its
 * ancestors.  Bit (j % 64) of word j / 64 of row i is set iff j == i or j is
 * an ancestor of i (the root is an ancestor of every node).
 *   node_parent  device int32 [B, n] (root -1, parent index < node index)
 *   mask         device uint64 [B, n, ceil(n/64)] (out)
 * Limits: 1 <= n <= 4096.
 * ------------------------------------------------------------------------ */
int eagle_tree_mask(const int32_t *node_parent, int B, int n, uint64_t *mask,
                    eagle_stream_t stream);

/* ------------------------------------------------------------------------
 * Stage 3 — tree attention.
 * [EAGLE-1] sections "用語解説" (Tree Attention) and "Tree Attention の役割":
 * the target scores every branch of the tree in one forward pass; with the
 * [EAGLE-2] mask each tree node attends to the prefix and to its own
 * ancestors.  For node i (0..n-1, n = m+1), query head h, KV head
 * g = h / (Hq/Hkv):
 *   keys = k_cache[b, g, 0:kv_len[b]]  ++  { k_tree[b, g, j] : mask bit j of row i }
 * The root is tree node 0 and counts once: this kv_len is the number of
 * positions before it.
 *   s = scale * <q[b, i, h], key>,  out[b, i, h] = softmax(s) . values,
 *   lse[b, i, h] = ln sum exp(s).
 *   q          [B, n, Hq, dh]        dtype
 *   k_cache    [B, Hkv, Lmax, dh]    dtype   (v_cache alike)
 *   kv_len     device int32 [B], 0 <= kv_len[b] <= Lmax
 *   k_tree     [B, Hkv, n, dh]       dtype   (v_tree alike)
 *   mask       device uint64 [B, n, ceil(n/64)] (as eagle_tree_mask writes)
 *   out        [B, n, Hq, dh]        dtype   (out)
 *   lse        device float [B, n, Hq]  (out; may be NULL)
 *   status     device int32 (out; may be NULL): EAGLE_ERR_TIMEOUT if a
 *              bounded wait inside the kernel gave up
 * Arithmetic: fp32 accumulation and softmax.  bf16 inputs run on the tensor
 * cores (tcgen05, operands staged by TMA, accumulators in tensor memory,
 * probabilities rounded to bf16 for the P.V product); fp32 inputs run on the
 * CUDA cores.  Cache rows at or beyond kv_len[b] are never read; every row
 * of k_tree / v_tree must hold finite values.
 * Workspace (bf16): a launch that splits the KV prefix of a head over
 * several CTAs needs one slot per CTA (fp32 O rows and (m, l) per row); each
 * CTA leaves its partial results there.  When every CTA of the launch is
 * resident at once (one wave) the splits of a head are one thread-block
 * cluster and merge from L2 after a cluster barrier; otherwise a second
 * kernel merges them.  An unsplit launch needs none (size 0).  fp32:
 * partial results and weights.
 * Limits: Hq % Hkv == 0, dh in {64, 128}, 1 <= n <= 4096, B*Hkv <= 65535.
 * ------------------------------------------------------------------------ */
size_t eagle_tree_attn_workspace_size(int dtype, int B, int n, int Hq, int Hkv,
                                      int dh, int Lmax);

/* Kernels one eagle_tree_attn call with these arguments launches (1 or 2:
 * the attention, and the merge of a split launch of several waves, or the
 * fp32 combine); 0 for invalid arguments.  Host only. */
int eagle_tree_attn_kernel_count(int dtype, int B, int n, int Hq, int Hkv,
                                 int dh, int Lmax);

int eagle_tree_attn(const void *q, const void *k_cache, const void *v_cache,
                    const int32_t *kv_len, const void *k_tree,
                    const void *v_tree, const uint64_t *mask, int dtype, int B,
                    int n, int Hq, int Hkv, int dh, int Lmax, float scale,
                    void *out, float *lse, int32_t *status, void *workspace,
                    size_t workspace_bytes, eagle_stream_t stream);

/* ------------------------------------------------------------------------
 * Stage 3 over a paged KV prefix (block-table attention).
 * Same computation as eagle_tree_attn; the prefix K/V live in page pools
 *   k_pages, v_pages  bf16 [num_pages, Hkv, page_size, dh]
 *   block_table       device int32 [B, max_pages]: logical page p of
 *                     sequence b is physical page block_table[b, p]
 * so prefix position L of sequence b is row L % page_size of page
 * block_table[b, L / page_size] (entries for pages at or beyond kv_len are
 * not read).  kv_len[b] is clamped to max_pages * page_size.  Other
 * arguments as in eagle_tree_attn.  Workspace from
 * eagle_tree_attn_paged_workspace_size.
 * Device errors: a block-table entry outside [0, num_pages) for a page the
 * prefix uses sets EAGLE_ERR_INVALID (page 0 is read in its place).
 * Limits: bf16 only (other dtypes EAGLE_ERR_UNSUPPORTED); dh in {64, 128};
 * page_size a power of two in [16, 4096]; max_pages * page_size <= 2^24.
 * ------------------------------------------------------------------------ */
size_t eagle_tree_attn_paged_workspace_size(int dtype, int B, int n, int Hq,
                                            int Hkv, int dh, int max_pages,
                                            int page_size);

int eagle_tree_attn_paged(const void *q, const void *k_pages,
                          const void *v_pages, const int32_t *block_table,
                          int max_pages, int page_size, int num_pages,
                          const int32_t *kv_len, const void *k_tree,
                          const void *v_tree, const uint64_t *mask, int dtype,
                          int B, int n, int Hq, int Hkv, int dh, float scale,
                          void *out, float *lse, int32_t *status,
                          void *workspace, size_t workspace_bytes,
                          eagle_stream_t stream);

/* ------------------------------------------------------------------------
 * Stage 4 — verification walk.
 * [EAGLE-1] section "検証方法": each draft token is accepted or rejected by
 * the ratio of target and draft distributions; after a rejection the rest is
 * discarded and a token resampled; the output follows the target exactly
 * ([EAGLE-2]: lossless, rejection sampling as in EAGLE-1; temp=0 greedy).
 * Row i of the target logits is the target's distribution after node i.
 *   GREEDY: from the root, a = argmax of the current row (ties -> lower
 *     token); move to the child carrying a while one exists; a is the bonus.
 *   SAMPLE (temperature T > 0): children are point-mass drafts.  With
 *     e_t = exp(x_t/T - max), Z = sum e, S = tokens rejected at this node:
 *     child x (token t) is accepted iff u[b,x,0] * (Z - sum_S e) < e_t;
 *     otherwise t joins S.  With no child accepted, the bonus is the
 *     smallest t not in S whose cumulative residual mass exceeds
 *     u[b,cur,1] * (Z - sum_S e).  Children are tried in node-index order.
 *   target     dtype, row (b, i) starts at element (b*(m+1) + i) * ld
 *   node_tok, node_parent   device int32 [B, m+1] (as stage 2 writes)
 *   uniforms   device float [B, m+1, 2] in [0, 1) (SAMPLE; NULL for GREEDY)
 *   accept_len device int32 [B]            (out; accepted draft tokens)
 *   path_nodes device int32 [B, D+1]       (out; root first; -1 padded)
 *   out_tokens device int32 [B, D+1]       (out; accepted tokens, then the
 *                                           bonus token; -1 padded)
 *   status     device int32 (out; may be NULL): EAGLE_ERR_INVALID when the
 *              walk meets a row with no finite logit (greedy: no argmax) or
 *              with no residual mass (sampling), or a child token outside
 *              [0, V) (sampling); the bonus token is then -1
 * D bounds the tree depth.  Limits: V*elemsize and ld*elemsize multiples of
 * 16 bytes; 1 <= m+1 <= 4096; D >= 1.
 * ------------------------------------------------------------------------ */
size_t eagle_verify_workspace_size(int B, int m, int V);

int eagle_verify(const void *target, int dtype, int64_t ld,
                 const int32_t *node_tok, const int32_t *node_parent, int B,
                 int m, int D, int V, int mode, float temperature,
                 const float *uniforms, int32_t *accept_len,
                 int32_t *path_nodes, int32_t *out_tokens, int32_t *status,
                 void *workspace, size_t workspace_bytes,
                 eagle_stream_t stream);

/* ------------------------------------------------------------------------
 * Stage 4 without caller scratch: eagle_verify_noalloc.
 * The paper has no counterpart to this entry point.  It serves callers that
 * cannot allocate device memory for a workspace: a plugin or custom-op hook
 * inside a host runtime that owns every device buffer and hands the op only
 * its inputs and outputs; a serving loop that must not call cudaMalloc once
 * it is running (cudaMalloc can synchronise the device and stall the work
 * in flight); a process whose device memory is all handed to its own pool.
 * Same arguments, results and device errors as eagle_verify, without the
 * workspace arguments.  The per-chunk statistics records that eagle_verify
 * keeps in its workspace live instead in one array inside the library
 * (a file-scope __device__ array of EAGLE_VERIFY_NOALLOC_SCRATCH_BYTES
 * bytes), which every GPU that loads the library holds until the process
 * exits.  Nothing is allocated by the call itself.
 *   - A request whose records exceed the array (eagle_verify_workspace_size
 *     > EAGLE_VERIFY_NOALLOC_SCRATCH_BYTES) returns EAGLE_ERR_WORKSPACE and
 *     launches nothing.  8 MiB covers B * (m+1) * ceil(V/2048) <= 524288
 *     records, e.g. B = 64, m = 60, V = 201088.
 *   - The first call on a device looks up the array's device address (with
 *     that device current) and keeps it; make that first call before any
 *     stream capture.
 *   - Every call shares the one array, and it keeps the last call's
 *     records.  No record needs clearing: each call writes every record it
 *     reads.  Two calls that may overlap on the GPU (on different streams
 *     without an ordering between them, or on one device from two threads
 *     through unordered streams) race on the array and give wrong results.
 * ------------------------------------------------------------------------ */
#define EAGLE_VERIFY_NOALLOC_SCRATCH_BYTES (8u << 20)

int eagle_verify_noalloc(const void *target, int dtype, int64_t ld,
                         const int32_t *node_tok, const int32_t *node_parent,
                         int B, int m, int D, int V, int mode,
                         float temperature, const float *uniforms,
                         int32_t *accept_len, int32_t *path_nodes,
                         int32_t *out_tokens, int32_t *status,
                         eagle_stream_t stream);

/* ------------------------------------------------------------------------
 * Stage 4 with draft distributions — speculative-sampling verification of a
 * tree whose tokens were drawn from the draft's distribution q.
 * [EAGLE-1] section "検証方法": a drafted token t is accepted with
 * probability min(1, p(t)/q(t)); after a rejection the target distribution is
 * replaced by the residual norm(max(0, p - q)) and a token is finally drawn
 * from it, so the output follows the target exactly.  Tree form: at node cur
 * the children (node-index order, all drafted from q = softmax(draft row of
 * cur / T)) are tested in turn against the current residual R = max(0, p -
 * C q) with normaliser S (C = 0, S = 1 before any rejection; a rejection
 * adds S to C and S becomes sum over the vocabulary of the new R):
 *   child x with token t is accepted iff u[b,x,0] * S * q(t) < R(t);
 * with no child accepted (or at a leaf) the bonus is the smallest token
 * whose cumulative R exceeds u[b,cur,1] * sum(R).  A residual that sums to 0
 * is replaced by p.  p = softmax(target row / T).
 *   target     dtype, row (b, i) at element (b*(m+1) + i) * ld_t
 *   draft      dtype, draft logits [B, D, k, V], row (b, d, j) at element
 *              ((b*D + d)*k + j) * ld_d (the rows eagle_draft_topk reads)
 *   node_tok, node_parent, node_row   device int32 [B, m+1] as stage 2
 *              writes them; node_row[b, i] = d*k + j names the draft row of
 *              every node that has children
 *   uniforms   device float [B, m+1, 2] in [0, 1)
 *   accept_len, path_nodes, out_tokens, status   as in eagle_verify
 * No workspace: the CTAs of a sequence (one thread-block cluster of up to
 * 8, each over a slice of the vocabulary) keep their state in shared memory
 * and exchange their partial sums through distributed shared memory.
 * Device errors: a node with children whose node_row is outside [0, D*k),
 * a token outside [0, V) or no residual mass set EAGLE_ERR_INVALID.
 * Limits: temperature > 0; V*elemsize, ld_t*elemsize and ld_d*elemsize
 * multiples of 16 bytes; 16-byte aligned logits; 1 <= m+1 <= 4096;
 * 1 <= D; 1 <= k <= 32; B <= 65535 (else EAGLE_ERR_UNSUPPORTED).
 * ------------------------------------------------------------------------ */
int eagle_verify_draft(const void *target, const void *draft, int dtype,
                       int64_t ld_t, int64_t ld_d, const int32_t *node_tok,
                       const int32_t *node_parent, const int32_t *node_row,
                       int B, int m, int D, int k, int V, float temperature,
                       const float *uniforms, int32_t *accept_len,
                       int32_t *path_nodes, int32_t *out_tokens,
                       int32_t *status, eagle_stream_t stream);

/* ------------------------------------------------------------------------
 * After verification — commit the accepted path's keys and values.
 * [EAGLE-1] section "検証方法" / [EAGLE-2]: the accepted draft tokens become
 * part of the sequence; everything after a rejection is discarded.  The
 * root's K/V is already the last prefix position: the caller has stored it
 * after the attention, whose kv_len was one less (the root was its tree node
 * 0); eagle_kv8_commit_root stores it too.  For each sequence b with
 * a = accept_len[b], nodes path_nodes[b, 1..a] (as eagle_verify writes them)
 * have their rows of k_tree/v_tree [B, Hkv, n, dh] copied, in path order, to
 * positions kv_len[b] .. kv_len[b]+a-1 of the cache, and kv_len[b] becomes
 * kv_len[b] + a (updated in place).
 *   cache        block_table == NULL: contiguous k_cache/v_cache
 *                [B, Hkv, Lmax, dh]; otherwise page pools [num_pages, Hkv,
 *                page_size, dh] addressed through block_table [B, max_pages]
 *                (the caller has mapped the pages the new positions need)
 *   slot_mapping device int32 [B, n] (out, may be NULL): node i's position
 *                after the commit (root kv_len-1), -1 for nodes not kept
 * Device errors: a path node outside [1, n), a = accept_len outside [0, D],
 * kv_len < 1, or new positions beyond the cache (Lmax, or an unmapped page)
 * set EAGLE_ERR_INVALID and leave that sequence unchanged.
 * Limits: dh*elemsize a multiple of 16 bytes; 1 <= D <= 64; n <= 4096; page
 * rules as for eagle_tree_attn_paged.
 * ------------------------------------------------------------------------ */
int eagle_kv_commit(const void *k_tree, const void *v_tree, int dtype, int B,
                    int n, int Hkv, int dh, const int32_t *accept_len,
                    const int32_t *path_nodes, int D, void *k_cache,
                    void *v_cache, int Lmax, const int32_t *block_table,
                    int max_pages, int page_size, int num_pages,
                    int32_t *kv_len, int32_t *slot_mapping, int32_t *status,
                    eagle_stream_t stream);

/* ------------------------------------------------------------------------
 * Pages for new tokens: block tables and slot maps from request lengths.
 * The explainers name the KV cache of the serving systems but no layout; this
 * is the bookkeeping behind the block tables that eagle_tree_attn_paged,
 * eagle_kv_commit and the 8-bit cache below read, kept on the device so that
 * a step needs no host round trip.
 * With P = page_size, need_b = ceil((kv_len[b] + new_len[b]) / P) and
 * add_b = max(0, need_b - page_count[b]): request b gets add_b pages from the
 * free list, a stack whose top is free_pages[free_count - 1].  The j-th page
 * taken over all requests (requests in order, logical pages in order) is
 * free_pages[free_count - 1 - j]; it is written to
 * block_table[b, page_count[b] ...], page_count[b] becomes
 * max(page_count[b], need_b) and free_count drops by the pages taken.  The
 * new tokens are numbered request by request: token t of request b is its
 * position kv_len[b] + (t - new_start[b]), and
 *   slot_map[t] = block_table[b, position / P] * P + position % P,
 * -1 for T > t >= the number of new tokens.
 *   kv_len       device int32 [B]: tokens already in each request's cache
 *   new_len      device int32 [B]: tokens about to be written (0 allowed);
 *                before a tree step, the root and the most nodes that the
 *                verification can accept after it
 *   block_table  device int32 [B, max_pages]  (in/out; other entries stay)
 *   page_count   device int32 [B]             (in/out: pages mapped)
 *   free_pages   device int32 [num_pages]     (in; distinct page numbers
 *                below free_count)
 *   free_count   device int32 [1]             (in/out)
 *   slot_map     device int32 [T]             (out; may be NULL with T = 0)
 *   new_start    device int32 [B+1]           (out; may be NULL): sums of
 *                new_len before each request, then the total
 *   status       device int32 (out; may be NULL): EAGLE_ERR_PAGES when the
 *                free list holds too few pages; EAGLE_ERR_INVALID for a
 *                negative length, a request beyond max_pages pages, a
 *                page_count outside [0, max_pages], a free_count outside
 *                [0, num_pages], or more than T new tokens with a slot_map.
 *                Nothing is written then.  A page number outside
 *                [0, num_pages) in either list gives slot -1 and
 *                EAGLE_ERR_INVALID (one that is taken from the free list
 *                becomes block_table entry -1, with or without a slot_map).
 * Limits: 1 <= B <= 4096; T <= 2^30; page rules as for
 * eagle_tree_attn_paged; num_pages * page_size < 2^31.
 * ------------------------------------------------------------------------ */
int eagle_page_map(const int32_t *kv_len, const int32_t *new_len, int B,
                   int page_size, int max_pages, int num_pages,
                   int32_t *block_table, int32_t *page_count,
                   const int32_t *free_pages, int32_t *free_count,
                   int32_t *slot_map, int T, int32_t *new_start,
                   int32_t *status, eagle_stream_t stream);

/* eagle_page_map for a loop that does not look at `status` before what comes
 * next (a captured one cannot).  When the map is refused, slot_map and
 * new_start would keep what an earlier call left there, and eagle_kv8_append
 * would write through slots that may belong to another request by then.  Here
 * a refusal is written out: slot_map becomes -1 throughout (the append skips
 * such tokens), new_start 0, and
 *   granted      device int32 [1] (out): 1, or 0 when the map is refused, so
 *                that kv_len + granted * new_len are the lengths after it
 * Everything else is as eagle_page_map leaves it, status included. */
int eagle_page_reserve(const int32_t *kv_len, const int32_t *new_len, int B,
                       int page_size, int max_pages, int num_pages,
                       int32_t *block_table, int32_t *page_count,
                       const int32_t *free_pages, int32_t *free_count,
                       int32_t *slot_map, int T, int32_t *new_start,
                       int32_t *granted, int32_t *status,
                       eagle_stream_t stream);

/* Pages back to the free list.  Request b keeps its first
 * min(page_count[b], ceil(keep_len[b] / P)) pages (keep_len 0: none; its
 * kv_len: what it uses now) and gives back the others; a negative keep_len
 * leaves it as it is.  Of R pages given back, in the order in which
 * eagle_page_map takes them, the k-th goes to
 * free_pages[free_count + R - 1 - k]: releasing what a map took restores the
 * stack.  Their block_table entries become -1, page_count the pages kept,
 * free_count grows by R.
 *   keep_len     device int32 [B]; the other arrays as in eagle_page_map
 *   status       EAGLE_ERR_INVALID (nothing written) for a page_count outside
 *                [0, max_pages], a free_count below 0, a free list that
 *                would exceed num_pages entries, or an entry to be given back
 *                that is no page (outside [0, num_pages)).
 * Limits as for eagle_page_map. */
int eagle_page_release(const int32_t *keep_len, int B, int page_size,
                       int max_pages, int num_pages, int32_t *block_table,
                       int32_t *page_count, int32_t *free_pages,
                       int32_t *free_count, int32_t *status,
                       eagle_stream_t stream);

/* ------------------------------------------------------------------------
 * Rotary positions of queries and keys, into the tree attention's layouts.
 * The target's layers rotate the pair (x_a, x_b) number j of each head by the
 * angle position * inv_freq[j] before the attention:
 *   x_a' = factor * (x_a cos - x_b sin),  x_b' = factor * (x_b cos + x_a sin)
 * for j < rot_dim / 2; the pair is (j, j + rot_dim/2) or, with `interleaved`,
 * (2j, 2j + 1).  Columns rot_dim .. dh-1 are copied.  The position of node i
 * of sequence b is pos_base[b] + pos_off[b, i] + shift (pos_base NULL: 0;
 * pos_off NULL: i).  For a tree pass the attention's kv_len (the positions
 * before the root), node_depth and shift = 0; where kv_len counts the root
 * already, shift = -1.
 *   q, k, v    dtype, node (b, i) starts at element (b*n + i) * ld_q (ld_k,
 *              ld_v), its heads dh apart: slices of one fused projection do.
 *              v may be NULL (then v_tree is unused)
 *   inv_freq   device double [rot_dim/2] (eagle_rope_freqs computes them)
 *   pos_base   device int32 [B] or NULL;  pos_off  device int32 [B, n] or NULL
 *   q_out      dtype [B, n, Hq, dh]   (out; may be q itself when ld_q = Hq*dh)
 *   k_tree     dtype [B, Hkv, n, dh]  (out)
 *   v_tree     dtype [B, Hkv, n, dh]  (out: v in that layout)
 * Other outputs must not overlap the inputs.  Angles are reduced in 64-bit
 * fixed point (turns): one is off by at most 2^-25 pi + position * inv_freq *
 * 2^-52 radians (1.3e-7 up to positions of 2^27, 6e-7 at 2^31).  cos, sin and the
 * rotation are float32, rounded once to the output type.
 * Limits: n >= 1; B*n <= 2^24; Hq, Hkv >= 1; rot_dim even, 2 <= rot_dim <=
 * dh <= 512; dh*elemsize and ld*elemsize multiples of 16 bytes, tensors
 * 16-byte aligned.
 * ------------------------------------------------------------------------ */
int eagle_rope(const void *q, const void *k, const void *v, int dtype, int B,
               int n, int Hq, int Hkv, int dh, int64_t ld_q, int64_t ld_k,
               int64_t ld_v, const double *inv_freq, int rot_dim,
               int interleaved, float factor, const int32_t *pos_base,
               const int32_t *pos_off, int shift, void *q_out, void *k_tree,
               void *v_tree, eagle_stream_t stream);

/* eagle_rope after a norm of each head of q and k, in one pass: with
 *   r = 1 / sqrt(mean over the head's dh columns of x_c^2 + eps),
 *   y_c = x_c * r * (weight[c] + weight_offset)
 * the head y turns as eagle_rope turns x (so columns past rot_dim are y); v is
 * copied.
 *   q_weight, k_weight  dtype [dh], the same for every head; NULL: y_c = x_c * r
 *              (weight_offset counts for nothing then)
 * The other arguments are eagle_rope's.  Everything between the element read and
 * the one written is float32, rounded once; sums of squares past float32's range
 * give zeros.  A head that holds an infinity or NaN spoils no other.
 * Limits: those of eagle_rope; eps > 0 and finite, weight_offset finite, weights
 * 16-byte aligned. */
int eagle_qk_norm_rope(const void *q, const void *k, const void *v, int dtype,
                       int B, int n, int Hq, int Hkv, int dh, int64_t ld_q,
                       int64_t ld_k, int64_t ld_v, const void *q_weight,
                       const void *k_weight, float weight_offset, float eps,
                       const double *inv_freq, int rot_dim, int interleaved,
                       float factor, const int32_t *pos_base,
                       const int32_t *pos_off, int shift, void *q_out,
                       void *k_tree, void *v_tree, eagle_stream_t stream);

/* The frequencies of eagle_rope, computed on the host in double:
 * f_j = theta^(-2j / rot_dim), stretched for contexts longer than the
 * orig_len tokens a model was trained on:
 *   EAGLE_ROPE_PLAIN   f_j
 *   EAGLE_ROPE_LINEAR  f_j / stretch
 *   EAGLE_ROPE_BANDS   by the turns t_j = orig_len f_j / 2pi that pair j makes
 *                      over the trained context: f_j / stretch at t_j <= low,
 *                      f_j at t_j >= high, linear in t_j between
 *   EAGLE_ROPE_YARN    the same ends, as pair indexes rounded outwards to whole
 *                      pairs, but linear in the pair's index between, and
 *                      *factor = 0.1 ln(stretch) + 1 (1 for the others).  A
 *                      model whose ramp keeps the ends unrounded (GPT-OSS's
 *                      does) passes its own inv_freq to eagle_rope
 *   inv_freq  HOST double [rot_dim/2] (out);  factor  HOST float (out; may be
 *             NULL)
 * Limits: rot_dim even, >= 2; theta > 1; stretch >= 1; BANDS and YARN:
 * orig_len >= 1, 0 < low < high; all of them finite. */
#define EAGLE_ROPE_PLAIN 0
#define EAGLE_ROPE_LINEAR 1
#define EAGLE_ROPE_BANDS 2
#define EAGLE_ROPE_YARN 3
int eagle_rope_freqs(int rot_dim, double theta, int kind, double stretch,
                     int orig_len, double low, double high, double *inv_freq,
                     float *factor);

/* ------------------------------------------------------------------------
 * The paged KV cache in 8 bits.
 *   k_pages, v_pages  uint8 [num_pages, Hkv, page_size, dh]: e4m3 numbers
 *   k_scale, v_scale  float [num_pages, Hkv]: one scale for each page and head,
 *                     a power of two in [2^-64, 2^64]
 * A cache value is its e4m3 number times its page's scale.  The scale is 2^e
 * with the least e for which every row written to the page so far fits:
 * max |x| <= 448 * 2^e.  A power of two costs no precision in a floating
 * format (x / 2^e is exact, so a value is rounded once, to nearest even) and
 * leaves a cache value exact in 16 bits.  When later rows need a larger scale the
 * page's earlier rows are re-encoded; that too is exact but for numbers below
 * 2^-6 of the new scale.
 * Rows are written in order: a page's row 0 starts the page afresh (its old
 * scale and rows count no more), any other row joins the rows before it.
 * A value that is not finite is stored as NaN, counts for no maximum and sets
 * EAGLE_ERR_INVALID; one beyond 448 * 2^64 is stored as the largest number.
 *
 * eagle_kv8_append writes T tokens (a prompt's, or one per sequence) to
 * the slots of eagle_page_map:
 *   k, v      dtype; token t's head h starts at element
 *             t*token_stride + h*head_stride
 *   slot_map  device int32 [T]: page * page_size + row; negative entries are
 *             skipped.  The tokens of one page are neighbours in slot_map with
 *             consecutive rows (as eagle_page_map lists them): a neighbour in
 *             the same page that breaks the sequence is skipped and sets
 *             EAGLE_ERR_INVALID, as does a slot past the pool.  So does a page
 *             that comes again after skipped tokens (up to 1024 of them) or
 *             within 32 tokens: its first tokens are written, the later ones
 *             skipped.  A page that is listed in two places further apart ends
 *             up unspecified.
 *   status    device int32 (out; may be NULL)
 * Limits: 0 <= T <= 2^30; dh a multiple of 16, at most 512; strides *
 * elemsize multiples of 16 bytes, tensors 16-byte aligned; page_size a power
 * of two in [16, 4096]; num_pages * page_size < 2^31; Hkv <= 32767.
 * ------------------------------------------------------------------------ */
int eagle_kv8_append(const void *k, const void *v, int dtype, int T, int Hkv,
                     int dh, int64_t token_stride, int64_t head_stride,
                     const int32_t *slot_map, uint8_t *k_pages,
                     uint8_t *v_pages, float *k_scale, float *v_scale,
                     int page_size, int num_pages, int32_t *status,
                     eagle_stream_t stream);

/* eagle_kv_commit into the 8-bit cache: the accepted path's rows of
 * k_tree/v_tree [B, Hkv, n, dh] join the cache at kv_len[b] .., kv_len[b]
 * grows by accept_len[b].  Arguments, slot_mapping and device errors as in
 * eagle_kv_commit with a block table: the root is stored already, and kv_len
 * is one more than the attention's.  Limits: those of eagle_kv_commit and of
 * eagle_kv8_append. */
int eagle_kv8_commit(const void *k_tree, const void *v_tree, int dtype, int B,
                     int n, int Hkv, int dh, const int32_t *accept_len,
                     const int32_t *path_nodes, int D, uint8_t *k_pages,
                     uint8_t *v_pages, float *k_scale, float *v_scale,
                     const int32_t *block_table, int max_pages, int page_size,
                     int num_pages, int32_t *kv_len, int32_t *slot_mapping,
                     int32_t *status, eagle_stream_t stream);

/* The commit of a decoding loop: the root's rows too.  The loop has one rule:
 * kv_len counts the positions before the root, the tree holds the root as
 * node 0 (position kv_len, depth 0), so
 *   eagle_page_map with new_len = D + 1 -> eagle_rope with pos_base = kv_len,
 *   pos_off = node_depth, shift = 0 -> eagle_tree_attn_kv8 with kv_len ->
 *   eagle_verify -> this call -> eagle_page_release with kv_len
 * and the bonus token is the next root.  Nodes path_nodes[b, 0..a] (the root
 * first) go to positions kv_len[b] .. kv_len[b]+a, and kv_len[b] becomes
 * kv_len[b] + a + 1; slot_mapping gives the root kv_len[b] and node
 * path_nodes[b, p] kv_len[b] + p, by the kv_len before.  With several layers
 * every call but the last gets a copy of kv_len.
 * Device errors as in eagle_kv8_commit, but kv_len 0 is a length like others
 * and path_nodes[b, 0] has to be 0.  Limits of eagle_kv8_commit. */
int eagle_kv8_commit_root(const void *k_tree, const void *v_tree, int dtype,
                          int B, int n, int Hkv, int dh,
                          const int32_t *accept_len, const int32_t *path_nodes,
                          int D, uint8_t *k_pages, uint8_t *v_pages,
                          float *k_scale, float *v_scale,
                          const int32_t *block_table, int max_pages,
                          int page_size, int num_pages, int32_t *kv_len,
                          int32_t *slot_mapping, int32_t *status,
                          eagle_stream_t stream);

/* ------------------------------------------------------------------------
 * Stage 3 over the 8-bit paged cache.
 * The computation of eagle_tree_attn_paged with the prefix's keys and values
 * read from the 8-bit cache above; queries and tree K/V stay bf16.  n = 1
 * (mask word 1) is plain decoding of one token per sequence.
 *   k_pages, v_pages, k_scale, v_scale   as above; scales that are not powers
 *              of two in range are read as the power of two below, clamped
 *   block_table, max_pages, page_size, num_pages, kv_len, k_tree, v_tree,
 *   mask, scale, out, lse, workspace      as in eagle_tree_attn_paged; bits of
 *              the mask past the last node count for nothing
 *   status     EAGLE_ERR_INVALID for a block-table entry outside
 *              [0, num_pages) on a page that the prefix uses (page 0 is read
 *              in its place), EAGLE_ERR_TIMEOUT as in eagle_tree_attn
 * A row without any key (kv_len 0, empty mask row) gives zeros and lse =
 * -inf; a row that attends to a NaN of the cache gives NaN.  Rows of a page at
 * or beyond kv_len may be read but never count, whatever they hold; nor do
 * tree nodes that no row of the mask names.  q, and k_tree and v_tree of the
 * nodes that some row names, must be finite.
 * What is rounded beside the output:
 *   - An element of k_tree or v_tree is exact down to 2^-25 of the largest
 *     magnitude M among its neighbours and off by up to 2^-33 M below that.
 *     Neighbours are the nodes of one block of 16 to 128 of a head (page_size
 *     decides) that any row names (with more than 64 nodes: any of up to 256
 *     neighbouring query rows), so a large node costs rows bits that do not
 *     name it.
 *   - A weight p_k meets its value in f16, with the value's scale 2^e_k (a
 *     page's, or a tree block's power of two) joined to it: key k is off by up
 *     to |v_k| (2^-11 p_k + 2^-31 2^-e_k max_j(p_j 2^e_j)).  Where one row's
 *     value scales lie 2^20 and more apart, an outlier on one page thus costs
 *     the keys of the others bits, in every column; up to 2^100 apart they
 *     keep their weight in the sum (below 2^-32 of it is lost), further apart
 *     out and lse may leave them out.
 *   - Scores are float32: where one passes 2^127, rows that name its key are
 *     undefined; scores of 0 are 0 whatever q and k are multiplied with.
 * Limits: dtype EAGLE_BF16 (else EAGLE_ERR_UNSUPPORTED); dh in {64, 128};
 * scale > 0; page rules as for eagle_tree_attn_paged; num_pages*Hkv < 2^31;
 * n * Hq/Hkv <= 2^23; workspace 16-byte aligned (else EAGLE_ERR_INVALID).
 * ------------------------------------------------------------------------ */
size_t eagle_tree_attn_kv8_workspace_size(int dtype, int B, int n, int Hq,
                                          int Hkv, int dh, int max_pages,
                                          int page_size);

int eagle_tree_attn_kv8(const void *q, const uint8_t *k_pages,
                        const uint8_t *v_pages, const float *k_scale,
                        const float *v_scale, const int32_t *block_table,
                        int max_pages, int page_size, int num_pages,
                        const int32_t *kv_len, const void *k_tree,
                        const void *v_tree, const uint64_t *mask, int dtype,
                        int B, int n, int Hq, int Hkv, int dh, float scale,
                        void *out, float *lse, int32_t *status,
                        void *workspace, size_t workspace_bytes,
                        eagle_stream_t stream);

/* ------------------------------------------------------------------------
 * Long contexts: attention to the pages that a query selects.
 * Three calls: bounds of each page's keys, kept beside the pages; the pages whose
 * bounds allow a query, rounded to 8 bits, the greatest products; the attention over
 * those pages and the tree.  A query is a node of the tree and a KV head (the heads that share it
 * choose together), and what it selects depends on nothing but itself, kv_len, the
 * prefix's scales and bounds: not on the tree around it, the batch or the launch.
 * Verification over selected pages is not decoding token by token over selected
 * pages: a node attends to the tree's path beside its `top` pages, a token decoded
 * alone has that path in pages that take places of `top`.  Node i of a path selects
 * the pages that its token selects alone (with kv_len + i, the path's rows stored)
 * where last >= 1 and positions kv_len - 1 .. kv_len + i - 1 lie in one page; the keys
 * are then the same, the path's own up to their rounding to e4m3.  A path that
 * goes on into another page (any node but the root, where kv_len is a multiple of
 * page_size), or last = 0, may give other lists, and so other tokens.
 *
 * eagle_kv8_bounds renews the bounds of every page that holds positions
 * from_len[b] .. kv_len[b]-1 of a request, from all of the page's rows before
 * kv_len[b]: after an append or a commit, with the length before it.  An append that
 * gives a page a larger scale leaves its bounds in the old one's units until this
 * call, also where the new rows are not counted in the end: a from_len of the length
 * before less one always renews the last page, and eagle_kv8_select comes before the
 * append or after this call.
 *   k_pages    as in eagle_kv8_append; block_table, max_pages, page_size,
 *              num_pages as in eagle_tree_attn_paged
 *   from_len, kv_len   device int32 [B]; nothing is done where kv_len <= from_len;
 *              a negative from_len counts as 0, kv_len is clamped to max_pages *
 *              page_size
 *   k_bounds   uint8 [num_pages, Hkv, 2, dh]  (in/out): e4m3 numbers in units of
 *              the page's k_scale: over the page's rows, the least number of each
 *              column rounded down to a multiple of 1/2, then the greatest rounded
 *              up (both are e4m3 numbers); -448 and 448 where a row holds NaN.
 *              Pages that are not touched keep theirs.  A request that is cut short
 *              keeps the wider bounds of its last page until a call with a from_len
 *              below its new length
 *   status     EAGLE_ERR_INVALID for a block-table entry outside [0, num_pages)
 *              on a touched page (it is skipped).  A page belongs to one request:
 *              the bounds of one that two requests touch are unspecified
 * Limits: dh in {64, 128}; B <= 65535 (else EAGLE_ERR_UNSUPPORTED);
 * num_pages*Hkv < 2^31; page rules as for eagle_tree_attn_paged.
 * ------------------------------------------------------------------------ */
int eagle_kv8_bounds(const uint8_t *k_pages, const int32_t *block_table,
                     int max_pages, int page_size, int num_pages,
                     const int32_t *from_len, const int32_t *kv_len, int B,
                     int Hkv, int dh, uint8_t *k_bounds, int32_t *status,
                     eagle_stream_t stream);

/* The `top` pages of each node i and KV head g, out of the ceil(kv_len[b] / P)
 * pages of its sequence's prefix.  A query row (node i, head h) counts as whole
 * numbers q'_c = rint(q_c / 2^e) with 64 <= max |q'_c| <= 128 (e between -32 and 32,
 * |q'_c| at most 128 beyond; an element that is not finite counts as 0), and the
 * score of a page with bounds lo, hi and scale s is
 *   max over the heads h of g of  2^e s (sum over q'_c > 0 of q'_c hi_c
 *                                        + sum over q'_c < 0 of q'_c lo_c),
 * the greatest product with q' of any key within the bounds.  It ranks pages by the
 * rounded row, and is no bound for q itself: q' is off by up to 2^(e-1) a column, the
 * score by up to 2^(e-1) s times the sum of max(|lo|, |hi|), and columns below 1/256 of
 * the row's largest count for nothing.
 * Every score is exact in float32, in any order of the sum.  Selected are the first
 * `first` and the last `last` pages of the prefix, then the greatest scores, ties to
 * the lower page; all of them where the prefix has no more than `top`.
 *   q          dtype [B, n, Hq, dh], as for the attention (rotated)
 *   k_bounds   as above;  k_scale as in eagle_kv8_append (read as the power of two
 *              below, clamped to its range)
 *   sel        device int32 [B, n, Hkv, top] (out): logical page numbers,
 *              ascending, then -1
 *   score      device float [B, n, Hkv, top] (out; may be NULL): their scores, also
 *              of pages that are selected without one, then -inf
 *   status     EAGLE_ERR_INVALID for a block-table entry outside [0, num_pages)
 *              (page 0's bounds are read in its place)
 * Workspace: the scores of all pages, one float for each node, KV head and page of the
 * table (max_pages, whatever the lengths): 2.1 GB for 4096 nodes, 8 heads, 16384 pages.
 * Limits: dtype EAGLE_BF16, dh in {64, 128}, Hq/Hkv <= 32, max_pages and top <=
 * 16384, B*Hkv <= 65535, B*n*Hkv <= 2^24, num_pages*Hkv < 2^30 (else
 * EAGLE_ERR_UNSUPPORTED); 1 <= n <= 4096; 0 <= first, last; first + last <= top;
 * page rules as for eagle_tree_attn_paged; workspace 16-byte aligned. */
size_t eagle_kv8_select_workspace_size(int dtype, int B, int n, int Hq, int Hkv,
                                       int dh, int max_pages, int page_size);

int eagle_kv8_select(const void *q, int dtype, const uint8_t *k_bounds,
                     const float *k_scale, const int32_t *block_table,
                     int max_pages, int page_size, int num_pages,
                     const int32_t *kv_len, int B, int n, int Hq, int Hkv,
                     int dh, int top, int first, int last, int32_t *sel,
                     float *score, int32_t *status, void *workspace,
                     size_t workspace_bytes, eagle_stream_t stream);

/* eagle_tree_attn_kv8 with the prefix of node i and KV head g cut down to the pages
 * that sel[b, i, g] lists: the keys are the positions below kv_len[b] of those
 * pages and the tree nodes of the node's mask row.
 *   sel        device int32 [B, n, Hkv, top], as eagle_kv8_select writes it: logical
 *              pages, ascending, ended by a negative entry or by `top`
 *   status     as in eagle_tree_attn_kv8; EAGLE_ERR_INVALID also for a listed page
 *              at or past the prefix's end (it counts for nothing) and for one that
 *              does not ascend (the rows of that node and head are unspecified then;
 *              nothing is read out of range)
 * Everything else, what is rounded and a row without any key included, is as for
 * eagle_tree_attn_kv8.  A NaN of the cache reaches the rows of the nodes that list
 * its page; rows of other nodes of the same sequence and KV head may become NaN too,
 * where they share a kernel's tile with those.
 * Workspace: for many rows the union of the nodes' lists, and partial results.
 * Limits: those of eagle_tree_attn_kv8; Hq/Hkv <= 32 and B*n*Hkv <= 2^24 (else
 * EAGLE_ERR_UNSUPPORTED); top >= 1, top * page_size <= 2^24. */
size_t eagle_tree_attn_kv8_pages_workspace_size(int dtype, int B, int n, int Hq,
                                                int Hkv, int dh, int top,
                                                int max_pages, int page_size);

int eagle_tree_attn_kv8_pages(const void *q, const uint8_t *k_pages,
                              const uint8_t *v_pages, const float *k_scale,
                              const float *v_scale, const int32_t *block_table,
                              int max_pages, int page_size, int num_pages,
                              const int32_t *kv_len, const void *k_tree,
                              const void *v_tree, const uint64_t *mask,
                              const int32_t *sel, int top, int dtype, int B,
                              int n, int Hq, int Hkv, int dh, float scale,
                              void *out, float *lse, int32_t *status,
                              void *workspace, size_t workspace_bytes,
                              eagle_stream_t stream);

/* ------------------------------------------------------------------------
 * The whole step in one call, and as one recorded graph.
 * [EAGLE-2] section "動的ドラフトツリーの構築アルゴリズム" (draft confidences,
 * then the tree), [EAGLE-1] sections "Tree Attention の役割" (the target
 * scores the tree in one pass) and "検証方法" (then verification): the
 * stages run in that order, each on the previous one's results:
 *   eagle_draft_topk -> eagle_tree_build (with the mask) -> eagle_tree_attn
 *   -> eagle_verify
 * on one stream, each kernel chained to the previous one.  The target
 * logits are an input: the target's layers between the attention and its
 * logits are not part of the library.
 *
 * eagle_step_args names every buffer of the four calls; each field means
 * what the argument of the same name means there (n = m + 1 tree nodes):
 *   draft_logits, draft_ld            eagle_draft_topk's logits, ld
 *   tok, conf, stats                  its outputs (stats may be NULL)
 *   root_tok, node_tok ... node_row   eagle_tree_build's (root_tok,
 *                                     node_depth, node_score, node_src and
 *                                     node_row may be NULL)
 *   mask                              required: the attention reads it
 *   q, k_cache, v_cache, kv_len, k_tree, v_tree, scale, attn_out, lse
 *                                     eagle_tree_attn's (attn_out is its
 *                                     `out`; lse may be NULL)
 *   target, target_ld, uniforms, accept_len, path_nodes, out_tokens
 *                                     eagle_verify's (uniforms only for
 *                                     EAGLE_SAMPLE)
 *   status                            one word shared by every stage (may
 *                                     be NULL)
 * dtype applies to the draft logits, the attention tensors and the target
 * logits alike.
 * ------------------------------------------------------------------------ */
typedef struct eagle_step_args {
  int dtype;
  int B, D, k, m, V;
  int Hq, Hkv, dh, Lmax;
  int mode;
  float temperature;
  float scale;
  const void *draft_logits;
  int64_t draft_ld;
  int32_t *tok;
  float *conf;
  float *stats;
  const int32_t *root_tok;
  int32_t *node_tok, *node_parent, *node_depth;
  float *node_score;
  int32_t *node_src, *node_row;
  uint64_t *mask;
  const void *q, *k_cache, *v_cache;
  const int32_t *kv_len;
  const void *k_tree, *v_tree;
  void *attn_out;
  float *lse;
  const void *target;
  int64_t target_ld;
  const float *uniforms;
  int32_t *accept_len, *path_nodes, *out_tokens;
  int32_t *status;
} eagle_step_args;

/* Bytes of the one workspace a step needs (the stages' workspaces, each at
 * a 256-byte aligned offset); 0 for invalid arguments.  Host only. */
size_t eagle_step_workspace_size(const eagle_step_args *args);

/* The four calls in order on `stream`.  Returns the first nonzero status
 * of a call (the calls after it are not made); the arguments of each call
 * are checked by that call. */
int eagle_step(const eagle_step_args *args, void *workspace,
               size_t workspace_bytes, eagle_stream_t stream);

/* A step recorded once into a CUDA graph; each launch replays all of its
 * kernels with one call.  The graph holds the buffers' addresses (and the
 * tensor maps built from them), so every buffer and the workspace must stay
 * allocated, at the same address, until the graph is destroyed; their
 * contents (inputs, kv_len) may change between launches.
 * eagle_step_graph_create first runs the step once on a stream of its own
 * (work that produces the inputs on other streams must have completed) and
 * waits for it (one-time kernel set-up happens outside the recording; the
 * outputs are then those of that run), then records the step on that
 * stream (capture mode local to the calling thread) and instantiates the
 * graph.  Unlike the other calls it allocates (the stream and the graph)
 * and synchronises; the launches do neither.  On failure *graph is NULL.
 * Destroy a graph only after the launches made with it have completed. */
typedef struct eagle_step_graph_s *eagle_step_graph_t;

int eagle_step_graph_create(const eagle_step_args *args, void *workspace,
                            size_t workspace_bytes, eagle_step_graph_t *graph);
int eagle_step_graph_launch(eagle_step_graph_t graph, eagle_stream_t stream);
int eagle_step_graph_destroy(eagle_step_graph_t graph);

#ifdef __cplusplus
}
#endif

#endif /* EAGLE_H */
