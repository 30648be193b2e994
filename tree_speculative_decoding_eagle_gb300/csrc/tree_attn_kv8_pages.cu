// Attention over selected pages of the 8-bit cache: the prefix of node i and KV head
// g is the pages that its list names.
//
// Few query rows a KV head (single tokens, small trees): a node and KV head is taken
// as a sequence of its own, its rows the grouped heads, its block table the list
// (tree_attn_kv8_tokens.cu up to eight heads, the few-row kernel beyond: 64 tokens, 64
// heads on 4 of 128, 32 pages of 64 43 us, 134 MB, 46 % of the copy rate).
//
// Many rows (trees, prompt chunks): nodes of one tree choose much the same pages, and
// a key tile costs the tensor-core kernel the same for one row and for 256.  So a
// first kernel makes, for each M-group of query rows, the ascending list of the pages
// that any of its nodes names, and for each node a bit a listed page; the kernel of
// tree_attn_kv8_kernel.cuh then runs over that list as it does over a prefix, and a
// row gives the keys of pages without its bit weights of 2^-inf.
// What that gains depends on the nodes of a group and on how far they agree, which is
// known on the device alone: figures at kListRows.  Where no two nodes share a page
// and the lists together are the prefix, lists cost more than the attention to all of
// it: 285 against 277 us for 16 x 49 nodes, 28 against 22 for one such tree with 132 pages
// of 16, at the worst measured 77 against 44 (256 nodes, 1024 pages of 16).
//
// What bounds the attention over lists: each M-tile's chain S - softmax - P - O, as
// for a whole prefix, although two fifths of the warps have no row that counts a page
// of the tile (issue slots 44 %, tensor pipe 41 % of active cycles), and the last wave.
// Measured, on the device, lists included: 16 x 49 nodes, 64 heads on 8 of 128, 16 of 64
// to 128 pages of 64 126 us (a group lists 45 and 40; the lists take 5; 219 with every node
// a sequence of its own); 64 x 61 nodes, 64 heads on 8 of 64, 8 of 64 pages of 128 323
// us (a group lists 24; 829; the whole prefix 690).  An M-tile that passes over the tiles
// it does not count (a fifth and a seventh of them) makes the roles' hand-overs
// irregular: 150 and 380 us.
#include "tree_attn_kv8_kernel.cuh"

namespace eagle {

// tree_attn_kv8_few.cu
size_t attn_kv8_few_workspace_bytes(int B, int n, int Hq, int Hkv, int dh, int Lmax, int num_sms);
cudaError_t launch_tree_attn_kv8_pages_few(const Kv8SelArgs &a, const void *k_pages, const void *v_pages, int dh, int Lmax, void *ws,
                                           int num_sms, cudaStream_t st);

// tree_attn_kv8_tokens.cu
size_t attn_kv8_tokens_workspace_bytes(int64_t nodes, int Hkv, int dh, int positions, int num_sms);
cudaError_t launch_tree_attn_kv8_tokens(Kv8SelArgs a, const void *k_pages, const void *v_pages, int dh, int positions, void *ws,
                                        int num_sms, cudaStream_t st);

constexpr int kUnionPages = 16384;  // pages of a request that a group's map holds
constexpr int kUnionWarps = 8;
// Query rows of a KV head from which nodes share lists: more than a CTA of the
// few-row kernel holds.  Measured (us on the device, lists / every node alone by
// tree_attn_kv8_tokens.cu; nodes that agree, half agree, share nothing), 512 heads of
// sequences in all, 8192 keys:
//   dh 128, 16 pages of 64:  5 nodes of 8 heads 81 / 95, 139 / 96, 266 / 119; 9 of 8 108 / 162,
//     195 / 163, 497 / 181; 10 of 4 82 / 174, 164 / 174, 420 / 185; 40 of 1 89 / 663, 219 / 663,
//     447 / 666; 49 of 8 (128 heads) 72 / 221, 140 / 221, 285 / 221
//   dh 64, 8 pages of 128:   5 of 8 67 / 79, 116 / 80, 223 / 82; 9 of 8 70 / 130, 138 / 131,
//     343 / 134; 10 of 4 68 / 141, 144 / 142, 354 / 144; 40 of 1 75 / 534, 190 / 534, 379 / 535;
//     61 of 8 174 / 824, 351 / 824, 716 / 824
// So lists win for nodes that agree, and for many nodes whether they do or not; five to
// ten nodes of 4 or 8 heads that half agree or less are faster alone, which this rule on
// rows does not see.
constexpr int kListRows = 33;

struct UnionArgs {
  const int32_t *sel, *block_table, *kv_len;
  int32_t *lens, *pages, *status;
  uint32_t *bits;
  int n, Hkv, G, top, group_rows, group_nodes, list_stride, bit_words;
  int log_page, max_pages, num_pages;
};

// One CTA per (M-group, (sequence, KV head)).
__global__ void __launch_bounds__(kUnionWarps * 32) kv8_union_kernel(UnionArgs a) {
  constexpr int WORDS = kUnionPages / 32;
  __shared__ uint32_t map[WORDS];                   // a bit a page of the request
  __shared__ int before[WORDS];                     // pages of the words before
  __shared__ uint32_t row_words[kUnionWarps][WORDS];
  __shared__ int part[kUnionWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bg = blockIdx.y, b = bg / a.Hkv, g = bg % a.Hkv;
  const int64_t cl = static_cast<int64_t>(bg) * gridDim.x + blockIdx.x;
  const int r0 = blockIdx.x * a.group_rows, i0 = r0 / a.G, i1 = (min(a.n * a.G, r0 + a.group_rows) - 1) / a.G;
  const int P = 1 << a.log_page;
  for (int w = tid; w < WORDS; w += kUnionWarps * 32) map[w] = 0;
  pdl_wait();
  const int L = static_cast<int>(min(static_cast<int64_t>(max(a.kv_len[b], 0)), static_cast<int64_t>(a.max_pages) << a.log_page));
  const int live = (L + P - 1) >> a.log_page;
  __syncthreads();
  // A node's entries, 32 at a time, up to its first negative one: `with` gets the page
  // of each that is one of the prefix's (-1 in the other lanes); the whole warp calls it.
  const auto entries_of = [&](int i, auto with, bool tell) {
    const int32_t *list = a.sel + ((static_cast<int64_t>(b) * a.n + i) * a.Hkv + g) * a.top;
    int last = -1;
    for (int c = 0; c < a.top; c += 32) {
      const int page = c + lane < a.top ? list[c + lane] : -1;
      const uint32_t on = __ballot_sync(0xffffffffu, page >= 0);
      const int count = on == 0xffffffffu ? 32 : __ffs(~on) - 1;
      const int prev = __shfl_up_sync(0xffffffffu, page, 1);
      const bool mine = lane < count;
      if (tell && mine && (page >= live || page <= (lane ? prev : last))) report(a.status, EAGLE_ERR_INVALID);
      with(mine && page < live ? page : -1);
      last = __shfl_sync(0xffffffffu, page, 31);
      if (count < 32) break;
    }
  };
  for (int i = i0 + warp; i <= i1; i += kUnionWarps)
    entries_of(i, [&](int page) { if (page >= 0) atomicOr(&map[page >> 5], 1u << (page & 31)); }, true);
  __syncthreads();
  // places: two words a thread
  int count[2], sum = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    count[k] = __popc(map[2 * tid + k]);
    sum += count[k];
  }
  int x = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) part[warp] = x;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kUnionWarps; ++w) {
    if (w < warp) x += part[w];
    total += part[w];
  }
  before[2 * tid] = x - sum;
  before[2 * tid + 1] = x - count[1];
  __syncthreads();
  const auto place_of = [&](int page) { return before[page >> 5] + __popc(map[page >> 5] & ((1u << (page & 31)) - 1u)); };
  for (int p = tid; p < live; p += kUnionWarps * 32) {
    if (!((map[p >> 5] >> (p & 31)) & 1u)) continue;
    const int place = place_of(p);
    int page = a.block_table[static_cast<int64_t>(b) * a.max_pages + p];
    if (page < 0 || page >= a.num_pages) {
      report(a.status, EAGLE_ERR_INVALID);  // outside the pool: read page 0
      page = 0;
    }
    a.pages[cl * a.list_stride + place] = page;
    if (place == total - 1) a.lens[cl] = ((total - 1) << a.log_page) + min(P, L - (p << a.log_page));
  }
  if (total == 0 && tid == 0) a.lens[cl] = 0;
  const int row = (total + 31) >> 5;
  for (int i = i0 + warp; i <= i1; i += kUnionWarps) {
    for (int w = lane; w < row; w += 32) row_words[warp][w] = 0;
    __syncwarp();
    entries_of(i, [&](int page) {
      if (page >= 0) {
        const int place = place_of(page);
        atomicOr(&row_words[warp][place >> 5], 1u << (place & 31));
      }
    }, false);
    __syncwarp();
    uint32_t *dst = a.bits + (cl * a.group_nodes + (i - i0)) * a.bit_words;
    for (int w = lane; w < row; w += 32) dst[w] = row_words[warp][w];
    __syncwarp();
  }
}

// Positions a node's list holds at most.
static int listed_positions(int top, int max_pages, int page_size) { return (top < max_pages ? top : max_pages) * page_size; }

struct ListPlan {
  bool lists;
  Kv8Plan p;
  int group_nodes, list_stride, bit_words;
  size_t pages_off, bits_off, part_off, bytes;
};

static ListPlan list_plan(int B, int n, int Hq, int Hkv, int dh, int top, int max_pages, int page_size, int num_sms) {
  ListPlan l = {};
  const int G = Hq / Hkv, rows = n * G;
  l.lists = rows >= kListRows && max_pages <= kUnionPages;
  if (!l.lists) {
    const int positions = listed_positions(top, max_pages, page_size);
    l.bytes = G <= 8 ? attn_kv8_tokens_workspace_bytes(static_cast<int64_t>(B) * n, Hkv, dh, positions, num_sms)
                     : attn_kv8_few_workspace_bytes(B * n, 1, Hq, Hkv, dh, positions, num_sms);
    return l;
  }
  // The lists' lengths are known on the device alone.  Where the groups fill the SMs,
  // the KV split is chosen for groups whose nodes name twice what one of them does, else
  // for the longest list there can be: SMs that idle cost nothing, and nodes that share
  // no page would leave each group alone with a long list.  Measured (us on the device,
  // chosen by twice one node's / by the longest; nodes that agree, half agree, share
  // nothing): 49 nodes of 64 heads on 8 of 128, 4 of 132 pages of 16 19 / 23, 26 / 24,
  // 51 / 28; 61 nodes, 32 heads with keys of their own, 4 of 256 pages 18 / 27, 31 / 29,
  // 92 / 43; 256 nodes, 8 heads of 64, 8 of 1024 pages of 16 44 / 45, 71 / 50, 271 / 77.
  const int64_t guess = min(static_cast<int64_t>(max_pages), static_cast<int64_t>(2) * top);
  l.p = kv8_plan(B, n, Hq, Hkv, dh, static_cast<int>(guess * page_size), num_sms);
  const int group_rows = l.p.MT * 128;
  l.group_nodes = min(n, (group_rows + G - 2) / G + 1);
  l.list_stride = static_cast<int>(min(static_cast<int64_t>(max_pages), static_cast<int64_t>(l.group_nodes) * top));
  l.bit_words = (l.list_stride + 31) / 32;
  const size_t groups = static_cast<size_t>(B) * Hkv * l.p.mgroups;
  if (groups < static_cast<size_t>(num_sms) * l.p.ctas_per_sm)
    l.p = kv8_plan(B, n, Hq, Hkv, dh, l.list_stride * page_size, num_sms);
  const auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  l.pages_off = up(groups * sizeof(int32_t));
  l.bits_off = l.pages_off + up(groups * l.list_stride * sizeof(int32_t));
  l.part_off = l.bits_off + up(groups * l.group_nodes * l.bit_words * sizeof(uint32_t));
  l.bytes = l.part_off;
  if (l.p.S > 1) l.bytes += groups * l.p.S * kv8_slot_rows(l.p, rows) * (dh + 2) * sizeof(float);
  return l;
}

size_t attn_kv8_pages_workspace_bytes(int B, int n, int Hq, int Hkv, int dh, int top, int max_pages, int page_size, int num_sms) {
  return list_plan(B, n, Hq, Hkv, dh, top, max_pages, page_size, num_sms).bytes;
}

cudaError_t launch_tree_attn_kv8_pages(const void *q, const uint8_t *k_pages, const uint8_t *v_pages, const float *k_scale,
                                       const float *v_scale, const int32_t *block_table, int max_pages, int page_size,
                                       int num_pages, const int32_t *kv_len, const void *k_tree, const void *v_tree,
                                       const uint64_t *mask, const int32_t *sel, int top, int B, int n, int Hq, int Hkv,
                                       int dh, float scale, void *out, float *lse, void *ws, int32_t *status, int num_sms,
                                       cudaStream_t st) {
  const ListPlan l = list_plan(B, n, Hq, Hkv, dh, top, max_pages, page_size, num_sms);
  Kv8Args a = {};
  a.q = reinterpret_cast<const __nv_bfloat16 *>(q);
  a.k_tree = reinterpret_cast<const __nv_bfloat16 *>(k_tree);
  a.v_tree = reinterpret_cast<const __nv_bfloat16 *>(v_tree);
  a.k_scale = k_scale; a.v_scale = v_scale;
  a.block_table = block_table; a.kv_len = kv_len; a.mask = mask;
  a.B = B; a.n = n; a.Hq = Hq; a.Hkv = Hkv; a.G = Hq / Hkv; a.W = (n + 63) / 64;
  a.page_size = page_size; a.max_pages = max_pages; a.num_pages = num_pages;
  while ((1 << a.log_page) < page_size) ++a.log_page;
  a.scale_log2 = scale * kLog2e;
  a.out = reinterpret_cast<__nv_bfloat16 *>(out);
  a.lse = lse; a.status = status;
  if (!l.lists) {
    Kv8SelArgs s;
    static_cast<Kv8Args &>(s) = a;
    s.B = B * n; s.n = 1;
    s.sel = sel; s.top = top; s.nodes = n;
    const int positions = listed_positions(top, max_pages, page_size);
    return a.G <= 8 ? launch_tree_attn_kv8_tokens(s, k_pages, v_pages, dh, positions, ws, num_sms, st)
                    : launch_tree_attn_kv8_pages_few(s, k_pages, v_pages, dh, positions, ws, num_sms, st);
  }
  if (!ws) return cudaErrorInvalidValue;
  unsigned char *base = reinterpret_cast<unsigned char *>(ws);
  const UnionArgs u = {sel, block_table, kv_len, reinterpret_cast<int32_t *>(base), reinterpret_cast<int32_t *>(base + l.pages_off),
                       status, reinterpret_cast<uint32_t *>(base + l.bits_off), n, Hkv, a.G, top, l.p.MT * 128, l.group_nodes,
                       l.list_stride, l.bit_words, a.log_page, max_pages, num_pages};
  const cudaError_t e = launch_chained(kv8_union_kernel, dim3(l.p.mgroups, B * Hkv), dim3(kUnionWarps * 32), 0, st, u);
  if (e != cudaSuccess) return e;
  Kv8UnionArgs t;
  static_cast<Kv8Args &>(t) = a;
  t.lens = u.lens; t.pages = u.pages; t.bits = u.bits;
  t.list_stride = l.list_stride; t.group_nodes = l.group_nodes; t.bit_words = l.bit_words;
  return launch_kv8<true>(t, k_pages, v_pages, dh, l.p, base + l.part_off, st);
}

}  // namespace eagle
