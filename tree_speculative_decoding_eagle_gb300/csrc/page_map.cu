// Pages of a free list to requests and back: block tables and slot maps from
// the requests' lengths, without a host round trip.
//
// Per request b: pages wanted need_b = ceil((kv_len + new_len) / P), taken
// add_b = max(0, need_b - page_count_b).  The j-th page taken over all
// requests is free[free_count - 1 - j], so a request's first page follows from
// the exclusive sum of add_b, and a token's place from the exclusive sum of
// new_len: two prefix sums over at most 4096 requests, then independent writes
// for every new table entry and every token.
//
// What bounds it: latency.  One thread-block cluster (1 to 8 CTAs by the
// number of tokens); every CTA reads all lengths and makes the sums itself in
// shared memory (12 bytes a request, from L2 after the first), which
// costs less than handing them over, and then writes its share of the outputs.
// Measured, a map and a release together (two launches in a graph): 6.7 us for
// one request, 11.6 us for 512 requests with up to 32768 new tokens, whose 0.2
// MB would stream in 0.03 us: the chain is two launches, the lengths, two sums,
// a bisection and the free list's entries.
// Everything that is updated in place (page_count, free_count) is written only
// after a cluster barrier that every CTA reaches with its reads done.
#include "common.cuh"
#include "sm100.cuh"

namespace eagle {

using namespace sm100;

constexpr int kPageThreads = 1024;
constexpr int kPageTokensPerCta = 4096;  // four tokens a thread
constexpr int kPageMaxB = 4096;

struct PageArgs {
  const int32_t *kv_len, *new_len;  // release: keep_len, unused
  int B, log_page, max_pages, num_pages;
  int32_t *block_table, *page_count, *free_pages, *free_count;
  int32_t *slot_map, *new_start, *status;
  int T;
  int32_t *granted;  // map: with it a refusal is written out too
};

// Shared arrays, B (+ 1) entries each.
struct PageSmem {
  int32_t *kv, *count, *start, *first;
  __device__ explicit PageSmem(int32_t *p, int B) : kv(p), count(p + B), start(p + 2 * B), first(p + 3 * B + 1) {}
};
static size_t page_smem_bytes(int B) { return static_cast<size_t>(4 * B + 2) * sizeof(int32_t); }

// Exclusive sums of (x, y) over the CTA's 1024 threads, in thread order;
// returns the totals through tx, ty.  64 bits: 4096 requests of 2^24 tokens
// pass 2^32.
__device__ __forceinline__ void block_exclusive_sum2(int64_t &x, int64_t &y, int64_t &tx, int64_t &ty,
                                                     int64_t (*part)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t x0 = x, y0 = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t ax = __shfl_up_sync(0xffffffffu, x, o), ay = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) { x += ax; y += ay; }
  }
  if (lane == 31) { part[warp][0] = x; part[warp][1] = y; }
  __syncthreads();
  int64_t px = part[lane][0], py = part[lane][1];  // 32 warps
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t ax = __shfl_up_sync(0xffffffffu, px, o), ay = __shfl_up_sync(0xffffffffu, py, o);
    if (lane >= o) { px += ax; py += ay; }
  }
  const int64_t bx = __shfl_sync(0xffffffffu, px, warp ? warp - 1 : 0), by = __shfl_sync(0xffffffffu, py, warp ? warp - 1 : 0);
  tx = __shfl_sync(0xffffffffu, px, 31);
  ty = __shfl_sync(0xffffffffu, py, 31);
  x = x - x0 + (warp ? bx : 0);
  y = y - y0 + (warp ? by : 0);
  __syncthreads();  // part may be reused
}

// Largest b in [0, B) with start[b] <= t (start ascending, start[0] = 0, t
// below the total): empty requests never win against the next one.
__device__ __forceinline__ int owner_of(const int32_t *start, int B, int t) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPageThreads) page_map_kernel(PageArgs a) {
  extern __shared__ int32_t page_smem[];
  __shared__ int64_t part[32][2];
  __shared__ int bad_s;
  const PageSmem s(page_smem, a.B);
  const int tid = threadIdx.x, rank = blockIdx.x, ctas = gridDim.x;
  const int P = 1 << a.log_page;
  if (tid == 0) bad_s = 0;
  pdl_wait();
  const int fc = *a.free_count;
  __syncthreads();
  int64_t tokens = 0, pages = 0;
  bool bad = fc < 0 || fc > a.num_pages;
  for (int b0 = 0; b0 < a.B; b0 += kPageThreads) {
    const int b = b0 + tid;
    int kv = 0, nw = 0, cnt = 0;
    if (b < a.B) {
      kv = a.kv_len[b];
      nw = a.new_len[b];
      cnt = a.page_count[b];
      if (kv < 0 || nw < 0 || cnt < 0 || cnt > a.max_pages ||
          static_cast<int64_t>(kv) + nw > (static_cast<int64_t>(a.max_pages) << a.log_page)) {
        bad = true;
        kv = nw = cnt = 0;
      }
    }
    const int need = (kv + nw + P - 1) >> a.log_page;
    int64_t x = nw, y = max(0, need - cnt), tx, ty;
    block_exclusive_sum2(x, y, tx, ty, part);
    if (b < a.B) {
      s.kv[b] = kv;
      s.count[b] = cnt;
      // beyond T or the free list nothing is written: the clamp only keeps 32 bits
      s.start[b] = static_cast<int32_t>(min(tokens + x, static_cast<int64_t>(INT32_MAX)));
      s.first[b] = static_cast<int32_t>(min(pages + y, static_cast<int64_t>(INT32_MAX)));
    }
    tokens += tx;
    pages += ty;
  }
  if (bad) bad_s = 1;
  if (tid == 0) {
    s.start[a.B] = static_cast<int32_t>(min(tokens, static_cast<int64_t>(INT32_MAX)));
    s.first[a.B] = static_cast<int32_t>(min(pages, static_cast<int64_t>(INT32_MAX)));
  }
  __syncthreads();
  int err = 0;
  if (bad_s || (a.slot_map && tokens > a.T) || tokens > INT32_MAX) err = EAGLE_ERR_INVALID;
  else if (pages > fc) err = EAGLE_ERR_PAGES;
  // every CTA's reads of page_count and free_count are done
  if (ctas > 1) {
    cluster_arrive_release();
    cluster_wait();
  }
  pdl_trigger();
  if (err) {  // the same in every CTA
    if (rank == 0 && tid == 0) report(a.status, err);
    if (a.granted) {  // nothing granted: no slot, no token
      for (int t = rank * kPageThreads + tid; t < a.T; t += ctas * kPageThreads) a.slot_map[t] = -1;
      if (a.new_start)
        for (int b = rank * kPageThreads + tid; b <= a.B; b += ctas * kPageThreads) a.new_start[b] = 0;
      if (rank == 0 && tid == 0) *a.granted = 0;
    }
    return;
  }
  // new table entries, and the requests' own words
  bool lost = false;  // a page number outside the pool
  for (int j = rank * kPageThreads + tid; j < pages; j += ctas * kPageThreads) {
    const int b = owner_of(s.first, a.B, j), page = a.free_pages[fc - 1 - j];
    const bool ok = page >= 0 && page < a.num_pages;
    lost |= !ok;
    a.block_table[static_cast<int64_t>(b) * a.max_pages + s.count[b] + (j - s.first[b])] = ok ? page : -1;
  }
  for (int b = rank * kPageThreads + tid; b < a.B; b += ctas * kPageThreads) {
    const int add = s.first[b + 1] - s.first[b];
    if (add) a.page_count[b] = s.count[b] + add;
    if (a.new_start) a.new_start[b] = s.start[b];
  }
  if (rank == 0 && tid == 0) {
    if (pages) *a.free_count = fc - static_cast<int>(pages);
    if (a.new_start) a.new_start[a.B] = static_cast<int32_t>(tokens);
    if (a.granted) *a.granted = 1;
  }
  // slots: a thread takes four neighbouring tokens, finds the first one's
  // request by bisection and walks on from there
  const int n_tok = static_cast<int>(tokens);
  for (int t0 = (rank * kPageThreads + tid) * 4; t0 < a.T; t0 += ctas * kPageThreads * 4) {
    int b = t0 < n_tok ? owner_of(s.start, a.B, t0) : 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int t = t0 + u;
      if (t >= a.T) break;
      int slot = -1;
      if (t < n_tok) {
        while (t >= s.start[b + 1]) ++b;
        const int pos = s.kv[b] + (t - s.start[b]);
        const int lp = pos >> a.log_page;
        const int page = lp < s.count[b] ? a.block_table[static_cast<int64_t>(b) * a.max_pages + lp]
                                         : a.free_pages[fc - 1 - (s.first[b] + lp - s.count[b])];
        if (page >= 0 && page < a.num_pages) slot = (page << a.log_page) + (pos & (P - 1));
        else lost = true;
      }
      a.slot_map[t] = slot;
    }
  }
  if (lost) report(a.status, EAGLE_ERR_INVALID);
}

// R pages to the free list, U a thread at a time.  Every page number is looked at
// before the first is handed on; a thread's first U stay in registers meanwhile.
// False (and nothing written) where one is no page; the same in every thread.
template <int U>
__device__ __forceinline__ bool give_back(const PageArgs &a, const PageSmem &s, int fc, int R) {
  const int tid = threadIdx.x;
  const auto entry_of = [&](int j) {
    const int b = owner_of(s.first, a.B, j);
    return a.block_table + static_cast<int64_t>(b) * a.max_pages + s.kv[b] + (j - s.first[b]);
  };
  int32_t *entry[U];
  int page[U];
  bool lost = false;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int j = tid + u * kPageThreads;
    entry[u] = j < R ? entry_of(j) : nullptr;
    page[u] = entry[u] ? *entry[u] : 0;
  }
#pragma unroll
  for (int u = 0; u < U; ++u) lost |= page[u] < 0 || page[u] >= a.num_pages;
  if (U > 1)
    for (int j = tid + U * kPageThreads; j < R; j += kPageThreads) {
      const int p = *entry_of(j);
      lost |= p < 0 || p >= a.num_pages;
    }
  if (__syncthreads_or(lost)) {
    if (tid == 0) report(a.status, EAGLE_ERR_INVALID);
    return false;
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (entry[u]) {
      a.free_pages[fc + R - 1 - (tid + u * kPageThreads)] = page[u];
      *entry[u] = -1;
    }
  if (U > 1)
    for (int j = tid + U * kPageThreads; j < R; j += kPageThreads) {
      int32_t *e = entry_of(j);
      a.free_pages[fc + R - 1 - j] = *e;
      *e = -1;
    }
  return true;
}

// Gives pages back.  One CTA: a step returns a handful, and the largest
// release is one word read and two written a page.
__global__ void __launch_bounds__(kPageThreads) page_release_kernel(PageArgs a) {
  extern __shared__ int32_t page_smem[];
  __shared__ int64_t part[32][2];
  __shared__ int bad_s;
  const PageSmem s(page_smem, a.B);  // kv: pages kept, first: exclusive sums of pages given back
  const int tid = threadIdx.x;
  const int P = 1 << a.log_page;
  if (tid == 0) bad_s = 0;
  pdl_wait();
  const int fc = *a.free_count;
  __syncthreads();
  int64_t pages = 0;
  bool bad = fc < 0;
  for (int b0 = 0; b0 < a.B; b0 += kPageThreads) {
    const int b = b0 + tid;
    int keep = 0, cnt = 0;
    if (b < a.B) {
      const int len = a.kv_len[b];
      cnt = a.page_count[b];
      if (cnt < 0 || cnt > a.max_pages) { bad = true; cnt = 0; }
      keep = len < 0 ? cnt : min(cnt, static_cast<int>((static_cast<int64_t>(len) + P - 1) >> a.log_page));
    }
    int64_t x = 0, y = cnt - keep, tx, ty;
    block_exclusive_sum2(x, y, tx, ty, part);
    if (b < a.B) {
      s.kv[b] = keep;
      s.count[b] = cnt;
      s.first[b] = static_cast<int32_t>(min(pages + y, static_cast<int64_t>(INT32_MAX)));
    }
    pages += ty;
  }
  if (bad) bad_s = 1;
  __syncthreads();
  pdl_trigger();
  if (bad_s || fc + pages > a.num_pages) {
    if (tid == 0) report(a.status, EAGLE_ERR_INVALID);
    return;
  }
  const int R = static_cast<int>(pages);
  // a step's release in few instructions: they come from memory too (6.7 us against 7.1 with a map)
  if (!(R <= kPageThreads ? give_back<1>(a, s, fc, R) : give_back<4>(a, s, fc, R))) return;
  for (int b = tid; b < a.B; b += kPageThreads)
    if (s.count[b] != s.kv[b]) a.page_count[b] = s.kv[b];
  if (tid == 0 && R) *a.free_count = fc + R;
}

static int log2_of(int p) {
  int l = 0;
  while ((1 << l) < p) ++l;
  return l;
}

cudaError_t launch_page_map(const int32_t *kv_len, const int32_t *new_len, int B, int page_size, int max_pages,
                            int num_pages, int32_t *block_table, int32_t *page_count, const int32_t *free_pages,
                            int32_t *free_count, int32_t *slot_map, int T, int32_t *new_start, int32_t *granted,
                            int32_t *status, cudaStream_t st) {
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = set_smem_limit_once(page_map_kernel, static_cast<int>(page_smem_bytes(kPageMaxB)), configured);
  if (e != cudaSuccess) return e;
  PageArgs a = {kv_len, new_len, B, log2_of(page_size), max_pages, num_pages, block_table, page_count,
                const_cast<int32_t *>(free_pages), free_count, slot_map, new_start, status, T, granted};
  int ctas = 1;
  while (ctas < 8 && ctas * kPageTokensPerCta < T) ctas *= 2;
  return launch_chained_cluster(page_map_kernel, dim3(ctas), dim3(kPageThreads), page_smem_bytes(B), st, ctas, a);
}

cudaError_t launch_page_release(const int32_t *keep_len, int B, int page_size, int max_pages, int num_pages,
                                int32_t *block_table, int32_t *page_count, int32_t *free_pages, int32_t *free_count,
                                int32_t *status, cudaStream_t st) {
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = set_smem_limit_once(page_release_kernel, static_cast<int>(page_smem_bytes(kPageMaxB)), configured);
  if (e != cudaSuccess) return e;
  PageArgs a = {keep_len, nullptr, B, log2_of(page_size), max_pages, num_pages, block_table, page_count,
                free_pages, free_count, nullptr, nullptr, status, 0, nullptr};
  return launch_chained(page_release_kernel, dim3(1), dim3(kPageThreads), page_smem_bytes(B), st, a);
}

}  // namespace eagle
