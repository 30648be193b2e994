// The pages of the 8-bit cache that a query is to attend to: for each node, KV head
// and page the greatest product that the page's bounds allow with the query rounded to
// 8 bits, and the `top` pages with the greatest.
//
// A query row (node i, head h) is taken as whole numbers q' = rint(q 2^-e), e the
// power of two that puts its largest magnitude into [64, 128], |q'| <= 128.  With
// the bounds lo, hi of a page's columns (multiples of 1/2 up to 448, kv8_bounds.cu)
//   u = sum_c max(q'_c, 0) hi_c + min(q'_c, 0) lo_c
// is a sum of at most 128 multiples of 1/2 up to 128 * 448: below 2^23, so a float32
// sum of it is exact whatever its order.  The score u 2^(e + page scale's exponent)
// is exact too, and the pages chosen for a query over one prefix are the same in a
// tree, alone, in any batch and on any launch shape.  (A token decoded after its
// path has been stored has another prefix: its list is the same while `last` >= 1
// and the path stays in the prefix's last page.)
// The node's score of a page is the largest over the heads that share the KV head.
//
// Two kernels.  Scores: kv8_score.cu.  Choice (here): a row's scores as ordered
// 32-bit keys in registers, a search by halving for the greatest key that `top` of
// them reach, ties to the lower pages, places by votes.
// What bounds the choice: issue slots with many rows (6272 rows of 512 scores 15 us alone
// with cold caches, ALU 51 % of active cycles), latency with few (512 rows of up to 2048
// scores 10.6 us, 32 rows 8.8).  Both kernels, one after another on the device: 39.4,
// 47.6 and 15.1 us.  Launching the choice as soon as the scores' last CTAs run gains nothing
// (47.5 -> 51 us: its CTAs wait in the way).
#include "kv8_select.cuh"

namespace eagle {

// T threads (32, or whole CTAs of 128 and more) a row; a warp takes 32 V neighbouring
// pages, lane by lane, so that a vote gives the places of 32 of them.
template <int T, int V>
__global__ void __launch_bounds__(T < 128 ? 64 : T, T < 128 ? 20 : 1) kv8_choose_kernel(SelectArgs a, int row_count) {
  constexpr int THREADS = T < 128 ? 64 : T, WARPS = T / 32;
  __shared__ int part[2][THREADS / 32];
  const int lane = threadIdx.x & 31, warp = (threadIdx.x % T) >> 5;
  const int row = blockIdx.x * (THREADS / T) + threadIdx.x / T;  // B * n * Hkv is at most 2^24
  pdl_wait();
  pdl_trigger();
  if (row >= row_count) return;  // whole warps: T < 128 has one warp a row
  const int b = static_cast<uint32_t>(row) / static_cast<uint32_t>(a.n * a.Hkv);
  const int np = live_pages(a, b), K = min(a.top, np);
  const int p0 = warp * 32 * V + lane;  // this lane's pages: p0, p0 + 32, ..
  const float *src = a.scores + static_cast<int64_t>(row) * a.stride + p0;
  int turn = 0;
  const auto row_sum = [&](int x) {  // over the row's threads
    x = __reduce_add_sync(0xffffffffu, x);
    if constexpr (WARPS > 1) {
      if (lane == 0) part[turn][warp] = x;
      __syncthreads();
      x = __reduce_add_sync(0xffffffffu, lane < WARPS ? part[turn][lane] : 0);
      turn ^= 1;  // the next sum's words: those of the one before have been read by then
    }
    return x;
  };
  uint32_t key[V];  // 0 past the prefix, the greatest number where a page is selected without its score
#pragma unroll
  for (int j = 0; j < V; ++j) key[j] = p0 + 32 * j < np ? __float_as_uint(src[32 * j]) : 0u;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int at = p0 + 32 * j;
    // (a score is finite unless the bounds hold NaN; its key stays between the two)
    const uint32_t by_score = min(max(ordered_u32(__uint_as_float(key[j])), 1u), 0xfffffffeu);
    key[j] = at >= np ? 0u : (at < a.first || at >= np - a.last) ? 0xffffffffu : by_score;
  }
  // The greatest key that at least K of them reach: count(lo) >= K > count(hi).
  uint32_t lo = 1u, hi = 0xffffffffu;
  int reach = np;
  if (K < np) {
    const auto count = [&](uint32_t bar) {
      int c = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) c += key[j] >= bar;
      return row_sum(c);
    };
    const int forced = min(np, a.first + a.last);  // below K where K < np and first + last < top
    if (forced >= K) {
      lo = hi;
      reach = count(hi);
    } else {
      // the least and the greatest key without the forced ones
      uint32_t least = 0xffffffffu, most = 0u;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        least = min(least, key[j] - 1u);  // no page: the greatest number
        most = max(most, key[j] + 1u);    // forced: 0
      }
      least = __reduce_min_sync(0xffffffffu, least);
      most = __reduce_max_sync(0xffffffffu, most);
      if constexpr (WARPS > 1) {
        if (lane == 0) { part[0][warp] = static_cast<int>(least); part[1][warp] = static_cast<int>(most); }
        __syncthreads();
        least = __reduce_min_sync(0xffffffffu, lane < WARPS ? static_cast<uint32_t>(part[0][lane]) : 0xffffffffu);
        most = __reduce_max_sync(0xffffffffu, lane < WARPS ? static_cast<uint32_t>(part[1][lane]) : 0u);
        __syncthreads();
      }
      lo = least + 1u;  // all reach it
      hi = most;        // the forced ones alone do
      // 7 halvings on average for 16 of 512 pages, 9 for 32 of 2048 (12 and 13 by
      // interpolation on the counts: the greatest scores lie far apart)
      while (reach != K && hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        const int c = count(mid);
        if (c >= K) {
          lo = mid;
          reach = c;
        } else {
          hi = mid;
        }
      }
    }
  }
  int32_t *dst = a.sel + static_cast<int64_t>(row) * a.top;
  float *dst_s = a.sel_score ? a.sel_score + static_cast<int64_t>(row) * a.top : nullptr;
  const uint32_t below = (1u << lane) - 1u;
  const auto take = [&](int at, int j) {
    dst[at] = p0 + 32 * j;
    if (dst_s) dst_s[at] = src[32 * j];  // again: a few of many
  };
  // of the warps before this one (whole CTAs only)
  const auto before = [&](int x) {
    if constexpr (WARPS > 1) {
      x = __reduce_add_sync(0xffffffffu, x);
      __syncthreads();
      if (lane == 0) part[0][warp] = x;
      __syncthreads();
      return __reduce_add_sync(0xffffffffu, lane < warp ? part[0][lane] : 0);
    }
    return 0;
  };
  if (reach == K) {
    int mine = 0, place = 0;
    if constexpr (WARPS > 1) {
#pragma unroll
      for (int j = 0; j < V; ++j) mine += key[j] >= lo;
      place = before(mine);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t on = __ballot_sync(0xffffffffu, key[j] >= lo);
      if (!on) continue;
      if (key[j] >= lo) take(place + __popc(on & below), j);
      place += __popc(on);
    }
  } else {  // all that pass lo and, of those equal to it, the first `ties`
    int greater = 0, equal = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      greater += key[j] > lo;
      equal += key[j] == lo;
    }
    const int ties = K - row_sum(greater);
    int tied = before(equal), place = before(greater) + min(tied, ties);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const uint32_t eq = __ballot_sync(0xffffffffu, key[j] == lo);
      const bool mine = key[j] > lo || (key[j] == lo && tied + __popc(eq & below) < ties);
      const uint32_t on = __ballot_sync(0xffffffffu, mine);
      if (mine) take(place + __popc(on & below), j);
      place += __popc(on);
      tied += __popc(eq);
    }
  }
  for (int i = K + warp * 32 + lane; i < a.top; i += T) {
    dst[i] = -1;
    if (dst_s) dst_s[i] = -INFINITY;
  }
}

// Floats of a row of scores: whole steps of eight pages.
static int score_stride(int max_pages) { return (max_pages + 7) / 8 * 8; }

size_t kv8_select_workspace_bytes(int B, int n, int Hkv, int max_pages) {
  return static_cast<size_t>(B) * n * Hkv * score_stride(max_pages) * sizeof(float);
}

template <int T, int V>
static cudaError_t launch_choose(const SelectArgs &a, cudaStream_t st) {
  constexpr int THREADS = T < 128 ? 64 : T;
  const int rows = a.B * a.n * a.Hkv, per_cta = THREADS / T;
  const dim3 grid((rows + per_cta - 1) / per_cta);
  return launch_chained(kv8_choose_kernel<T, V>, grid, dim3(THREADS), 0, st, a, rows);
}

// kv8_score.cu
cudaError_t launch_kv8_score(const SelectArgs &a, int dh, int num_sms, cudaStream_t st);

cudaError_t launch_kv8_select(const void *q, const uint8_t *bounds, const float *k_scale, const int32_t *block_table,
                              int max_pages, int page_size, int num_pages, const int32_t *kv_len, int B, int n, int Hq,
                              int Hkv, int dh, int top, int first, int last, int32_t *sel, float *score, void *ws,
                              int32_t *status, int num_sms, cudaStream_t st) {
  int log_page = 0, log_g = 0;
  while ((1 << log_page) < page_size) ++log_page;
  while ((1 << log_g) < Hq / Hkv) ++log_g;
  const SelectArgs a = {reinterpret_cast<const __nv_bfloat16 *>(q), bounds, k_scale, block_table, kv_len,
                        reinterpret_cast<float *>(ws), sel, score, status, B, n, Hq, Hkv, Hq / Hkv, log_g,
                        log_page, max_pages, num_pages, score_stride(max_pages), top, first, last};
  const cudaError_t e = launch_kv8_score(a, dh, num_sms, st);
  if (e != cudaSuccess) return e;
  // by what the threads' registers hold (16 keys each).  The table's width decides, as
  // the host knows it: 64 tokens of 8 KV heads with 100 pages each take 19 us, scores
  // included, in a table of 2048 and 37 in one of 8192; with 2048 pages 119 in the latter.
  if (max_pages <= 512) return launch_choose<32, 16>(a, st);
  if (max_pages <= 2048) return launch_choose<128, 16>(a, st);
  return launch_choose<1024, 16>(a, st);
}

}  // namespace eagle
