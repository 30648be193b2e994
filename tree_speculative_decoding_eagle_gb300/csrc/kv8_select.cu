// The pages of the 8-bit cache that a query is to attend to: for each node, KV head
// and page the greatest product that the page's bounds allow, and the `top` pages
// with the greatest.
//
// A query row (node i, head h) is taken as whole numbers q' = rint(q 2^-e), e the
// power of two that puts its largest magnitude into [64, 128], |q'| <= 128.  With
// the bounds lo, hi of a page's columns (multiples of 1/2 up to 448, kv8_bounds.cu)
//   u = sum_c max(q'_c, 0) hi_c + min(q'_c, 0) lo_c
// is a sum of at most 128 multiples of 1/2 up to 128 * 448: below 2^23, so a float32
// sum of it is exact whatever its order.  The score u 2^(e + page scale's exponent)
// is exact too, and the pages chosen for a node are the same in a tree, alone, in
// any batch and on any launch shape: verification with selected pages accepts what
// decoding token by token with selected pages would have produced.
// The node's score of a page is the largest over the heads that share the KV head.
//
// Two kernels.  Scores: kv8_score.cu.  Choice (here): a row's scores as ordered
// 32-bit keys in registers, a search for the greatest key that `top` of them reach
// (by interpolation on the counts, every third step by halving), ties to the lower
// pages, one prefix sum for the places.
#include "kv8_select.cuh"

namespace eagle {

// T threads (a power of two, 32 or more) a row, V neighbouring scores a thread.
template <int T, int V>
__global__ void __launch_bounds__(T < 128 ? 128 : T) kv8_choose_kernel(SelectArgs a, int64_t row_count) {
  constexpr int THREADS = T < 128 ? 128 : T, WARPS = T / 32;
  __shared__ int part[2][THREADS / 32];
  const int tid = threadIdx.x % T, lane = tid & 31, warp = tid >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (THREADS / T) + threadIdx.x / T;
  pdl_wait();
  pdl_trigger();
  if (row >= row_count) return;  // whole warps: T < 128 has one warp a row
  const int b = static_cast<int>(row / (static_cast<int64_t>(a.n) * a.Hkv));
  const int np = live_pages(a, b), K = min(a.top, np);
  const float *src = a.scores + row * a.stride;
  // sum over the row's threads (and, with `before`, of the threads before this one)
  int turn = 0;
  const auto row_sum = [&](int x) {
    x = __reduce_add_sync(0xffffffffu, x);
    if constexpr (WARPS > 1) {
      if (lane == 0) part[turn][warp] = x;
      __syncthreads();
      x = __reduce_add_sync(0xffffffffu, lane < WARPS ? part[turn][lane] : 0);
      turn ^= 1;  // the next sum's words: those of the one before have been read by then
    }
    return x;
  };
  float s[V];
  uint32_t key[V];
#pragma unroll
  for (int j = 0; j < V; j += 4) {
    const int p = tid * V + j;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (p < np) x = *reinterpret_cast<const float4 *>(src + p);
    s[j] = x.x; s[j + 1] = x.y; s[j + 2] = x.z; s[j + 3] = x.w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = p + i;
      // (a score is finite unless the bounds hold NaN; its key stays between)
      key[j + i] = at >= np ? 0u : (at < a.first || at >= np - a.last) ? 0xffffffffu : max(ordered_u32(s[j + i]), 1u);
    }
  }
  // The greatest key that at least K of them reach: count(lo) >= K > count(hi).
  uint32_t lo = 1u, hi = 0xffffffffu;  // live keys lie in between; first + last <= top, so hi + 1 is reached by fewer
  int reach = np;
  if (K < np) {
    const auto count = [&](uint32_t bar) {
      int c = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) c += key[j] >= bar;
      return row_sum(c);
    };
    const int forced = count(hi);
    if (forced >= K) {
      lo = hi;
      reach = forced;
    } else {
      // the least and the greatest key without the forced ones
      uint32_t least = 0xffffffffu, most = 0u;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (key[j]) least = min(least, key[j]);
        if (key[j] != 0xffffffffu) most = max(most, key[j]);
      }
      least = __reduce_min_sync(0xffffffffu, least);
      most = __reduce_max_sync(0xffffffffu, most);
      if constexpr (WARPS > 1) {
        __syncthreads();
        if (lane == 0) { part[0][warp] = static_cast<int>(least); part[1][warp] = static_cast<int>(most); }
        __syncthreads();
        least = __reduce_min_sync(0xffffffffu, lane < WARPS ? static_cast<uint32_t>(part[0][lane]) : 0xffffffffu);
        most = __reduce_max_sync(0xffffffffu, lane < WARPS ? static_cast<uint32_t>(part[1][lane]) : 0u);
        __syncthreads();
      }
      lo = least;      // all reach it
      hi = most + 1u;  // the forced ones alone do
      int above = forced;
      for (int step = 1; reach != K && hi - lo > 1; ++step) {
        uint32_t mid = lo + (hi - lo) / 2;
        if (step % 3) {
          const float share = (static_cast<float>(reach - K) + 0.5f) / static_cast<float>(reach - above);
          mid = min(max(lo + static_cast<uint32_t>(static_cast<float>(hi - lo) * share), lo + 1), hi - 1);
        }
        const int c = count(mid);
        if (c >= K) {
          lo = mid;
          reach = c;
        } else {
          hi = mid;
          above = c;
        }
      }
    }
  }
  // more than K reach lo: those equal to it in order of their pages, after all greater ones
  int spare = 0, mine = 0, equal = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    mine += key[j] > lo;
    equal += key[j] == lo;
  }
  if (reach == K) {
    mine += equal;
    equal = 0;
  } else {
    spare = K - row_sum(mine);
  }
  // places: exclusive sums over the threads before of (taken for sure, equal)
  int x = mine, y = equal;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int ax = __shfl_up_sync(0xffffffffu, x, o), ay = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) { x += ax; y += ay; }
  }
  if constexpr (WARPS > 1) {
    __syncthreads();
    if (lane == 31) { part[0][warp] = x; part[1][warp] = y; }
    __syncthreads();
    int px = lane < warp ? part[0][lane] : 0, py = lane < warp ? part[1][lane] : 0;
    px = __reduce_add_sync(0xffffffffu, px);
    py = __reduce_add_sync(0xffffffffu, py);
    x += px;
    y += py;
  }
  int at = x - mine, same = y - equal;  // taken before this thread's first page: at + min(same, spare)
  int32_t *dst = a.sel + row * a.top;
  float *dst_s = a.sel_score ? a.sel_score + row * a.top : nullptr;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const bool tie = reach != K && key[j] == lo;
    const bool take = key[j] > lo || (key[j] == lo && (reach == K || same < spare));
    if (take) {
      const int place = at + min(same, spare);
      dst[place] = tid * V + j;
      if (dst_s) dst_s[place] = s[j];
      if (!tie) ++at;
    }
    if (tie) ++same;
  }
  for (int i = K + tid; i < a.top; i += T) {
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
  constexpr int THREADS = T < 128 ? 128 : T;
  const int64_t rows = static_cast<int64_t>(a.B) * a.n * a.Hkv;
  const dim3 grid(static_cast<unsigned>((rows * T + THREADS - 1) / THREADS));
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
  if (max_pages <= 512) return launch_choose<32, 16>(a, st);
  if (max_pages <= 2048) return launch_choose<128, 16>(a, st);
  return launch_choose<1024, 16>(a, st);
}

}  // namespace eagle
