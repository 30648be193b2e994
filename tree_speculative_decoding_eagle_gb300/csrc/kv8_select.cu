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
// Two kernels.  Scores: a tile of 16 rows (nodes by heads, the heads padded to a
// power of two) against 8 pages a step on warp-level f16 MMAs, q' and the bounds
// being exact in f16; a lane's 16-byte pieces of the bounds are B fragments once
// converted, because the order of the columns in the sum is free.  Choice: a row's
// scores as ordered 32-bit keys in registers, bisection on the key that `top` of
// them reach, ties to the lower pages, one prefix sum for the places.
#include "kv8_select.cuh"

namespace eagle {

constexpr int kScoreWarps = 4;

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Scores of a tile of rows against the pages of a chunk, eight a step.  blockIdx.x:
// chunk of pages, blockIdx.y: (sequence, KV head), blockIdx.z: tiles of rows.
// Row r of tile T of 16: padded row T * 16 + r = node << log_g | head.  With more
// than 16 heads a node's two tiles belong to one warp (MT = 2).
// The bounds come through a ring of asynchronous copies, kStages steps ahead; a lane
// reads back what it copied itself, so no lane waits for another.  Page numbers and
// scales are read for four steps (a batch) at a time, a batch ahead of the copies.
constexpr int kStages = 4;

template <int DH, int MT>
__global__ void __launch_bounds__(kScoreWarps * 32) kv8_score_kernel(SelectArgs a, int row_warps, int pages_per_cta) {
  constexpr int STEPS = DH / 16, NV = DH / 64;  // MMA steps a bound, 16-byte pieces of a lane
  __shared__ uint4 ring[kScoreWarps][kStages][2 * NV][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, gr = lane >> 2, t = lane & 3;
  const int bg = blockIdx.y, b = bg / a.Hkv, g = bg % a.Hkv;
  const int rw = warp % row_warps, pw = warp / row_warps, page_warps = kScoreWarps / row_warps;
  const int tile = (blockIdx.z * row_warps + rw) * MT;
  const int rows = a.n << a.log_g;
  pdl_wait();
  const int np = live_pages(a, b);
  const int p_begin = blockIdx.x * pages_per_cta, p_end = min(np, p_begin + pages_per_cta);
  const int p_first = p_begin + pw * 8, p_step = page_warps * 8;  // this warp's steps
  if (p_first >= p_end || tile * 16 >= rows) return;
  const int steps = (p_end - p_first + p_step - 1) / p_step;

  // lane 8 s + i of batch k looks after page i of step 4 k + s: its block of the pool
  const int32_t *table = a.block_table + static_cast<int64_t>(b) * a.max_pages;
  const auto block_at = [&](int batch) {
    const int p = p_first + (batch * 4 + (lane >> 3)) * p_step + (lane & 7);
    int page = 0;
    if (p < p_end) {
      page = table[p];
      if (page < 0 || page >= a.num_pages) {
        report(a.status, EAGLE_ERR_INVALID);  // outside the pool: read page 0
        page = 0;
      }
    }
    return page * a.Hkv + g;  // num_pages * Hkv fits 31 bits
  };
  uint4(*mine)[2 * NV][32] = ring[warp];
  const auto request = [&](int step, int blocks) {
    const int block = __shfl_sync(0xffffffffu, blocks, (step & 3) * 8 + gr);
    if (step < steps) {
      const uint8_t *src = a.bounds + static_cast<int64_t>(block) * 2 * DH + t * (DH / 4);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        cp_async16(&mine[step % kStages][i][lane], src + i * 16);
        cp_async16(&mine[step % kStages][NV + i][lane], src + DH + i * 16);
      }
    }
    cp_async_commit();
  };
  const int block0 = block_at(0);
  int block = block_at(1), block_ahead = block_at(2);  // of the next batch, and of the one after
#pragma unroll
  for (int s = 0; s < kStages; ++s) request(s, block0);
  float ps = a.k_scale[block0], ps_next = a.k_scale[block];

  uint32_t qp[MT][STEPS][4], qn[MT][STEPS][4];
  float row_scale[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int rho = (tile + m) * 16 + gr + 8 * r, node = rho >> a.log_g, h = rho & ((1 << a.log_g) - 1);
      const bool there = rho < rows && h < a.G;
      uint4 x[DH / 32];
      float amax = 0.f;
#pragma unroll
      for (int c = 0; c < DH / 32; ++c) {
        x[c] = make_uint4(0, 0, 0, 0);
        if (there)
          x[c] = __ldg(reinterpret_cast<const uint4 *>(
              a.q + ((static_cast<int64_t>(b) * a.n + node) * a.Hq + g * a.G + h) * DH + t * (DH / 4) + c * 8));
        amax = fmaxf(amax, finite_amax8(x[c]));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int e = whole_exponent(amax);
      const float f = exponent_scale(-e);
      row_scale[m][r] = exponent_scale(e);
#pragma unroll
      for (int c = 0; c < DH / 32; ++c) {
        const uint32_t w[4] = {whole_half2(x[c].x, f), whole_half2(x[c].y, f), whole_half2(x[c].z, f), whole_half2(x[c].w, f)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          qp[m][2 * c + (i >> 1)][2 * (i & 1) + r] = half2_max0(w[i]);
          qn[m][2 * c + (i >> 1)][2 * (i & 1) + r] = half2_min0(w[i]);
        }
      }
    }

  for (int step = 0; step < steps; ++step) {
    if (step && (step & 3) == 0) {  // the next batch
      ps = ps_next;
      block = block_ahead;
      ps_next = a.k_scale[block];
      block_ahead = block_at((step >> 2) + 2);
    }
    cp_async_wait<kStages - 1>();
    const int p0 = p_first + step * p_step;
    uint4 lo[NV], hi[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      lo[i] = mine[step % kStages][i][lane];
      hi[i] = mine[step % kStages][NV + i][lane];
    }
    float c[MT][4], cn[MT][4];  // two chains of MMAs
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 4; ++e) c[m][e] = cn[m][e] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const uint32_t l[4] = {lo[i].x, lo[i].y, lo[i].z, lo[i].w}, h[4] = {hi[i].x, hi[i].y, hi[i].z, hi[i].w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t h0 = e4m3_to_half2(h[w] & 0xffffu), h1 = e4m3_to_half2(h[w] >> 16);
        const uint32_t l0 = e4m3_to_half2(l[w] & 0xffffu), l1 = e4m3_to_half2(l[w] >> 16);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          mma_f16(c[m], qp[m][i * 4 + w], h0, h1);
          mma_f16(cn[m], qn[m][i * 4 + w], l0, l1);
        }
      }
    }
    request(step + kStages, block);  // into the stage just read: kStages is a batch
    // columns 2t, 2t + 1 of the result are pages p0 + 2t, p0 + 2t + 1
    const float scale = exponent_scale(scale_exponent(ps));
    const float s0 = __shfl_sync(0xffffffffu, scale, (step & 3) * 8 + 2 * t), s1 = __shfl_sync(0xffffffffu, scale, (step & 3) * 8 + 2 * t + 1);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int h = ((tile + m) * 16 + gr + 8 * r) & ((1 << a.log_g) - 1);
        c[m][2 * r] += cn[m][2 * r];
        c[m][2 * r + 1] += cn[m][2 * r + 1];
        c[m][2 * r] = h < a.G ? c[m][2 * r] * row_scale[m][r] * s0 : -INFINITY;
        c[m][2 * r + 1] = h < a.G ? c[m][2 * r + 1] * row_scale[m][r] * s1 : -INFINITY;
        for (int o = 0; o < min(a.log_g, 3); ++o) {  // the heads of a node: rows gr that share its upper bits
          c[m][2 * r] = fmaxf(c[m][2 * r], __shfl_xor_sync(0xffffffffu, c[m][2 * r], 4 << o));
          c[m][2 * r + 1] = fmaxf(c[m][2 * r + 1], __shfl_xor_sync(0xffffffffu, c[m][2 * r + 1], 4 << o));
        }
      }
    if (a.log_g >= 4) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        c[m][0] = fmaxf(c[m][0], c[m][2]);
        c[m][1] = fmaxf(c[m][1], c[m][3]);
      }
    }
    if constexpr (MT == 2) {
      c[0][0] = fmaxf(c[0][0], c[1][0]);
      c[0][1] = fmaxf(c[0][1], c[1][1]);
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {  // a node's first row writes; MT = 2: one node a pair of tiles
      const int rho = tile * 16 + gr + 8 * r;
      if (rho >= rows || (rho & ((1 << a.log_g) - 1))) continue;
      float *dst = a.scores + ((static_cast<int64_t>(b) * a.n + (rho >> a.log_g)) * a.Hkv + g) * a.stride + p0 + 2 * t;
      *reinterpret_cast<float2 *>(dst) = make_float2(c[0][2 * r], c[0][2 * r + 1]);
    }
  }
}

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

template <int DH, int MT>
static cudaError_t launch_score(const SelectArgs &a, int num_sms, cudaStream_t st) {
  // Row tiles over a CTA's warps first, so that they share the bounds in L1; what
  // warps are left split the pages.  Pages are cut into chunks until every SM has
  // eight CTAs, a chunk being at least one step of each warp.
  const int tiles = ((a.n << a.log_g) + 16 * MT - 1) / (16 * MT);
  int row_warps = 1;
  while (row_warps < kScoreWarps && row_warps < tiles) row_warps *= 2;
  const int z = (tiles + row_warps - 1) / row_warps, step = 8 * (kScoreWarps / row_warps);
  const int64_t base = static_cast<int64_t>(a.B) * a.Hkv * z, want = (8ll * num_sms + base - 1) / base;
  const int most = (a.max_pages + step - 1) / step, chunks = static_cast<int>(want < most ? want : most);
  const int per = ((a.max_pages + chunks - 1) / chunks + step - 1) / step * step;
  const dim3 grid((a.max_pages + per - 1) / per, a.B * a.Hkv, z);
  return launch_chained(kv8_score_kernel<DH, MT>, grid, dim3(kScoreWarps * 32), 0, st, a, row_warps, per);
}

template <int T, int V>
static cudaError_t launch_choose(const SelectArgs &a, cudaStream_t st) {
  constexpr int THREADS = T < 128 ? 128 : T;
  const int64_t rows = static_cast<int64_t>(a.B) * a.n * a.Hkv;
  const dim3 grid(static_cast<unsigned>((rows * T + THREADS - 1) / THREADS));
  return launch_chained(kv8_choose_kernel<T, V>, grid, dim3(THREADS), 0, st, a, rows);
}

// kv8_score_tc.cu
cudaError_t launch_kv8_score_tc(const SelectArgs &a, int dh, int num_sms, cudaStream_t st);

// Padded rows of a sequence and KV head from which the scores are computed on
// tcgen05 tiles of 128 pages by up to 256 rows.
constexpr int kTileRows = 64;

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
  cudaError_t e;
  if ((n << log_g) >= kTileRows) e = launch_kv8_score_tc(a, dh, num_sms, st);
  else if (dh == 128) e = log_g == 5 ? launch_score<128, 2>(a, num_sms, st) : launch_score<128, 1>(a, num_sms, st);
  else e = log_g == 5 ? launch_score<64, 2>(a, num_sms, st) : launch_score<64, 1>(a, num_sms, st);
  if (e != cudaSuccess) return e;
  if (max_pages <= 512) return launch_choose<32, 16>(a, st);
  if (max_pages <= 2048) return launch_choose<128, 16>(a, st);
  return launch_choose<1024, 16>(a, st);
}

}  // namespace eagle
