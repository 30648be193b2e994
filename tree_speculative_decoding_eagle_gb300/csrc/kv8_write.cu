// Keys and values into the 8-bit paged cache.
//
// A page's rows of one head share the scale 2^e, the least with
// max |x| <= 448 * 2^e over every row written to the page so far.  Work is cut
// into runs: neighbouring tokens that land in one page.  A run of a head is
// one team's work: the largest magnitude of its rows, the exponent (joined
// with the page's when earlier rows stay), the rows divided by 2^e and rounded
// once to e4m3; when the exponent grew, the page's earlier rows are re-encoded
// at the new one.  Two runs never share a page (a second one that is near is
// found and skipped), so nothing is atomic and the result does not depend on an
// order.
//
// What bounds it: HBM for prompts (2 or 4 bytes read, 1 written an element),
// latency for single tokens and commits.  Measured: 65536 tokens of 8 heads of
// 128, bf16, pages of 64: 77.6 us (5.2 TB/s, 78 % of a copy's rate; 403 MB; 76.8
// without the look for an interrupted page); one token of each of 64 requests, 8
// heads of 64: 4.3 us (4.2); the accepted paths of 8 trees, 40 heads of 128: 7.9
// us with a copy of kv_len before it.
#include "kv8.cuh"
#include "sm100.cuh"

namespace eagle {

using namespace sm100;

constexpr int kWriteWarps = 8;

// A team's barrier: its warps are neighbours in the CTA.
__device__ __forceinline__ void team_sync(int team, int warps) {
  if (warps == 1) __syncwarp();
  else asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(warps * 32) : "memory");
}

// 16 elements of a row, as loaded and as floats.
template <typename T> struct Chunk {
  static constexpr int kVecs = 16 / VecTraits<T>::kElems;
  uint4 v[kVecs];
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = ld_stream16(p + i * VecTraits<T>::kElems);
  }
  // Largest magnitude as a float's bits; above every finite one's if an element
  // is infinite or NaN.
  __device__ __forceinline__ uint32_t magnitude() const {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) m = sizeof(T) == 2 ? __vmaxu2(m, w[j] & 0x7fff7fffu) : max(m, w[j] & 0x7fffffffu);
    }
    return sizeof(T) == 2 ? max(m & 0xffff0000u, m << 16) : m;
  }
  __device__ __forceinline__ void floats(float (&x)[16]) const {
    constexpr int E = VecTraits<T>::kElems;
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      float y[E];
      VecTraits<T>::unpack(v[i], y);
#pragma unroll
      for (int e = 0; e < E; ++e) x[i * E + e] = y[e];
    }
  }
};
__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) <= 3.402823466e38f; }

// Rows of a run as neighbouring tokens, and as nodes of a path.
template <typename T> struct LinearRows {
  const T *base;
  int64_t stride;
  __device__ __forceinline__ const T *operator()(int r) const { return base + r * stride; }
};
template <typename T> struct PathRows {
  const T *base;
  const int *node;
  int dh;
  __device__ __forceinline__ const T *operator()(int r) const { return base + static_cast<int64_t>(node[r]) * dh; }
};

// Chunks a thread keeps between the two looks at a run (the largest magnitude,
// then the rounding); a longer run's others are read again, from L2.
constexpr int kHeld = 4;

// One run: rows 0..count-1 (row_of gives their source) into rows
// first..first+count-1 of a page of one head.  `red` is the team's shared
// scratch (one float a warp).  Called by every thread of the team.
template <typename T, typename RowOf>
__device__ __forceinline__ void write_run(RowOf row_of, int count, uint8_t *page, float *scale, int first, int dh,
                                          int team, int warps, int tw, float *red, int32_t *status) {
  const int lane = threadIdx.x & 31, tt = tw * 32 + lane, nt = warps * 32;
  const int cpr = dh / 16, chunks = count * cpr;  // 16-element chunks a row, of the run
  // A thread's chunks are nt apart: where a whole number of rows is that, the
  // column stays and a row step is all there is to compute.
  const bool steady = nt % cpr == 0;
  const int row_step = nt / cpr, row_first = tt / cpr, col = (tt - row_first * cpr) * 16;
  const auto source = [&](int c, int u) {
    return steady ? row_of(row_first + u * row_step) + col : row_of(c / cpr) + (c % cpr) * 16;
  };
  Chunk<T> held[kHeld];
#pragma unroll
  for (int u = 0; u < kHeld; ++u)
    if (tt + u * nt < chunks) held[u].load(source(tt + u * nt, u));
  const float s_old = first > 0 ? *scale : 1.f;
  uint32_t top = 0;
#pragma unroll
  for (int u = 0; u < kHeld; ++u)
    if (tt + u * nt < chunks) top = max(top, held[u].magnitude());
  for (int c = tt + kHeld * nt, u = kHeld; c < chunks; c += nt, ++u) {
    Chunk<T> k;
    k.load(source(c, u));
    top = max(top, k.magnitude());
  }
  const bool odd = top >= 0x7f800000u;  // something is not finite: the largest of the others
  float amax = __uint_as_float(top);
  if (odd) {
    amax = 0.f;
    for (int c = tt, u = 0; c < chunks; c += nt, ++u) {
      Chunk<T> k;
      k.load(source(c, u));
      float x[16];
      k.floats(x);
#pragma unroll
      for (int i = 0; i < 16; ++i) amax = fmaxf(amax, is_finite(x[i]) ? fabsf(x[i]) : 0.f);
    }
  }
  amax = warp_max(amax);
  if (warps > 1) {
    if (lane == 0) red[tw] = amax;
    team_sync(team, warps);
    for (int w = 0; w < warps; ++w) amax = fmaxf(amax, red[w]);
  }
  int e = block_exponent(amax), e_old = e;
  if (first > 0) {
    e_old = scale_exponent(s_old);
    e = max(e, e_old);
  }
  team_sync(team, warps);  // every thread has the page's scale (and red) before it changes
  if (tt == 0) *scale = exponent_scale(e);
  if (odd || amax > 448.f * exponent_scale(kScaleMax)) report(status, EAGLE_ERR_INVALID);
  const float inv = exponent_scale(-e);
  const auto round_to_page = [&](const Chunk<T> &k, int c) {
    float x[16];
    k.floats(x);
    if (odd) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (!is_finite(x[i])) x[i] = __uint_as_float(0x7fffffffu);
    }
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = e4m3_pair(x[4 * i] * inv, x[4 * i + 1] * inv) | (e4m3_pair(x[4 * i + 2] * inv, x[4 * i + 3] * inv) << 16);
    *reinterpret_cast<uint4 *>(page + static_cast<int64_t>(first) * dh + static_cast<int64_t>(c) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  };
#pragma unroll
  for (int u = 0; u < kHeld; ++u)
    if (tt + u * nt < chunks) round_to_page(held[u], tt + u * nt);
  for (int c = tt + kHeld * nt, u = kHeld; c < chunks; c += nt, ++u) {
    Chunk<T> k;
    k.load(source(c, u));
    round_to_page(k, c);
  }
  if (e > e_old) {  // the page's earlier rows at the new scale (rare: a new largest magnitude)
    const float f = exp2f(static_cast<float>(e_old - e));
    for (int c = tt; c < first * cpr; c += nt) {
      uint4 *p = reinterpret_cast<uint4 *>(page) + c;
      uint4 v = *p;
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t a = e4m3_to_half2(w[i] & 0xffffu), b = e4m3_to_half2(w[i] >> 16);
        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&a));
        const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&b));
        w[i] = e4m3_pair(x.x * f, x.y * f) | (e4m3_pair(y.x * f, y.y * f) << 16);
      }
      *p = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Skipped tokens that a run's first token looks past for an earlier one of its
// page (beside the 32 tokens before its piece, which it always looks at): eight
// rounds of loads, only where nothing but skipped tokens precedes a run that does
// not begin a page.
constexpr int kLookBack = 1024;

struct AppendArgs {
  const void *k, *v;
  int64_t token_stride, head_stride;
  const int32_t *slot_map;
  uint8_t *k_pages, *v_pages;
  float *k_scale, *v_scale;
  int T, Hkv, dh, log_page, num_pages;
  int block;  // tokens a CTA looks after (those whose run begins there)
  int units;  // (head, K or V) pairs a CTA looks after
  int warps;  // warps a team
  int32_t *status;
};

// One CTA per (token block, `units` of the 2 Hkv (head, K or V) pairs), the pairs
// fastest, so that CTAs that run together read neighbouring heads of the same
// tokens.  A team finds its runs once for all of its pairs: finding one costs
// about what rounding a page of one head does (measured on 65536 tokens of 8
// heads of 128, pages of 64: 101 us with one pair a CTA, 84 with two, 76 with four, 80 with eight, before the look for
// interrupted pages).
template <typename T>
__global__ void __launch_bounds__(kWriteWarps * 32, sizeof(T) == 2 ? 3 : 2) kv8_append_kernel(AppendArgs a) {
  __shared__ float red[kWriteWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = warp / a.warps, tw = warp % a.warps, teams = kWriteWarps / a.warps;
  const int splits = (2 * a.Hkv + a.units - 1) / a.units, part = blockIdx.x / splits;
  const int u0 = (blockIdx.x - part * splits) * a.units, u1 = min(2 * a.Hkv, u0 + a.units);
  const int t0 = part * a.block, t1 = min(a.T, t0 + a.block);
  const int P = 1 << a.log_page;
  pdl_wait();
  pdl_trigger();
  const auto page_of = [&](int slot) {  // -1 for a token that is skipped
    if (slot < 0) return -1;
    const int page = slot >> a.log_page;
    return page < a.num_pages ? page : -1;
  };
  int seen = 0;  // leaders before this 32-token piece
  for (int p0 = t0; p0 < t1; p0 += 32) {
    const int slot = p0 + lane < t1 ? a.slot_map[p0 + lane] : -1;
    const int before = p0 - 32 + lane >= 0 ? a.slot_map[p0 - 32 + lane] : -1;
    int prev = __shfl_up_sync(0xffffffffu, slot, 1);
    const int s_before = __shfl_sync(0xffffffffu, before, 31);
    if (lane == 0) prev = s_before;
    const int page = page_of(slot), page_before = page_of(before);
    const bool same = page >= 0 && page == page_of(prev);
    // what is skipped: a slot past the pool, a row out of sequence
    if (u0 == 0 && warp == 0 && ((slot >= 0 && page < 0) || (same && slot != prev + 1))) report(a.status, EAGLE_ERR_INVALID);
    uint32_t lead = __ballot_sync(0xffffffffu, page >= 0 && !same);
    while (lead) {  // the same in every warp
      const int l = __ffs(lead) - 1;
      lead &= lead - 1;
      if (seen++ % teams != team) continue;
      const int s0 = __shfl_sync(0xffffffffu, slot, l), pg = s0 >> a.log_page, first = s0 & (P - 1);
      // A page whose tokens are interrupted (by skipped ones, or by others): two
      // runs of it would write its scale and rows at the same time.
      const uint32_t below = (1u << l) - 1u;
      bool again = (__ballot_sync(0xffffffffu, page == pg) & below) | __ballot_sync(0xffffffffu, page_before == pg);
      if (!again && first && !((__ballot_sync(0xffffffffu, page >= 0) & below) | __ballot_sync(0xffffffffu, page_before >= 0))) {
        bool found = false;
        for (int back = p0 - 32; !found && back > 0 && back > p0 - 32 - kLookBack; back -= 128) {
          int pages[4];
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int t = back - 32 * (w + 1) + lane;
            pages[w] = t >= 0 ? page_of(a.slot_map[t]) : -1;
          }
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t on = __ballot_sync(0xffffffffu, pages[w] >= 0);
            if (on && !found) {  // the nearest token that is not skipped
              found = true;
              again = __shfl_sync(0xffffffffu, pages[w], 31 - __clz(on)) == pg;
            }
          }
        }
      }
      if (again) {
        if (u0 == 0 && tw == 0 && lane == 0) report(a.status, EAGLE_ERR_INVALID);
        continue;
      }
      // the run: neighbours with the next slots, within the page; 96 tokens are
      // looked at with one latency
      int count = 1;
      for (bool whole = true; whole;) {
        bool next[3];
#pragma unroll
        for (int w = 0; w < 3; ++w) {
          const int o = count + 32 * w + lane;
          next[w] = first + o < P && p0 + l + o < a.T && a.slot_map[p0 + l + o] == s0 + o;
        }
#pragma unroll
        for (int w = 0; w < 3; ++w) {
          const uint32_t on = __ballot_sync(0xffffffffu, next[w]);
          if (whole) count += on == 0xffffffffu ? 32 : __ffs(~on) - 1;
          whole = whole && on == 0xffffffffu;
        }
      }
      for (int u = u0; u < u1; ++u) {
        const int g = u >> 1;
        const bool is_v = u & 1;
        const int64_t at = static_cast<int64_t>(pg) * a.Hkv + g;
        const T *row0 = reinterpret_cast<const T *>(is_v ? a.v : a.k) + g * a.head_stride + (p0 + l) * a.token_stride;
        write_run<T>(LinearRows<T>{row0, a.token_stride}, count, (is_v ? a.v_pages : a.k_pages) + (at << a.log_page) * a.dh,
                     (is_v ? a.v_scale : a.k_scale) + at, first, a.dh, team, a.warps, tw, red + team * a.warps, a.status);
      }
    }
  }
}

struct Commit8Args {
  const void *k_tree, *v_tree;
  int B, n, Hkv, dh, D, log_page, max_pages, num_pages;
  int skip;  // path entries before the first that is stored: 0 stores the root, 1 finds it stored
  const int32_t *accept_len, *path_nodes;
  uint8_t *k_pages, *v_pages;
  float *k_scale, *v_scale;
  const int32_t *block_table;
  int32_t *kv_len, *slot_mapping, *status;
};

// One cluster of CTAs per sequence, a warp per (head, K or V): kv_len, which is
// updated in place, is written after the cluster barrier that every CTA
// reaches with its reads of it done.
template <typename T>
__global__ void __launch_bounds__(kWriteWarps * 32) kv8_commit_kernel(Commit8Args a) {
  __shared__ int s_ok, s_path[65], s_page[8];
  const int b = blockIdx.y, rank = blockIdx.x, ctas = gridDim.x;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int P = 1 << a.log_page;
  pdl_wait();
  const int L = a.kv_len[b], acc = a.accept_len[b];
  const int rows = acc + 1 - a.skip;  // path[skip..acc]
  if (warp == 0) {
    bool ok = acc >= 0 && acc <= a.D && acc <= 64 && L >= a.skip &&
              static_cast<int64_t>(L) + rows <= (static_cast<int64_t>(a.max_pages) << a.log_page);
    if (ok) {
      for (int p = a.skip + lane; p <= acc; p += 32) {
        const int node = a.path_nodes[static_cast<int64_t>(b) * (a.D + 1) + p];
        s_path[p] = node;
        if (p == 0 ? node != 0 : node < 1 || node >= a.n) ok = false;
      }
      // at most 65 rows in pages of at least 16: five pages
      const int lp = (L >> a.log_page) + lane;
      if (rows > 0 && lp <= (L + rows - 1) >> a.log_page) {
        const int page = a.block_table[static_cast<int64_t>(b) * a.max_pages + lp];
        s_page[lane] = page;
        if (page < 0 || page >= a.num_pages) ok = false;
      }
    }
    ok = __all_sync(0xffffffffu, ok);
    if (lane == 0) {
      s_ok = ok;
      if (!ok && rank == 0) report(a.status, EAGLE_ERR_INVALID);
    }
  }
  __syncthreads();
  if (ctas > 1) {  // every CTA has read kv_len
    cluster_arrive_release();
    cluster_wait();
  }
  pdl_trigger();
  if (!s_ok) return;
  if (rank == 0 && tid == 0) a.kv_len[b] = L + rows;
  for (int u = rank * kWriteWarps + warp; u < 2 * a.Hkv; u += ctas * kWriteWarps) {
    const int g = u >> 1;
    const bool is_v = u & 1;
    const T *src = reinterpret_cast<const T *>(is_v ? a.v_tree : a.k_tree) +
                   (static_cast<int64_t>(b) * a.Hkv + g) * a.n * a.dh;
    for (int r = 0, lp = 0; r < rows; ++lp) {
      const int first = (L + r) & (P - 1), count = min(rows - r, P - first);
      const int64_t at = static_cast<int64_t>(s_page[lp]) * a.Hkv + g;
      write_run<T>(PathRows<T>{src, s_path + a.skip + r, a.dh}, count,
                   (is_v ? a.v_pages : a.k_pages) + (at << a.log_page) * a.dh, (is_v ? a.v_scale : a.k_scale) + at,
                   first, a.dh, 0, 1, 0, nullptr, a.status);
      r += count;
    }
  }
  if (a.slot_mapping) {
    for (int i = rank * kWriteWarps * 32 + tid; i < a.n; i += ctas * kWriteWarps * 32) {
      int slot = i == 0 ? L - a.skip : -1;
      for (int p = 1; p <= acc; ++p)
        if (s_path[p] == i) slot = L + p - a.skip;
      a.slot_mapping[static_cast<int64_t>(b) * a.n + i] = slot;
    }
  }
}

static int log2_page(int p) {
  int l = 0;
  while ((1 << l) < p) ++l;
  return l;
}

cudaError_t launch_kv8_append(const void *k, const void *v, int dtype, int T, int Hkv, int dh, int64_t token_stride,
                              int64_t head_stride, const int32_t *slot_map, uint8_t *k_pages, uint8_t *v_pages,
                              float *k_scale, float *v_scale, int page_size, int num_pages, int32_t *status,
                              int num_sms, cudaStream_t st) {
  AppendArgs a = {k, v, token_stride, head_stride, slot_map, k_pages, v_pages, k_scale, v_scale,
                  T, Hkv, dh, log2_page(page_size), num_pages, 0, 1, 0, status};
  // A team takes a run.  Long inputs: enough warps that a thread holds a whole
  // page's share (kHeld chunks), and as many pages a CTA as it has teams.  Few
  // rows (single tokens mostly): a warp a run, and CTAs cut down until the SMs
  // have four each.
  const int64_t rows = static_cast<int64_t>(T) * Hkv * 2;
  const int page_warps = page_size * (dh / 16) / (32 * kHeld);
  a.warps = 1;
  if (rows > 32ll * num_sms)
    while (a.warps < kWriteWarps && a.warps < page_warps) a.warps *= 2;
  const int teams = kWriteWarps / a.warps;
  a.block = teams * page_size;
  while (a.block > teams && static_cast<int64_t>((T + a.block - 1) / a.block) * Hkv * 2 < 4ll * num_sms) a.block /= 2;
  const int64_t blocks = (T + a.block - 1) / a.block;
  while (a.units < 2 * Hkv && blocks * ((2 * Hkv + 2 * a.units - 1) / (2 * a.units)) >= 12ll * num_sms) a.units *= 2;
  const int64_t ctas = blocks * ((2 * Hkv + a.units - 1) / a.units);
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(ctas));
  return dtype == EAGLE_BF16 ? launch_chained(kv8_append_kernel<__nv_bfloat16>, grid, dim3(kWriteWarps * 32), 0, st, a)
                             : launch_chained(kv8_append_kernel<float>, grid, dim3(kWriteWarps * 32), 0, st, a);
}

cudaError_t launch_kv8_commit(const void *k_tree, const void *v_tree, int dtype, int B, int n, int Hkv, int dh, bool root,
                              const int32_t *accept_len, const int32_t *path_nodes, int D, uint8_t *k_pages,
                              uint8_t *v_pages, float *k_scale, float *v_scale, const int32_t *block_table,
                              int max_pages, int page_size, int num_pages, int32_t *kv_len, int32_t *slot_mapping,
                              int32_t *status, cudaStream_t st) {
  Commit8Args a = {k_tree, v_tree, B, n, Hkv, dh, D, log2_page(page_size), max_pages, num_pages, root ? 0 : 1, accept_len,
                   path_nodes, k_pages, v_pages, k_scale, v_scale, block_table, kv_len, slot_mapping, status};
  int ctas = 1;  // a warp for each (head, K or V), eight CTAs at most
  while (ctas < 8 && ctas * kWriteWarps < 2 * Hkv) ctas *= 2;
  const dim3 grid(ctas, B);
  return dtype == EAGLE_BF16
             ? launch_chained_cluster(kv8_commit_kernel<__nv_bfloat16>, grid, dim3(kWriteWarps * 32), 0, st, ctas, a)
             : launch_chained_cluster(kv8_commit_kernel<float>, grid, dim3(kWriteWarps * 32), 0, st, ctas, a);
}

}  // namespace eagle
