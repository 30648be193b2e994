// Scores of pages for many query rows (trees, prompt chunks): the product of
// kv8_select.cu as a matrix product on the 5th-generation tensor cores.
//
// D[page, row] = sum over 2 dh of A[page, k] B[row, k] in f16 with float32
// accumulation: A holds a page's upper bounds, then its lower ones; B a row's whole
// numbers, first the positive ones (zeros elsewhere), then the negative.  Every
// product and sum is exact.  Pages are the rows of D, so a thread that reads D back
// owns a page: the largest score over the heads of a node is a maximum over
// neighbouring columns, within the thread, and a node's scores of 32 pages leave a
// warp as one line.
//
// A CTA takes up to 256 query rows (padded: node << LG | head; places past the last
// head repeat head 0) of one sequence and KV head and a chunk of its pages, 128 a tile.
// Roles: four converter warps (e4m3 from global memory to f16 in a ring of three
// halves of A tiles, in the 128-byte swizzle), one thread for the MMAs, four warps
// that take D from tensor memory (two buffers) to the scores.
// What bounds it: conversion and MMA are about even at 256 rows.
//
// Every wait is bounded; a timeout raises EAGLE_ERR_TIMEOUT in the status word, and
// the CTA completes its MMAs, frees tensor memory and exits.
#include "kv8_select.cuh"
#include "sm100.cuh"

namespace eagle {

using namespace sm100;

template <int DH>
struct ScoreShape {
  static constexpr int kPages = 128, kRows = 256, kRing = 3, kThreads = 288;
  static constexpr int kRowBytes = kRows * 2 * DH * 2;   // B: regions of 64 columns, [region][row][128 bytes]
  static constexpr int kHalfBytes = kPages * DH * 2;     // half an A tile: upper or lower bounds
  static constexpr int kBarOff = kRowBytes + kRing * kHalfBytes;
  static constexpr int kScaleOff = kBarOff + 128;
  static constexpr int kUsed = kScaleOff + kRows * 4 + 1024;
  // one CTA an SM in every form: a CTA takes all of tensor memory
  static constexpr int kSmem = kUsed < 120 * 1024 ? 120 * 1024 : kUsed;
  static_assert(kSmem <= 232448, "shared memory budget");
};

template <int DH, int LG>
__global__ void __launch_bounds__(288, 1) kv8_score_tc_kernel(SelectArgs a, int pages_per_cta) {
  using Sh = ScoreShape<DH>;
  constexpr int REG = DH / 64;  // regions of 64 columns in a bound
  extern __shared__ unsigned char score_smem[];
  unsigned char *sm = score_smem + ((1024u - (smem_u32(score_smem) & 1023u)) & 1023u);
  unsigned char *sB = sm, *sA = sm + Sh::kRowBytes;
  uint64_t *full = reinterpret_cast<uint64_t *>(sm + Sh::kBarOff);  // a half tile is written
  uint64_t *empty = full + Sh::kRing;                               // and read
  uint64_t *d_full = empty + Sh::kRing, *d_free = d_full + 2, *teardown = d_free + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(teardown + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  float *col_scale = reinterpret_cast<float *>(sm + Sh::kScaleOff);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bg = blockIdx.y, b = bg / a.Hkv, g = bg % a.Hkv;
  const int row0 = blockIdx.z * Sh::kRows, rows = min((a.n << LG) - row0, Sh::kRows);
  pdl_wait();
  const int np = live_pages(a, b);
  const int p_begin = blockIdx.x * pages_per_cta, p_end = min(np, p_begin + pages_per_cta);
  if (p_begin >= p_end) return;  // the whole CTA
  const int tiles = (p_end - p_begin + Sh::kPages - 1) / Sh::kPages;
  const int cols = (rows + 31) & ~31;

  if (tid == 0) {
    for (int i = 0; i < Sh::kRing; ++i) {
      mbar_init(&full[i], 4);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_free[i], 4);
    }
    mbar_init(teardown, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 8) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  } else {
    // the query rows: DH / 8 neighbouring lanes hold a row
    constexpr int CPR = DH / 8;
    for (int idx = tid; idx < cols * CPR; idx += 256) {  // whole warps: cols is a multiple of 32
      const int r = idx / CPR, c = idx % CPR, at = row0 + r, node = at >> LG;
      const int h = (at & ((1 << LG) - 1)) < a.G ? at & ((1 << LG) - 1) : 0;
      uint4 x = make_uint4(0, 0, 0, 0);
      if (node < a.n)
        x = __ldg(reinterpret_cast<const uint4 *>(a.q + ((static_cast<int64_t>(b) * a.n + node) * a.Hq + g * a.G + h) * DH + c * 8));
      float amax = finite_amax8(x);
#pragma unroll
      for (int o = 1; o < CPR; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const int e = whole_exponent(amax);
      const float f = exponent_scale(-e);
      const uint32_t w[4] = {whole_half2(x.x, f), whole_half2(x.y, f), whole_half2(x.z, f), whole_half2(x.w, f)};
      unsigned char *at_b = sB + (c / 8) * (Sh::kRows * 128) + sw128_offset(r, c % 8);
      *reinterpret_cast<uint4 *>(at_b) = make_uint4(half2_max0(w[0]), half2_max0(w[1]), half2_max0(w[2]), half2_max0(w[3]));
      *reinterpret_cast<uint4 *>(at_b + REG * (Sh::kRows * 128)) =
          make_uint4(half2_min0(w[0]), half2_min0(w[1]), half2_min0(w[2]), half2_min0(w[3]));
      if (c == 0) col_scale[r] = exponent_scale(e);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int32_t *table = a.block_table + static_cast<int64_t>(b) * a.max_pages;
  const auto block_at = [&](int p, bool tell) {  // of the pool; page 0's past the chunk or outside the pool
    int page = 0;
    if (p < p_end) {
      page = table[p];
      if (page < 0 || page >= a.num_pages) {
        if (tell) report(a.status, EAGLE_ERR_INVALID);
        page = 0;
      }
    }
    return page * a.Hkv + g;  // num_pages * Hkv fits 31 bits
  };

  if (warp == 8) {
    if (elect_one()) {
      // The converters wrote A, and all warps B, through the generic proxy: the fence
      // after each wait orders that before the MMAs.
      const uint32_t id = idesc_f16(Sh::kPages, cols, false);
      const uint32_t a_lo = static_cast<uint32_t>(sdesc_sw128(smem_u32(sA), 16, 1024));
      const uint32_t b_lo = static_cast<uint32_t>(sdesc_sw128(smem_u32(sB), 16, 1024));
      bool ok = true;
      for (int j = 0; j < tiles && ok; ++j) {
        if (j >= 2 && !wait_bounded(&d_free[j & 1], (j / 2 - 1) & 1, abort_flag)) break;
        tc_fence_after();
        for (int hf = 0; hf < 2; ++hf) {
          const int u = 2 * j + hf, st = u % Sh::kRing;
          if (!wait_bounded(&full[st], (u / Sh::kRing) & 1, abort_flag)) { ok = false; break; }
          fence_async_smem();
          const uint32_t ad = anew(a_lo + st * (Sh::kHalfBytes >> 4)), bd = anew(b_lo + hf * REG * ((Sh::kRows * 128) >> 4));
#pragma unroll
          for (int s = 0; s < DH / 16; ++s)
            mma_f16_ss(tmem + (j & 1) * 256, ad + (((s / 4) * (Sh::kPages * 128) + (s % 4) * 32) >> 4),
                       bd + (((s / 4) * (Sh::kRows * 128) + (s % 4) * 32) >> 4), id, hf > 0 || s > 0);
          mma_commit(&empty[st]);
        }
        if (ok) mma_commit(&d_full[j & 1]);
      }
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------- converters
    // A warp takes 32 pages of a tile.  In a step eight lanes of a quarter warp hold
    // eight pages' pieces of 16 columns, so their stores touch every bank once; the
    // quarters hold neighbouring pieces, so whole sectors are read.
    constexpr int LOADS = 4 * REG;
    const int cw = warp - 4, quarter = lane >> 3, l8 = lane & 7;
    int block[4], ahead[4];
    const auto blocks_of = [&](int j, int (&out)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) out[i] = block_at(p_begin + j * Sh::kPages + cw * 32 + i * 8 + l8, quarter == 0);
    };
    blocks_of(0, block);
    blocks_of(1, ahead);
    uint4 x[LOADS];
    const auto load = [&](int hf) {  // upper bounds first
#pragma unroll
      for (int i = 0; i < LOADS; ++i)
        x[i] = ld_stream16(a.bounds + (static_cast<int64_t>(block[i / REG]) * 2 + (1 - hf)) * DH + (quarter + 4 * (i % REG)) * 16);
    };
    load(0);
    for (int u = 0; u < 2 * tiles; ++u) {
      const int st = u % Sh::kRing;
      if (u >= Sh::kRing && !wait_bounded(&empty[st], (u / Sh::kRing - 1) & 1, abort_flag)) break;
      unsigned char *half = sA + st * Sh::kHalfBytes;
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int r = cw * 32 + (i / REG) * 8 + l8;
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t h[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          h[2 * k] = e4m3_to_half2(w[k] & 0xffffu);
          h[2 * k + 1] = e4m3_to_half2(w[k] >> 16);
        }
        unsigned char *region = half + (i % REG) * (Sh::kPages * 128);
        *reinterpret_cast<uint4 *>(region + sw128_offset(r, 2 * quarter)) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4 *>(region + sw128_offset(r, 2 * quarter + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
      }
      if (u + 1 < 2 * tiles) {
        if (u & 1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) block[i] = ahead[i];
          blocks_of((u >> 1) + 2, ahead);
        }
        load((u + 1) & 1);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[st]);
      __syncwarp();
    }
  } else {
    // ----------------------------------------------------------- D to the scores
    const uint32_t tD = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const int node0 = row0 >> LG;
    float *out = a.scores + ((static_cast<int64_t>(b) * a.n + node0) * a.Hkv + g) * a.stride;
    const int64_t per_node = static_cast<int64_t>(a.Hkv) * a.stride;
    int p = p_begin + warp * 32 + lane;
    float ks = a.k_scale[block_at(p, false)];
    for (int j = 0; j < tiles; ++j, p += Sh::kPages) {
      const float page_scale = exponent_scale(scale_exponent(ks));
      if (j + 1 < tiles) ks = a.k_scale[block_at(p + Sh::kPages, false)];
      if (!wait_bounded(&d_full[j & 1], (j / 2) & 1, abort_flag)) break;
      tc_fence_after();
      for (int c0 = 0; c0 < cols; c0 += 32) {
        float v[32];
        tmem_ld32(tD + (j & 1) * 256 + c0, v);
#pragma unroll
        for (int c = 0; c < 32; c += 4) {
          const float4 s = *reinterpret_cast<const float4 *>(col_scale + c0 + c);
          v[c] *= s.x; v[c + 1] *= s.y; v[c + 2] *= s.z; v[c + 3] *= s.w;
        }
#pragma unroll
        for (int c = 0; c < 32; c += 1 << LG) {
          float best = v[c];
#pragma unroll
          for (int h = 1; h < (1 << LG); ++h) best = fmaxf(best, v[c + h]);
          const int node = (c0 + c) >> LG;
          if (p < p_end && node0 + node < a.n) out[node * per_node + p] = best * page_scale;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&d_free[j & 1]);
      __syncwarp();
    }
  }

  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*abort_flag) {
    if (tid == 0) report(a.status, EAGLE_ERR_TIMEOUT);
    if (warp == 8 && elect_one()) {  // the thread that issued the MMAs: they complete before tensor memory is released
      volatile int never = 0;
      mma_commit(teardown);
      mbar_wait(teardown, 0, &never, 100000000ull);
    }
    __syncthreads();
  }
  if (warp == 8) tmem_dealloc(tmem, 512);
}

template <int DH, int LG>
static cudaError_t launch_score_tc_v(const SelectArgs &a, dim3 grid, int per, cudaStream_t st) {
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = set_smem_limit_once(kv8_score_tc_kernel<DH, LG>, ScoreShape<DH>::kSmem, configured);
  if (e != cudaSuccess) return e;
  return launch_chained(kv8_score_tc_kernel<DH, LG>, grid, dim3(ScoreShape<DH>::kThreads), ScoreShape<DH>::kSmem, st, a, per);
}

template <int DH>
static cudaError_t launch_score_tc_t(const SelectArgs &a, int num_sms, cudaStream_t st) {
  constexpr int kRows = ScoreShape<DH>::kRows, kPages = ScoreShape<DH>::kPages;
  const int blocks = ((a.n << a.log_g) + kRows - 1) / kRows, tiles = (a.max_pages + kPages - 1) / kPages;
  const int64_t base = static_cast<int64_t>(a.B) * a.Hkv * blocks;
  // Chunks of pages: waves of CTAs times the tiles of one and what it spends before
  // its first and after its last tile (about four tiles).
  int chunks = 1;
  double best = 1e30;
  for (int c = 1; c <= tiles; c = c < 16 ? c + 1 : c * 2) {
    const int per = (tiles + c - 1) / c;
    const double cost = static_cast<double>((base * c + num_sms - 1) / num_sms) * (per + 4);
    if (cost < best * 0.97) {
      best = cost;
      chunks = c;
    }
  }
  const int per = (tiles + chunks - 1) / chunks * kPages;
  const dim3 grid((a.max_pages + per - 1) / per, a.B * a.Hkv, blocks);
  switch (a.log_g) {
    case 0: return launch_score_tc_v<DH, 0>(a, grid, per, st);
    case 1: return launch_score_tc_v<DH, 1>(a, grid, per, st);
    case 2: return launch_score_tc_v<DH, 2>(a, grid, per, st);
    case 3: return launch_score_tc_v<DH, 3>(a, grid, per, st);
    case 4: return launch_score_tc_v<DH, 4>(a, grid, per, st);
    default: return launch_score_tc_v<DH, 5>(a, grid, per, st);
  }
}

cudaError_t launch_kv8_score_tc(const SelectArgs &a, int dh, int num_sms, cudaStream_t st) {
  return dh == 128 ? launch_score_tc_t<128>(a, num_sms, st) : launch_score_tc_t<64>(a, num_sms, st);
}

}  // namespace eagle
