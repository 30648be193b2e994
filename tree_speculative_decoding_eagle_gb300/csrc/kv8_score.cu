// Scores of pages: the product of kv8_select.cu as a matrix product on the
// 5th-generation tensor cores, in 8 bits, straight from the bounds' bytes.
//
// D[page, row] = sum over k of A[page, k] B[row, k] with float32 accumulation.  A is
// the bounds as they lie in memory: a page's lower bounds of a head, then its upper
// ones.  A row's whole numbers |q'| <= 128 do not fit e4m3's four bits, but q' =
// 16 a + b with whole |a|, |b| <= 8 does as two numbers, 16 a and b, so B is held
// twice and A meets both: each part has the row's negative numbers against the lower
// bounds, its positive ones against the upper, zeros elsewhere.  Every product is
// exact, every sum a multiple of 1/2 below 2^23.
// Pages are the rows of D, so a thread that reads D back owns a page: the largest
// score over the heads of a node is a maximum over neighbouring columns, within the
// thread, and a node's scores of 32 pages leave a warp as one line.
//
// A CTA takes up to NR query rows (padded: node << LG | head; places past the last
// head repeat head 0) of one sequence and KV head and a chunk of its pages, 128 a tile.
// Roles: eight producer warps (page numbers, and the bounds by TMA gathers of four
// rows of 128 bytes, in the 128-byte swizzle that the MMAs read, a ring of kRing tiles;
// eight, because a warp issues one gather in some 70 cycles: one producer took 2.2 us
// a tile), one thread for the MMAs, four warps that take D from tensor memory (two
// buffers) to the scores (eight with 256 rows).  All but the MMAs' warp make B ready
// first.
//
// What bounds it: HBM with few rows (NR = 32: two CTAs an SM), latency for one request,
// with many rows what a CTA does before its first tile and after its last (rows to B,
// scores out; issue slots 51 %) and the last wave.  Measured (alone, caches cold): 64
// tokens, 64 heads on 8 of 128, pages of 64, 32768 to 131072 keys 40 us (165 MB, 62 % of
// the copy rate: 512 CTAs on 304 places; a further whole wave of 304 equal ones, 159 MB,
// takes 30 us with its choice, 79 %); 16 x 49 nodes, the same heads, 512 pages 29 us (tensor pipe 26 %, ALU
// 39 % of active cycles, 1.7 waves of CTAs; tiles of 128 rows, two CTAs an SM: 4 us
// more); one token, 32 heads, 2048 pages 12 us.
//
// Every wait is bounded; a timeout raises EAGLE_ERR_TIMEOUT in the status word, and
// the CTA completes its copies and MMAs, frees tensor memory and exits.
#include "kv8_select.cuh"
#include "sm100.cuh"
#include "tmap.cuh"

namespace eagle {

using namespace sm100;

template <int DH, int NR>
struct ScoreShape {
  static constexpr int kPages = 128;
  static constexpr int kScorers = NR <= 32 ? 4 : 8;          // warps that take D to the scores
  static constexpr int kThreads = 32 * (kScorers + 9);
  static constexpr int kLines = DH / 64;                     // lines of 128 bytes that a page's two bounds take
  static constexpr int kOcc = NR <= 32 ? 2 : 1;              // CTAs an SM
  static constexpr int kTileBytes = kLines * kPages * 128;   // [line][page][128 bytes]
  static constexpr int kRowBytes = 2 * kLines * NR * 128;    // B: [part][line][row][128 bytes]
  static constexpr int kRing = DH == 128 ? 3 : 6;
  static constexpr int kBufBytes = kRowBytes + kRing * kTileBytes;
  // barriers, tensor-memory slot and abort flag, scales of B's columns: in the gap
  // before the 1 KB-aligned buffers when it holds them, else after the buffers
  static constexpr int kBarBytes = 192 + NR * 4;
  static constexpr int kUsed = kBufBytes + (1008 > 2 * kBarBytes - 16 ? 1008 : 2 * kBarBytes - 16);
  static constexpr int kTmemCols = 2 * NR;
  // no more CTAs an SM than tensor memory has room for
  static constexpr int kLeast = kOcc == 1 ? 120 * 1024 : 80 * 1024;
  static constexpr int kSmem = kUsed < kLeast ? kLeast : kUsed;
  static_assert(kOcc * (kSmem + 1024) <= 233472, "shared memory budget");
  static_assert(kOcc * kTmemCols <= 512, "tensor memory budget");
  static_assert((2 * kRing + 6) * 8 + 8 <= 192, "barriers");
};

// D[tmem] (+)= A B^T of e4m3 numbers with float32 accumulation (M 128, K 32).
__device__ __forceinline__ void mma_e4m3_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}
// Four rows of a map whose boxes are one row high, one after another from dst on.
__device__ __forceinline__ void tma_gather4(void *dst, const CUtensorMap *map, int r0, int r1, int r2, int r3, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(smem_u32(bar))
      : "memory");
}
// Eight elements of a row (bf16, the ones that are not finite as zeros) times f as
// whole numbers q' = 16 a + b, e4m3: in `high` the eight numbers 16 a, in `low` b.
// Rounding to whole numbers by adding 1.5 * 2^23; |q' / 16 - a| <= 1/2 but for what
// rounding q' adds, so |b| <= 8.
__device__ __forceinline__ void whole_parts(const uint4 &x, float f, uint2 &high, uint2 &low) {
  constexpr float kBig = 12582912.f;
  float v[8], hi[8], lo[8];
  VecTraits<__nv_bfloat16>::unpack(x, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float y = fminf(fmaxf(v[i] * f, -128.f), 128.f);
    const float whole = (y + kBig) - kBig, a = fmaf(y, 0.0625f, kBig) - kBig;
    hi[i] = 16.f * a;
    lo[i] = fmaf(-16.f, a, whole);
  }
  high = make_uint2(e4m3_pair(hi[0], hi[1]) | (e4m3_pair(hi[2], hi[3]) << 16), e4m3_pair(hi[4], hi[5]) | (e4m3_pair(hi[6], hi[7]) << 16));
  low = make_uint2(e4m3_pair(lo[0], lo[1]) | (e4m3_pair(lo[2], lo[3]) << 16), e4m3_pair(lo[4], lo[5]) | (e4m3_pair(lo[6], lo[7]) << 16));
}
// 0xff in the bytes of the elements that are negative.
__device__ __forceinline__ uint2 negative_bytes(const uint4 &x) {
  const uint32_t a = __byte_perm(x.x, x.y, 0x7531), b = __byte_perm(x.z, x.w, 0x7531);  // the upper byte of each
  return make_uint2(((a >> 7) & 0x01010101u) * 0xffu, ((b >> 7) & 0x01010101u) * 0xffu);
}

template <int DH, int LG, int NR>
__global__ void __launch_bounds__(ScoreShape<DH, NR>::kThreads, ScoreShape<DH, NR>::kOcc)
    kv8_score_kernel(const __grid_constant__ CUtensorMap map, SelectArgs a, int pages_per_cta) {
  using Sh = ScoreShape<DH, NR>;
  constexpr int kScorers = Sh::kScorers, kProducerWarp = kScorers, kProducers = 8, kMmaWarp = kScorers + 8, LINES = Sh::kLines;
  extern __shared__ unsigned char score_smem[];
  const uint32_t gap = (1024u - (smem_u32(score_smem) & 1023u)) & 1023u;
  unsigned char *sm = score_smem + gap;
  unsigned char *sB = sm, *sA = sm + Sh::kRowBytes;
  unsigned char *ctl = score_smem + (gap >= static_cast<uint32_t>(Sh::kBarBytes) ? 0u : gap + Sh::kBufBytes);
  uint64_t *full = reinterpret_cast<uint64_t *>(ctl);  // a tile of A has landed
  uint64_t *empty = full + Sh::kRing;                  // and is read
  uint64_t *d_full = empty + Sh::kRing, *d_free = d_full + 2, *b_full = d_free + 2, *teardown = b_full + 1;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(teardown + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  float *col_scale = reinterpret_cast<float *>(ctl + 192);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bg = blockIdx.y, b = bg / a.Hkv, g = bg % a.Hkv;
  const int row0 = blockIdx.z * NR, rows = min((a.n << LG) - row0, NR), cols = (rows + 31) & ~31;
  if (tid == 0) {
    for (int i = 0; i < Sh::kRing; ++i) {
      mbar_init(&full[i], kProducers);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_free[i], kScorers);
    }
    mbar_init(b_full, kScorers + kProducers);
    mbar_init(teardown, 1);
    *abort_flag = 0;
    mbar_init_fence();
    prefetch_tmap(&map);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, Sh::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  const int np = live_pages(a, b);
  const int p_begin = blockIdx.x * pages_per_cta, p_end = min(np, p_begin + pages_per_cta);
  const int tiles = p_end > p_begin ? (p_end - p_begin + Sh::kPages - 1) / Sh::kPages : 0;
  const int32_t *table = a.block_table + static_cast<int64_t>(b) * a.max_pages;
  // A page number as the table has it, and (later, so that nothing waits for it here)
  // its block of the pool: page 0's past the chunk or outside the pool.
  const auto page_at = [&](int p) { return p < p_end ? __ldg(table + p) : 0; };
  const auto block_of = [&](int page, bool tell) {
    if (page < 0 || page >= a.num_pages) {
      if (tell) report(a.status, EAGLE_ERR_INVALID);
      page = 0;
    }
    return page * a.Hkv + g;  // num_pages * Hkv fits 30 bits
  };
  int issued = 0;  // producer: tiles requested

  // The query rows into B: DH / 8 neighbouring lanes hold a row, four rows a thread
  // in flight.
  const auto build_rows = [&] {
    constexpr int CPR = DH / 8, AHEAD = 4, kBuilders = Sh::kThreads - 32;
    for (int i0 = tid; i0 < cols * CPR; i0 += AHEAD * kBuilders) {  // whole warps: cols is a multiple of 32
      uint4 x[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int idx = i0 + k * kBuilders, at = row0 + idx / CPR, node = at >> LG, h = at & ((1 << LG) - 1);
        x[k] = make_uint4(0, 0, 0, 0);
        if (idx < cols * CPR && node < a.n)
          x[k] = __ldg(reinterpret_cast<const uint4 *>(
              a.q + ((static_cast<int64_t>(b) * a.n + node) * a.Hq + g * a.G + (h < a.G ? h : 0)) * DH + idx % CPR * 8));
      }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int idx = i0 + k * kBuilders, r = idx / CPR, c = idx % CPR;
        if (idx >= cols * CPR) break;
        x[k] = finite8(x[k]);
        float amax = amax8(x[k]);
#pragma unroll
        for (int o = 1; o < CPR; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const int e = whole_exponent(amax);
        uint2 hi, lo;
        whole_parts(x[k], exponent_scale(-e), hi, lo);
        const uint2 neg = negative_bytes(x[k]);
#pragma unroll
        for (int side = 0; side < 2; ++side) {  // against the lower bounds, the upper ones
          const uint2 keep = side ? make_uint2(~neg.x, ~neg.y) : neg;
          const int byte = (LINES == 2 ? 0 : side * 64) + c * 8;  // of line `side`, or of half a line
          unsigned char *at_b = sB + (LINES == 2 ? side : 0) * (NR * 128) + sw128_offset(r, byte >> 4) + (byte & 8);
          *reinterpret_cast<uint2 *>(at_b) = make_uint2(hi.x & keep.x, hi.y & keep.y);
          *reinterpret_cast<uint2 *>(at_b + LINES * (NR * 128)) = make_uint2(lo.x & keep.x, lo.y & keep.y);
        }
        if (c == 0) col_scale[r] = exponent_scale(e);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(b_full);
    __syncwarp();
  };

  if (warp == kMmaWarp) {
    if (tiles && elect_one()) {
      // B came through the generic proxy: the fence after the wait orders that before
      // the MMAs.  A came by TMA.
      const uint32_t id = (1u << 4) | (static_cast<uint32_t>(cols >> 3) << 17) | (static_cast<uint32_t>(Sh::kPages >> 4) << 24);
      const uint32_t a_lo = static_cast<uint32_t>(sdesc_sw128(smem_u32(sA), 16, 1024));
      const uint32_t b_lo = static_cast<uint32_t>(sdesc_sw128(smem_u32(sB), 16, 1024));
      const bool ok = wait_bounded(b_full, 0, abort_flag);
      fence_async_smem();
      for (int j = 0; j < tiles && ok; ++j) {
        const int st = j % Sh::kRing;
        if (!wait_bounded(&full[st], (j / Sh::kRing) & 1, abort_flag)) break;
        if (j >= 2 && !wait_bounded(&d_free[j & 1], (j / 2 - 1) & 1, abort_flag)) break;
        tc_fence_after();
        const uint32_t ad = anew(a_lo + st * (Sh::kTileBytes >> 4)), bd = anew(b_lo);
#pragma unroll
        for (int s = 0; s < 2 * LINES * 4; ++s) {  // part, line, 32 bytes of it
          const int part = s / (LINES * 4), line = s / 4 % LINES;
          mma_e4m3_ss(tmem + (j & 1) * NR, ad + ((line * (Sh::kPages * 128) + s % 4 * 32) >> 4),
                      bd + (((part * LINES + line) * (NR * 128) + s % 4 * 32) >> 4), id, s > 0);
        }
        mma_commit(&empty[st]);
        mma_commit(&d_full[j & 1]);
      }
    }
    __syncwarp();
  } else if (warp >= kProducerWarp) {
    // Of a tile, a warp requests 16 pages: lane l (below 4) pages 4 l .. 4 l + 3 of
    // them, their numbers two tiles ahead.
    const int first = (warp - kProducerWarp) * 16 + 4 * (lane & 3);
    int ahead[2][4];
    const auto look = [&](int j, int (&to)[4]) {
#pragma unroll
      for (int i = 0; i < 4; ++i) to[i] = page_at(p_begin + j * Sh::kPages + first + i);
    };
    look(0, ahead[0]);
    look(1, ahead[1]);
    for (int j0 = 0; j0 < tiles; j0 += 2) {
      bool ok = true;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int j = j0 + k, st = j % Sh::kRing;
        if (!ok || j >= tiles) break;
        int blk[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) blk[i] = block_of(ahead[k][i], lane < 4) * LINES;
        look(j + 2, ahead[k]);
        if (j >= Sh::kRing && !wait_bounded(&empty[st], (j / Sh::kRing - 1) & 1, abort_flag)) { ok = false; break; }
        __syncwarp();
        if (lane == 0) mbar_arrive_expect_tx(&full[st], Sh::kTileBytes / kProducers);
        __syncwarp();
        unsigned char *dst = sA + st * Sh::kTileBytes + first * 128;
        if (lane < 4) {
#pragma unroll
          for (int line = 0; line < LINES; ++line)
            tma_gather4(dst + line * (Sh::kPages * 128), &map, blk[0] + line, blk[1] + line, blk[2] + line, blk[3] + line, &full[st]);
        }
        __syncwarp();
        issued = j + 1;
      }
      if (j0 == 0) build_rows();  // with the first two tiles on their way
      if (!ok) break;
    }
    __syncwarp();
  } else {
    if (tiles) build_rows();
    // ------------------------------------------------------- D to the scores
    // warps 0 .. 3 have D's rows 32 w .., with eight each has every other run of columns
    const int quarter = warp & 3, run0 = warp >> 2;
    const uint32_t tD = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const int node0 = row0 >> LG;
    float *out = a.scores + ((static_cast<int64_t>(b) * a.n + node0) * a.Hkv + g) * a.stride;
    const int64_t per_node = static_cast<int64_t>(a.Hkv) * a.stride;
    int p = p_begin + quarter * 32 + lane;
    float ks = a.k_scale[block_of(page_at(p), false)];
    int page = page_at(p + Sh::kPages);  // a tile ahead of its scale
    const bool ready = tiles && wait_bounded(b_full, 0, abort_flag);  // all warps' column scales
    for (int j = 0; j < tiles && ready; ++j, p += Sh::kPages) {
      const float page_scale = exponent_scale(scale_exponent(ks));
      ks = a.k_scale[block_of(page, false)];
      page = page_at(p + 2 * Sh::kPages);
      if (!wait_bounded(&d_full[j & 1], (j / 2) & 1, abort_flag)) break;
      tc_fence_after();
      for (int c0 = 32 * run0; c0 < cols; c0 += 8 * kScorers) {
        float v[32];
        tmem_ld32(tD + (j & 1) * NR + c0, v);
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
          if (p < p_end && node0 + node < a.n) out[node * per_node + p] = fmaf(best, page_scale, 0.f);  // a zero is +0: keys are ordered by bits
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
    volatile int never = 0;
    if (warp == kMmaWarp && elect_one()) {  // the thread that issued the MMAs: they complete before tensor memory is released
      mma_commit(teardown);
      mbar_wait(teardown, 0, &never, 100000000ull);
    }
    if (warp >= kProducerWarp && warp < kMmaWarp && lane == 0)  // copies still in flight complete before shared memory is released
      for (int j = max(0, issued - Sh::kRing); j < issued; ++j)
        mbar_wait(&full[j % Sh::kRing], (j / Sh::kRing) & 1, &never, 100000000ull);
    __syncthreads();
  }
  if (warp == kMmaWarp) tmem_dealloc(tmem, Sh::kTmemCols);
}

template <int DH, int LG, int NR>
static cudaError_t launch_score_v(const CUtensorMap &map, const SelectArgs &a, dim3 grid, int per, cudaStream_t st) {
  using Sh = ScoreShape<DH, NR>;
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = set_smem_limit_once(kv8_score_kernel<DH, LG, NR>, Sh::kSmem, configured);
  if (e != cudaSuccess) return e;
  return launch_chained(kv8_score_kernel<DH, LG, NR>, grid, dim3(Sh::kThreads), Sh::kSmem, st, map, a, per);
}

template <int DH, int NR>
static cudaError_t launch_score_t(const CUtensorMap &map, const SelectArgs &a, int num_sms, cudaStream_t st) {
  using Sh = ScoreShape<DH, NR>;
  const int blocks = ((a.n << a.log_g) + NR - 1) / NR, tiles = (a.max_pages + Sh::kPages - 1) / Sh::kPages;
  const int64_t base = static_cast<int64_t>(a.B) * a.Hkv * blocks, slots = static_cast<int64_t>(num_sms) * Sh::kOcc;
  // Chunks of pages: waves of CTAs times the tiles of one and what it spends before
  // its first and after its last tile (about four tiles).
  int chunks = 1;
  double best = 1e30;
  for (int c = 1; c <= tiles; c = c < 16 ? c + 1 : c * 2) {
    const double load = static_cast<double>(base * c) / slots;
    const double waves = load < 3.0 ? static_cast<double>((base * c + slots - 1) / slots) : load + 0.5;
    const double cost = waves * ((tiles + c - 1) / c + 4);
    if (cost < best * 0.97) {
      best = cost;
      chunks = c;
    }
  }
  const int per = (tiles + chunks - 1) / chunks * Sh::kPages;
  const dim3 grid((a.max_pages + per - 1) / per, a.B * a.Hkv, blocks);
  switch (a.log_g) {
    case 0: return launch_score_v<DH, 0, NR>(map, a, grid, per, st);
    case 1: return launch_score_v<DH, 1, NR>(map, a, grid, per, st);
    case 2: return launch_score_v<DH, 2, NR>(map, a, grid, per, st);
    case 3: return launch_score_v<DH, 3, NR>(map, a, grid, per, st);
    case 4: return launch_score_v<DH, 4, NR>(map, a, grid, per, st);
    default: return launch_score_v<DH, 5, NR>(map, a, grid, per, st);
  }
}

// The bounds as lines of 128 bytes (a page's two bounds of a head are one line or
// two), in boxes of one line, swizzled.
static bool make_bounds_map(CUtensorMap *map, const void *base, int64_t lines) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {128, static_cast<cuuint64_t>(lines)};
  cuuint64_t strides[1] = {128};
  cuuint32_t box[2] = {128, 1}, estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t launch_kv8_score(const SelectArgs &a, int dh, int num_sms, cudaStream_t st) {
  CUtensorMap map;
  if (!make_bounds_map(&map, a.bounds, static_cast<int64_t>(a.num_pages) * a.Hkv * (dh / 64))) return cudaErrorInvalidValue;
  const bool few = (a.n << a.log_g) <= 32;
  if (dh == 128) return few ? launch_score_t<128, 32>(map, a, num_sms, st) : launch_score_t<128, 256>(map, a, num_sms, st);
  return few ? launch_score_t<64, 32>(map, a, num_sms, st) : launch_score_t<64, 256>(map, a, num_sms, st);
}

}  // namespace eagle
