// The kernel of stage 3 over the 8-bit paged cache: tree-masked attention whose prefix keys
// and values are e4m3 numbers with a power-of-two scale for each page and head.
//
// The mathematics.  Everything runs in f16 on the tensor cores.  An e4m3 number is
// an f16 number.  A bf16 query row becomes f16 over a power of two of its own, tree
// keys and values over one that a block of nodes shares (16, or a tile of 64 or 128
// in the one-scale form); both put the largest magnitude M at 2^8 to 2^9, so what is
// above 2^-25 M is exact and the rest off by up to 2^-33 M.  The powers of two
// never touch the tiles; they go into the softmax's float32 arithmetic.  With
// q = 2^a q', k = 2^ke k', v = 2^ve v' (ke, ve of a group of 16 keys, which no
// page splits):
//   s  = (scale log2e 2^(a+ke)) <q', k'>           score, base 2
//   P' = 2^(s + ve - m + 6),  m >= max(s + ve) - 8     in f16
//   O  = sum P' v',  l = sum_groups 2^-ve sum P',  out = O / l,
//   lse = ln 2 (m - 6 + log2 l)
// so P' stays below 2^14 and is rounded to 11 bits (bf16 would leave 8), down
// to 2^-20 of the row's largest; smaller ones are off by up to 2^-31 of it
// (f16's subnormals).  ve is part of P': on a page whose value scale is 2^-20 of
// another's, weights as large have those bits no more.  The cache's K and V are not
// rounded at all.
//
// One CTA per (sequence b, KV head g, group of MT 128-row M-tiles, KV split);
// query rows are (node, head-in-group) pairs, key tiles hold NK keys, first the
// prefix, then the tree nodes masked with the ancestor bits.  Roles:
//   * two producer warps, K's and V's: page numbers and scales two batches of 32
//     groups ahead, bytes by TMA into a ring of S8 staging buffers;
//   * converter warps: staging bytes (tree tiles: bf16 from global memory) to f16
//     in rings of SF tiles, K's and V's, in the 128-byte swizzle the MMAs read;
//     rows past the prefix's end become zeros.  K's ring runs ahead:
//     its tiles are free once S is taken, V's only after P.V;
//   * MMA thread and one softmax warpgroup per M-tile as in tree_attn_tc.cu:
//     S = Q K^T from shared memory, P from tensor memory.
// KV split over up to 8 CTAs and the merge of their results as there too.
//
// What bounds it.  With grouped heads, the softmax warps: of 3300 cycles that a
// 128-key tile of two M-tiles took at dh 64 (a trace of each role's waits, before
// the one-scale form) they waited in 360; in the one-scale form tensor pipe 34 %,
// ex2 35 %, issue slots 54 % of active cycles, HBM 9 %.  With few rows, each CTA's chain (length -
// page number - bytes - f16 - S - P - O) through the warps.  Measured (the same
// call on a 16-bit cache): 16 x 49 nodes, 64 heads on 8 of 128, 4096 keys 150 us
// (184; 702 TFLOP/s, 37 % of cuBLAS's bf16 rate); 64 x 61 nodes, 64 heads on 8 of
// 64, 8192 keys 690 us (688; 760 TFLOP/s, 40 %); 61 nodes, 32 heads of 128, 2048
// keys 22.1 us (17.8); 8 x 51 nodes, 40 heads of 128, 1024 to 4096 keys 127 us (125);
// a chain of 1024 nodes, 64 heads on 8 of 128, after 4096 keys 226 us.
// Two M-tiles a CTA (one converter warpgroup, which then takes K and V in turn)
// from 129 rows on, since a tile's conversion is shared by its M-tiles; two CTAs an
// SM up to 64 rows, where latency counts.
//
// Every wait is bounded; a timeout raises EAGLE_ERR_TIMEOUT in the status
// word and the CTA drains its copies and MMAs, frees tensor memory and exits.
#pragma once

#include "kv8_attn.cuh"

namespace eagle {

using namespace sm100;

// QR: query rows held per M-tile region (64 when there are at most 64: the
// 128-row MMAs then read rows 64-127 from what follows, and those rows' results
// are never used).  OCC: CTAs per SM.
// ONE: every key tile has one scale (pages no shorter than a tile; the tree's
// nodes then share a tile's power of two), so the softmax does nothing group by
// group.  Measured with it / without: 64 x 61 nodes, 64 heads on 8 of 64, 8192
// keys 690 / 737 us; 16 x 49 nodes, 64 heads on 8 of 128, 4096 keys 150 / 157 us.  A
// choice made per tile in one kernel costs more than it gains (registers spill).
template <int DH, int MT, int NK, int SF, int S8, int QR, int OCC, bool ONE>
struct Kv8Shape {
  static constexpr int kRegions = DH / 64;
  static constexpr int kQRegionBytes = QR * 128;
  static constexpr int kQBytes = MT * kRegions * kQRegionBytes;
  static constexpr int kTileBytes = kRegions * NK * 128;  // one f16 K (or V) tile
  static constexpr int kByteTile = NK * DH;               // one e4m3 K (or V) tile
  // Q, the rings of f16 K and V tiles, the staging of K's and V's bytes
  static constexpr int kVOff = kQBytes + SF * kTileBytes;
  static constexpr int kStagingOff = kVOff + SF * kTileBytes;
  static constexpr int kBarOff = kStagingOff + S8 * 2 * kByteTile;
  static constexpr int kGroups = NK / 16;
  static constexpr int kNumBars = 4 * S8 + 4 * SF + 4 * MT + 2 + (ONE ? 2 : 0);
  static constexpr int kNamedWords = MT == 1 ? QR / 64 : 64;   // mask words of n nodes (no more nodes than rows)
  // barriers, tensor-memory slot and abort flag, scales of the tiles' groups, the
  // nodes that the CTA's rows name, exponents of the query rows
  static constexpr int kScaleSlots = S8 + SF + 3;         // tiles between K's producer and the softmax
  static constexpr int kScaleOff = (kNumBars * 8 + 8 + 15) / 16 * 16;
  static constexpr int kBarBytes = kScaleOff + kScaleSlots * kGroups * 8 + kNamedWords * 8 + (ONE ? 32 : 0) + MT * QR;
  // The barriers sit in the gap before the 1 KB-aligned buffers when it holds
  // them, else after the buffers.
  static constexpr int kSmem = kBarOff + (1008 > 2 * kBarBytes - 16 ? 1008 : 2 * kBarBytes - 16);
  // Warpgroups that convert: K's and V's, or with two M-tiles (whose softmax has
  // the use of the issue slots) one that takes K and V in turn.
  static constexpr int kConvertGroups = MT == 1 ? 2 : 1;
  static constexpr int kGroupsAll = MT + kConvertGroups + 1;
  static constexpr int kThreads = kGroupsAll * 128;
  static constexpr int kColS = 0;                         // S_t at t*NK
  static constexpr int kColP = MT * NK;                   // P_t at kColP + t*NK/2
  static constexpr int kColO = MT * NK + MT * NK / 2;     // O_t at kColO + t*DH
  static constexpr int kCols = kColO + MT * DH;
  static constexpr int kTmemCols = kCols <= 128 ? 128 : (kCols <= 256 ? 256 : 512);
  // Registers: what a thread is launched with, and the warpgroups' shares of
  // it (softmax, converters, producers and MMA); they add up to the launch's.
  static constexpr int kLaunchRegs = 65536 / (kThreads * OCC) / 8 * 8;
  static constexpr int kRegsOther = kLaunchRegs < 80 ? 40 : 64;
  static constexpr int kRegsConvert = kLaunchRegs < 80 ? 40 : (kConvertGroups == 1 ? 72 : 56);
  static constexpr int kRegsLeft = (kGroupsAll * kLaunchRegs - kRegsOther - kConvertGroups * kRegsConvert) / MT / 8 * 8;
  static constexpr int kRegsSoftmax = kRegsLeft > 208 ? 208 : kRegsLeft;
  static_assert(QR == 128 || (QR == 64 && MT == 1), "64-row regions with one M-tile only");
  static_assert(!ONE || kConvertGroups == 1, "four warps exchange a tree tile's largest magnitude");
  static_assert(kCols <= 512 && kTmemCols * OCC <= 512, "tensor memory budget");
  static_assert(kSmem <= 232448 && OCC * (kSmem + 1024) <= 233472, "shared memory budget");
  static_assert(MT * kRegsSoftmax + kConvertGroups * kRegsConvert + kRegsOther <= kGroupsAll * kLaunchRegs, "register budget");
  // split: fp32 O rows in the rings and the staging after them, (m, l) in Q's buffer
  static_assert(MT * 128 * DH * 4 <= kBarOff - kQBytes, "partial O fits the rings and the staging");
  static_assert(MT * 128 * 8 <= kQBytes, "(m, l) fit the Q buffer");
};

template <int N> __device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }

// The same with A (packed f16 pairs) in tensor memory.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}

// The scales of a 16-key group as the softmax takes them: two powers of two in
// one word (the upper half of the float 2^ke, that of 2^-ve below it), and ve.
__device__ __forceinline__ uint32_t pack_scales(float k_pow2, float v_inverse) {
  return (__float_as_uint(k_pow2) & 0xffff0000u) | (__float_as_uint(v_inverse) >> 16);
}

// 64 fp32 columns of this thread's tensor-memory lane as two runs of 32, one wait.
__device__ __forceinline__ void tmem_ld32x2(uint32_t taddr, float (&a)[32], float (&b)[32]) {
  uint32_t r[32], q[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, "
      "%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3]), "=r"(q[4]), "=r"(q[5]), "=r"(q[6]), "=r"(q[7]), "=r"(q[8]), "=r"(q[9]), "=r"(q[10]), "=r"(q[11]), "=r"(q[12]), "=r"(q[13]), "=r"(q[14]), "=r"(q[15]), "=r"(q[16]), "=r"(q[17]), "=r"(q[18]), "=r"(q[19]), "=r"(q[20]), "=r"(q[21]), "=r"(q[22]), "=r"(q[23]), "=r"(q[24]), "=r"(q[25]), "=r"(q[26]), "=r"(q[27]), "=r"(q[28]), "=r"(q[29]), "=r"(q[30]), "=r"(q[31])
      : "r"(taddr), "r"(taddr + 32)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    a[i] = __uint_as_float(r[i]);
    b[i] = __uint_as_float(q[i]);
  }
}

__device__ __forceinline__ bool unlikely(bool x) { return __builtin_expect(x, 0); }

// What the launch over selected pages has beside (tree_attn_kv8_pages.cu): for each
// (sequence, KV head, M-group) the pages that any of its nodes selects, and for each
// of its nodes a bit a listed page.
struct Kv8UnionArgs : Kv8Args {
  const int32_t *lens;   // [cl]: keys of the listed pages
  const int32_t *pages;  // [cl][list_stride]: pages of the pool
  const uint32_t *bits;  // [cl][group_nodes][bit_words]
  int list_stride, group_nodes, bit_words;
};
template <bool SEL> struct Kv8KernelArgs { using type = Kv8Args; };
template <> struct Kv8KernelArgs<true> { using type = Kv8UnionArgs; };

// SEL: the prefix is the listed pages, one after another; a row counts those whose bit
// its node has.  MERGE: 0 the grid does not split the KV range; 1 the S splits of an item are
// one cluster and merge in this kernel; 2 tree_attn_kv8_merge_kernel merges.
template <int DH, int MT, int NK, int SF, int S8, int QR, int OCC, bool ONE, int MERGE, bool SEL>
__global__ void __launch_bounds__((MT == 1 ? 4 : MT + 2) * 128, OCC)
    tree_attn_kv8_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                         typename Kv8KernelArgs<SEL>::type a) {
  using Sh = Kv8Shape<DH, MT, NK, SF, S8, QR, OCC, ONE>;
  constexpr bool SPLIT = MERGE != 0;
  constexpr int NH = NK / 64, GR = Sh::kGroups;
  extern __shared__ unsigned char raw_smem[];
  // offsets from raw_smem, not address arithmetic: the compiler has to see that
  // every access is to shared memory (a generic one costs registers and time)
  const uint32_t gap = (1024u - (smem_u32(raw_smem) & 1023u)) & 1023u;
  unsigned char *sm = raw_smem + gap;
  unsigned char *sQ = sm;
  unsigned char *sK = sm + Sh::kQBytes, *sV = sm + Sh::kVOff;
  unsigned char *s8 = sm + Sh::kStagingOff;
  unsigned char *ctl = raw_smem + (gap >= static_cast<uint32_t>(Sh::kBarBytes) ? 0u : gap + Sh::kBarOff);
  // K's barriers, then V's: bytes landed, staging free, f16 tile written, tile read
  uint64_t *bytes_full = reinterpret_cast<uint64_t *>(ctl);  // [K, V][S8]
  uint64_t *bytes_empty = bytes_full + 2 * S8;
  uint64_t *tile_full = bytes_empty + 2 * S8;                // [K, V][SF]
  uint64_t *tile_empty = tile_full + 2 * SF;
  uint64_t *s_full = tile_empty + 2 * SF;
  uint64_t *s_free = s_full + MT;
  uint64_t *p_full = s_free + MT;
  uint64_t *o_done = p_full + MT;
  uint64_t *q_full = o_done + MT;
  uint64_t *teardown = q_full + 1;
  uint64_t *tree_sync = teardown + 1;  // [K, V]: the converter warps' exchange (ONE)
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(tree_sync + (ONE ? 2 : 0));
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  uint2 *scales = reinterpret_cast<uint2 *>(ctl + Sh::kScaleOff);                   // [kScaleSlots][GR]
  unsigned short *named = reinterpret_cast<unsigned short *>(scales + Sh::kScaleSlots * GR);  // a bit a node, 16 to a group
  volatile float *tree_max = reinterpret_cast<volatile float *>(named + 4 * Sh::kNamedWords);  // [K, V][4 converter warps]
  signed char *q_exp = reinterpret_cast<signed char *>(named + 4 * Sh::kNamedWords) + (ONE ? 32 : 0);  // [MT * QR]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // SEL: every sequence's full M-groups come first; the last ones, which have fewer
  // rows, then fill what those leave of the last wave (16 x 49 nodes with 8 heads, 1.7
  // waves: 131 -> 126 us; 64 x 61 nodes, 6.7 waves, whose two groups then find less of
  // each other's pages in L2: 321 -> 323; a choice at run time costs both 2 %).
  const int split = blockIdx.x, mg = SEL ? blockIdx.z : blockIdx.y, mgroups = SEL ? gridDim.z : gridDim.y;
  const int bg = SEL ? blockIdx.y : blockIdx.z, b = bg / a.Hkv, g = bg % a.Hkv;
  const int n = a.n;
  constexpr int kConvertWarp = MT * 4, kProducerWarp = kConvertWarp + 4 * Sh::kConvertGroups, kMmaWarp = kProducerWarp + 2;

  const int32_t *len_at = a.kv_len + b;
  if constexpr (SEL) len_at = a.lens + static_cast<int64_t>(bg) * mgroups + mg;
  if (tid == 0) prefetch_l2(len_at);
  if (tid == 32) {
    for (int i = 0; i < 2 * S8; ++i) {
      mbar_init(&bytes_full[i], 2);
      mbar_init(&bytes_empty[i], 4);
    }
    for (int i = 0; i < 2 * SF; ++i) {
      mbar_init(&tile_full[i], 4);
      mbar_init(&tile_empty[i], 1);
    }
    for (int t = 0; t < MT; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&s_free[t], 4);
      mbar_init(&p_full[t], 4);
      mbar_init(&o_done[t], 1);
    }
    mbar_init(q_full, 4 * MT);
    mbar_init(teardown, 1);
    for (int i = 0; i < (ONE ? 2 : 0); ++i) mbar_init(&tree_sync[i], 4);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (MT > 1 && a.W > 1) {
    if (tid >= 64 && tid < 64 + 2 * Sh::kNamedWords) reinterpret_cast<uint32_t *>(named)[tid - 64] = 0;
    __syncthreads();
  }
  pdl_wait();  // inputs of this step come from earlier kernels
  if (warp == kMmaWarp) {
    tmem_alloc(tmem_slot, Sh::kTmemCols);
    tmem_relinquish();
  }
  const int kv_len = *len_at;
  const int rows_total = n * a.G;
  // The nodes that any of the CTA's rows names: their mask words or'ed, so that
  // padding decides no block's power of two.  Here, while kv_len is on its way, since
  // a role's code pays for every register: in a warp's role of its own 70B takes 188
  // us, in the converters 160, here 150 (148 without).
  if (MT == 1 || a.W == 1) {  // at most 128 nodes (one M-tile), or 64: one warp, every row
    if (split == a.S - 1 && warp == kMmaWarp + 1) {
      const uint64_t *words = a.mask + static_cast<int64_t>(b) * n * a.W;
      for (int w = 0; w < a.W; ++w) {
        uint64_t any = 0;
#pragma unroll
        for (int u = 0; u < (MT == 1 ? QR : 64) / 32; ++u)
          if (lane + 32 * u < n) any |= words[(lane + 32 * u) * a.W + w];
        const uint32_t lo = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(any));
        const uint32_t hi = __reduce_or_sync(0xffffffffu, static_cast<uint32_t>(any >> 32));
        if (lane == 0) reinterpret_cast<uint2 *>(named)[w] = make_uint2(lo, hi);
      }
    }
  } else if (split == a.S - 1) {  // threads are words, and rows where there are fewer words
    const uint64_t *words = a.mask + static_cast<int64_t>(b) * n * a.W;
    const int i1 = (min(rows_total, (mg + 1) * MT * 128) - 1) / a.G;
    const int wl = a.W > 16 ? 32 : a.W > 8 ? 16 : a.W > 4 ? 8 : a.W > 2 ? 4 : a.W;  // words side by side
    for (int w = lane & (wl - 1); w < ((a.W + wl - 1) & ~(wl - 1)); w += wl) {
      uint64_t any = 0;
#pragma unroll 4
      for (int i = mg * MT * 128 / a.G + tid / wl; i <= i1; i += Sh::kThreads / wl)
        if (w < a.W) any |= words[static_cast<int64_t>(i) * a.W + w];
      uint32_t lo = static_cast<uint32_t>(any), hi = static_cast<uint32_t>(any >> 32);
      for (int o = wl; o < 32; o *= 2) {
        lo |= __shfl_xor_sync(0xffffffffu, lo, o);
        hi |= __shfl_xor_sync(0xffffffffu, hi, o);
      }
      if (lane < wl && w < a.W) {
        atomicOr(reinterpret_cast<uint32_t *>(named) + 2 * w, lo);
        atomicOr(reinterpret_cast<uint32_t *>(named) + 2 * w + 1, hi);
      }
    }
  }
  const int L = SEL ? kv_len : static_cast<int>(min(static_cast<int64_t>(max(kv_len, 0)), static_cast<int64_t>(a.max_pages) << a.log_page));
  const int n_ptiles = (L + NK - 1) / NK;
  const int tps = (n_ptiles + a.S - 1) / a.S;
  const int p0 = min(n_ptiles, split * tps), p1 = min(n_ptiles, p0 + tps);
  // Key tiles of this CTA: prefix tiles from pfx0, tree tiles from tree0.  A single
  // tree tile comes first (it needs no page numbers); several come last, so
  // that the producers' scales never wait for them.
  const int np = p1 - p0, ntt = (split == a.S - 1) ? (n + NK - 1) / NK : 0, T = np + ntt;
  const int pfx0 = ntt == 1 ? 1 : 0, tree0 = ntt == 1 ? 0 : np;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  int issued = 0;  // producers: tiles requested
  bool part_have = false;
  float part_m = -INFINITY, part_l = 0.f;

  if (warp >= kProducerWarp) {
    regs_dec<Sh::kRegsOther>();
    if (warp < kMmaWarp) {
      // ----------------------------------------------- producers: K's, V's warp
      // Lane i of batch k looks after group 32k + i of this CTA's prefix keys.
      const int kv = warp - kProducerWarp;
      const CUtensorMap *map = kv ? &v_map : &k_map;
      uint64_t *full = bytes_full + kv * S8, *empty = bytes_empty + kv * S8;
      if (lane == 0) prefetch_tmap(map);
      constexpr int TPB = 32 / GR;  // tiles a batch
      const int key_end = min(L, p1 * NK);
      const auto page_at = [&](int batch) {
        const int key = p0 * NK + (batch * 32 + lane) * 16;
        if (key >= key_end) return 0;
        if constexpr (SEL) return a.pages[(static_cast<int64_t>(bg) * mgroups + mg) * a.list_stride + (key >> a.log_page)];
        const int page = a.block_table[static_cast<int64_t>(b) * a.max_pages + (key >> a.log_page)];
        if (page >= 0 && page < a.num_pages) return page;
        report(a.status, EAGLE_ERR_INVALID);  // outside the pool: read page 0
        return 0;
      };
      int page = page_at(0), page_next = page_at(1);
      // K's warp also lists the scales of both: the softmax needs them with S
      const auto scale_at = [&](const float *of, int pg) { return kv ? 1.f : of[static_cast<int64_t>(pg) * a.Hkv + g]; };
      float ks = scale_at(a.k_scale, page), vs = scale_at(a.v_scale, page), ks_next = 1.f, vs_next = 1.f;
      for (int j = 0; j < np; ++j) {
        if (j % TPB == 0) {
          if (j) {
            page = page_next; ks = ks_next; vs = vs_next;
            page_next = page_at(j / TPB + 1);
          }
          // requested now, looked at a batch later
          ks_next = scale_at(a.k_scale, page_next);
          vs_next = scale_at(a.v_scale, page_next);
        }
        const int st = j % S8;
        if (j >= S8 && unlikely(!wait_bounded(&empty[st], (j / S8 - 1) & 1, abort_flag))) break;
        const int q = lane - (j % TPB) * GR;  // this lane's group of the tile
        const bool mine = q >= 0 && q < GR;
        const int key0 = (p0 + j) * NK, valid = min(NK, L - key0);
        // bytes first: the scales, which may still be on their way, are written
        // before the tile's conversion can begin (the barrier's second arrival)
        if (lane == 0)
          mbar_arrive_expect_tx(&full[st], (valid + a.page_box - 1) / a.page_box * a.page_box * DH);
        __syncwarp();
        if (mine && q * 16 < valid && ((q * 16) & (a.page_box - 1)) == 0)
          tma_load_3d(s8 + (st * 2 + kv) * Sh::kByteTile + q * 16 * DH, map, 0, (key0 + q * 16) & (a.page_size - 1),
                      page * a.Hkv + g, &full[st]);
        __syncwarp();
        issued = j + 1;
        if (mine && kv == 0) {
          const int ve = scale_exponent(vs);
          scales[((pfx0 + j) % Sh::kScaleSlots) * GR + q] =
              make_uint2(pack_scales(exponent_scale(scale_exponent(ks)), exponent_scale(-ve)), __float_as_uint(static_cast<float>(ve)));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
      }
    } else if (warp == kMmaWarp && elect_one()) {
      // ------------------------------------------------------------------- MMA
      // Per tile j: S of tile j+1 for every M-tile as soon as its softmax has
      // taken S(j), then P(j).V for every M-tile once P(j) is in tensor memory.
      // The converters wrote the tiles through the generic proxy: the fence
      // after each wait orders them before the MMAs.
      constexpr uint32_t id_s = idesc_f16(128, NK, false);
      constexpr uint32_t id_o = idesc_f16(128, DH, true);
      // Low words of the descriptors (address / 16 below 2^14, leading offset
      // above); the high words are one constant.  Each tile starts from a base
      // that the compiler takes as new: it would otherwise keep the two dozen
      // descriptors of a tile, and with this warp's share of registers spill them.
      const uint32_t q_lo = static_cast<uint32_t>(sdesc_sw128(smem_u32(sQ), 16, 1024));
      const uint32_t k_lo = static_cast<uint32_t>(sdesc_sw128(smem_u32(sK), 16, 1024));
      const uint32_t v_lo = static_cast<uint32_t>(sdesc_sw128(smem_u32(sV), NK * 128, 1024));
      auto issue_s = [&](int j, int t) {
        const uint32_t kd = anew(k_lo + (j % SF) * (Sh::kTileBytes >> 4));
        const uint32_t qd = anew(q_lo + t * Sh::kRegions * (Sh::kQRegionBytes >> 4));
#pragma unroll
        for (int s = 0; s < DH / 16; ++s)
          mma_f16_ss(tmem + Sh::kColS + t * NK, qd + (((s / 4) * Sh::kQRegionBytes + (s % 4) * 32) >> 4),
                     kd + (((s / 4) * (NK * 128) + (s % 4) * 32) >> 4), id_s, s > 0);
        mma_commit(&s_full[t]);
      };
      bool ok = T == 0 || (wait_bounded(q_full, 0, abort_flag) && wait_bounded(&tile_full[0], 0, abort_flag));
      if (ok && T > 0) {
        fence_async_smem();
        tc_fence_after();
        for (int t = 0; t < MT; ++t) issue_s(0, t);
        mma_commit(&tile_empty[0]);
      }
      for (int j = 0; j < T && ok; ++j) {
        const int st = j % SF;
        const bool next = j + 1 < T;
        if (next) {
          if (!wait_bounded(&tile_full[(j + 1) % SF], ((j + 1) / SF) & 1, abort_flag)) break;
          fence_async_smem();
          for (int t = 0; t < MT && ok; ++t) {
            if (!wait_bounded(&s_free[t], j & 1, abort_flag)) { ok = false; break; }
            tc_fence_after();
            issue_s(j + 1, t);
          }
          if (!ok) break;
          mma_commit(&tile_empty[(j + 1) % SF]);
        }
        if (!wait_bounded(&tile_full[SF + st], (j / SF) & 1, abort_flag)) break;
        fence_async_smem();
        const uint32_t vd = v_lo + st * (Sh::kTileBytes >> 4);
        for (int t = 0; t < MT && ok; ++t) {
          if (!wait_bounded(&p_full[t], j & 1, abort_flag)) { ok = false; break; }
          tc_fence_after();
          const uint32_t pcol = anew(tmem + Sh::kColP + t * (NK / 2)), vt = anew(vd);
#pragma unroll
          for (int s = 0; s < NK / 16; ++s)
            mma_f16_ts(tmem + Sh::kColO + t * DH, pcol + s * 8, vt + s * (2048 >> 4), id_o, (j > 0 || s > 0));
          mma_commit(&o_done[t]);
        }
        if (ok) mma_commit(&tile_empty[SF + st]);
      }
    }
  } else if (warp >= kConvertWarp) {
    // ------------------------------------------------------------- converters
    // Each warp takes whole groups of 16 keys.  In a step the eight lanes of a
    // quarter warp hold two rows' 16-byte pieces so chosen that both their loads
    // (rows of DH bytes) and their two stores (swizzled rows of 128 bytes) touch
    // every bank once: with DH = 128, columns 0-63 of one row and 64-127 of the
    // other, the next quarter the complement.
    regs_dec<Sh::kRegsConvert>();
    const int cw = warp & 3, quarter = lane >> 3, l8 = lane & 7;
    constexpr int STEPS = DH / 32;          // steps of 16 rows: 32 pieces each
    const int cc = DH == 128 ? l8 : l8 & 3;  // this lane's piece of the row
    const auto row_of = [&](int step) {
      return DH == 128 ? 4 * step + 2 * (quarter >> 1) + ((l8 >> 2) ^ (quarter & 1)) : 8 * step + 2 * quarter + (l8 >> 2);
    };
    const auto store = [&](unsigned char *tile, int r, const uint32_t (&h)[8]) {
      unsigned char *region = tile + (cc >> 2) * (NK * 128);
      *reinterpret_cast<uint4 *>(region + sw128_offset(r, 2 * (cc & 3))) = make_uint4(h[0], h[1], h[2], h[3]);
      *reinterpret_cast<uint4 *>(region + sw128_offset(r, 2 * (cc & 3) + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
    };
    const int kv0 = Sh::kConvertGroups == 2 ? (warp - kConvertWarp) >> 2 : 0;
    for (int jj = 0; jj < T * (3 - Sh::kConvertGroups); ++jj) {
      const int j = Sh::kConvertGroups == 2 ? jj : jj >> 1, kv = Sh::kConvertGroups == 2 ? kv0 : jj & 1;
      unsigned char *tiles = kv ? sV : sK;
      uint64_t *full = tile_full + kv * SF, *empty = tile_empty + kv * SF;
      const int st = j % SF, jp = j - pfx0;
      const bool prefix = jp >= 0 && jp < np;
      if (prefix && unlikely(!wait_bounded(&bytes_full[kv * S8 + jp % S8], (jp / S8) & 1, abort_flag))) break;
      if (j >= SF && unlikely(!wait_bounded(&empty[st], (j / SF - 1) & 1, abort_flag))) break;
      unsigned char *tile = tiles + st * Sh::kTileBytes;
      const int key0 = (prefix ? p0 + jp : j - tree0) * NK;
      const int valid = min(NK, (prefix ? L : n) - key0);
      if (__builtin_expect(prefix, 1)) {
        for (int grp = cw; grp < GR; grp += 4) {
          const unsigned char *src = s8 + ((jp % S8) * 2 + kv) * Sh::kByteTile;
          uint4 x[STEPS];
#pragma unroll
          for (int s = 0; s < STEPS; ++s) {
            const int r = grp * 16 + row_of(s);
            x[s] = *reinterpret_cast<const uint4 *>(src + r * DH + cc * 16);
            if (r >= valid) x[s] = make_uint4(0, 0, 0, 0);  // past the prefix: whatever the page holds
          }
#pragma unroll
          for (int s = 0; s < STEPS; ++s) {
            const uint32_t w[4] = {x[s].x, x[s].y, x[s].z, x[s].w};
            uint32_t h[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              h[2 * i] = e4m3_to_half2(w[i] & 0xffffu);
              h[2 * i + 1] = e4m3_to_half2(w[i] >> 16);
            }
            store(tile, grp * 16 + row_of(s), h);
          }
        }
      } else {
        // tree nodes: bf16 over a power of two, the group's or (ONE) the tile's;
        // all of a warp's groups are then loaded at once and their largest
        // magnitude is exchanged with the other warps'.  Nodes that no query row
        // of this CTA names are zeros, so that what they hold decides nothing.
        constexpr int GW = ONE ? GR / 4 : 1;
        const __nv_bfloat16 *src = (kv ? a.v_tree : a.k_tree) + (static_cast<int64_t>(bg) * n + key0) * DH;
        bool gave_up = false;
        for (int g0 = cw; g0 < GR; g0 += 4 * GW) {
          uint4 x[GW][STEPS], y[GW][STEPS];
          float amax = 0.f;
          uint32_t live = 0;  // bit 16 w + c: node c of the warp's group w
#pragma unroll
          for (int w = 0; w < GW; ++w) live |= static_cast<uint32_t>(named[(key0 >> 4) + g0 + 4 * w]) << (16 * w);
#pragma unroll
          for (int w = 0; w < GW; ++w)
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
              const int r = (g0 + 4 * w) * 16 + row_of(s);
              x[w][s] = y[w][s] = make_uint4(0, 0, 0, 0);
              if (r < valid && ((live >> (16 * w + row_of(s))) & 1u)) {
                const uint4 *p = reinterpret_cast<const uint4 *>(src + static_cast<int64_t>(r) * DH + cc * 16);
                x[w][s] = p[0];
                y[w][s] = p[1];
              }
            }
#pragma unroll
          for (int w = 0; w < GW; ++w)
#pragma unroll
            for (int s = 0; s < STEPS; ++s) amax = fmaxf(amax, fmaxf(amax8(x[w][s]), amax8(y[w][s])));
          amax = warp_max(amax);
          if constexpr (ONE) {
            // a slot is written again only after the other ring's exchange
            if (lane == 0) {
              tree_max[4 * kv + cw] = amax;
              mbar_arrive(&tree_sync[kv]);
            }
            __syncwarp();
            if (unlikely(!wait_bounded(&tree_sync[kv], (j - tree0) & 1, abort_flag))) { gave_up = true; break; }
#pragma unroll
            for (int w = 0; w < 4; ++w) amax = fmaxf(amax, tree_max[4 * kv + w]);
          }
          const int e = half_exponent(amax);
          const float f = pow2_clamped(-e);
#pragma unroll
          for (int w = 0; w < GW; ++w)
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
              const uint32_t h[8] = {bf16x2_to_half2(x[w][s].x, f), bf16x2_to_half2(x[w][s].y, f), bf16x2_to_half2(x[w][s].z, f),
                                     bf16x2_to_half2(x[w][s].w, f), bf16x2_to_half2(y[w][s].x, f), bf16x2_to_half2(y[w][s].y, f),
                                     bf16x2_to_half2(y[w][s].z, f), bf16x2_to_half2(y[w][s].w, f)};
              store(tile, (g0 + 4 * w) * 16 + row_of(s), h);
            }
          if (lane == 0) {
            uint2 *sc = scales + (j % Sh::kScaleSlots) * GR + g0;
            const uint32_t both = pack_scales(pow2_clamped(e), pow2_clamped(-e));
            reinterpret_cast<unsigned short *>(&sc->x)[kv ? 0 : 1] = static_cast<unsigned short>(kv ? both : both >> 16);
            if (kv) sc->y = __float_as_uint(static_cast<float>(e));
          }
        }
        if (unlikely(gave_up)) break;
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&full[st]);
        if (prefix) mbar_arrive(&bytes_empty[kv * S8 + jp % S8]);
      }
      __syncwarp();
    }
  } else {
    // ----------------------------------------------------------------- softmax
    regs_inc<Sh::kRegsSoftmax>();
    const int t = warp >> 2, qtr = warp & 3;
    // this M-tile's query rows to shared memory as f16, each over a power of
    // two of its own: 8 or 16 neighbouring lanes hold a row
    constexpr int CPR = DH / 8, kPieces = QR * CPR / 128, kAhead = 8;  // a thread's; requested together
    static_assert(kPieces % kAhead == 0 || kPieces < kAhead, "whole batches");
#pragma unroll 1
    for (int p0q = 0; p0q < kPieces; p0q += kAhead) {
      uint4 v[kAhead < kPieces ? kAhead : kPieces];
      constexpr int kBatch = kAhead < kPieces ? kAhead : kPieces;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int idx = (tid & 127) + (p0q + u) * 128, r = idx / CPR, c = idx % CPR;
        const int rho = (mg * MT + t) * 128 + r;
        v[u] = make_uint4(0, 0, 0, 0);
        if (rho < rows_total)
          v[u] = *reinterpret_cast<const uint4 *>(
              a.q + ((static_cast<int64_t>(b) * n + rho / a.G) * a.Hq + g * a.G + rho % a.G) * DH + c * 8);
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int idx = (tid & 127) + (p0q + u) * 128, r = idx / CPR, c = idx % CPR;
        float amax = amax8(v[u]);
#pragma unroll
        for (int o = 1; o < CPR; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const int e = half_exponent(amax);
        const float f = pow2_clamped(-e);
        *reinterpret_cast<uint4 *>(sQ + (t * Sh::kRegions + c / 8) * Sh::kQRegionBytes + sw128_offset(r, c % 8)) =
            make_uint4(bf16x2_to_half2(v[u].x, f), bf16x2_to_half2(v[u].y, f), bf16x2_to_half2(v[u].z, f), bf16x2_to_half2(v[u].w, f));
        if (c == 0) q_exp[t * QR + r] = static_cast<signed char>(e);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(q_full);
    asm volatile("bar.sync %0, 128;" ::"r"(t + 1) : "memory");  // the M-tile's exponents are written

    const int r = qtr * 32 + lane;
    const int rho = (mg * MT + t) * 128 + r;
    const bool row_ok = rho < rows_total;
    const bool warp_live = (mg * MT + t) * 128 + qtr * 32 < rows_total;  // warp-uniform
    const int i = row_ok ? rho / a.G : 0;
    const int hh = row_ok ? rho % a.G : 0;
    const float row_scale = a.scale_log2 * (row_ok ? pow2_clamped(q_exp[t * QR + r]) : 1.f);
    const uint32_t lane_base = static_cast<uint32_t>(qtr * 32) << 16;
    const uint32_t tS = tmem + lane_base + Sh::kColS + t * NK;
    const uint32_t tP = tmem + lane_base + Sh::kColP + t * (NK / 2);
    const uint32_t tO = tmem + lane_base + Sh::kColO + t * DH;
    const uint64_t *mrow = a.mask + (static_cast<int64_t>(b) * n + i) * a.W;
    // SEL: this row's bits, and the word of them at hand
    const uint32_t *bit_row = nullptr;
    int bit_at = -1;
    uint32_t bit_word = 0;
    if constexpr (SEL)
      bit_row = a.bits + ((static_cast<int64_t>(bg) * mgroups + mg) * a.group_nodes + (row_ok ? i - mg * MT * 128 / a.G : 0)) * a.bit_words;
    // m is the exponent base of this row's P' and O; it is raised only when the
    // row maximum exceeds it by more than 8, so O is rescaled rarely.
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < T; ++j) {
      uint32_t taken = 0xffffffffu;  // SEL: bit k: the row counts the tile's page k
      if constexpr (SEL) {
        if (j >= pfx0 && j - pfx0 < np) {
          const int first = ((p0 + j - pfx0) * NK) >> a.log_page;
          if (first >> 5 != bit_at) bit_word = bit_row[bit_at = first >> 5];
          taken = bit_word >> (first & 31);  // a tile's pages are in one word
        }
      }
      if (unlikely(!wait_bounded(&s_full[t], j & 1, abort_flag))) { ok = false; break; }
      tc_fence_after();
      const int jp = j - pfx0;
      const bool prefix = jp >= 0 && jp < np;
      // a tree tile's ve is its V converters' (the prefix's scales came with K)
      if (unlikely(!prefix) && unlikely(!wait_bounded(&tile_full[SF + j % SF], (j / SF) & 1, abort_flag))) { ok = false; break; }
      const uint2 *sc = scales + (j % Sh::kScaleSlots) * GR;
      const bool dense = prefix && (p0 + jp + 1) * NK <= L;  // no key of the tile is masked
      // never 0, since it multiplies the -inf of masked keys, nor infinite: a dot
      // product of finite numbers may be 0
      const auto group = [&](int q) {  // (factor, ve)
        const uint2 gs = sc[q];
        float2 fv = make_float2(fminf(fmaxf(row_scale * __uint_as_float(gs.x & 0xffff0000u), 1.2e-38f), 1e38f), __uint_as_float(gs.y));
        if constexpr (SEL)  // a page that the row does not count: weights of 2^-inf
          if (!((taken >> (q >> min(a.log_page - 4, 5))) & 1u)) fv.y = -INFINITY;
        return fv;
      };
      // Four groups' are kept for both passes; eight are read again (measured:
      // 70B 154 -> 152 us with four kept, GPT-OSS 734 -> 757 with eight).
      float2 held[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) held[q] = ONE || NH == 1 ? group(ONE ? 0 : q) : make_float2(0.f, 0.f);
      // S in halves of 64 columns.  With two halves the first is read once for
      // the maximum and again for its exponentials, after the second's: 64
      // scores in registers at a time instead of 128.
      float sv[2][32];
      const auto mask_half = [&](int h) {
        uint64_t keep;
        if (prefix) {
          const int valid = min(NK, L - (p0 + jp) * NK) - 64 * h;
          keep = valid >= 64 ? ~0ull : (valid <= 0 ? 0ull : ((1ull << valid) - 1ull));
        } else {  // bits past the last node count for nothing
          const int w = (j - tree0) * NH + h;
          keep = (row_ok && w < a.W) ? mrow[w] & (~0ull >> max(0, 64 * (w + 1) - n)) : 0ull;
        }
#pragma unroll
        for (int c = 0; c < 64; ++c) sv[c / 32][c % 32] = ((keep >> c) & 1ull) ? sv[c / 32][c % 32] : -INFINITY;
      };
      const auto half_max = [&](int h) {
        float x = -INFINITY;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float *s16 = sv[q / 2] + 16 * (q % 2);
          float y = s16[0];
#pragma unroll
          for (int c = 1; c < 15; c += 2) y = fmax3(y, s16[c], s16[c + 1]);
          if constexpr (ONE) {
            x = fmax3(x, y, s16[15]);
            if (q == 3) x = fmaf(x, held[0].x, held[0].y);
            continue;
          }
          const float2 fv = NH == 1 ? held[q] : group(4 * h + q);
          x = fmaxf(x, fmaf(fmaxf(y, s16[15]), fv.x, fv.y));
        }
        return x;
      };
      const auto release = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[t]);  // S has been read
        __syncwarp();  // or lane 0 would work on apart from the others
      };
      // SEL: a warp none of whose rows counts a page of the tile has weights of zero
      bool busy = warp_live;
      if constexpr (SEL) {
        const int pages = NK >> a.log_page;  // of a tile; 0: a page is longer
        busy = warp_live && __any_sync(0xffffffffu, row_ok && (taken & ((2u << max(pages - 1, 0)) - 1u)));
      }
      float tmax = -INFINITY;
      if (NH == 2 && busy) {
        tmem_ld32x2(tS, sv[0], sv[1]);
        if (unlikely(!dense)) mask_half(0);
        tmax = half_max(0);
      }
      if (busy) tmem_ld32x2(tS + 64 * (NH - 1), sv[0], sv[1]);
      if (NH == 1) release();
      if (busy) {
        if (unlikely(!dense)) mask_half(NH - 1);
        tmax = fmaxf(tmax, half_max(NH - 1));
      }
      const bool raise = tmax > m + 8.f;
      const float base = raise ? tmax : m;
      const float alpha = raise ? ex2_approx(m - tmax) : 1.f;  // m = -inf gives 0
      m = base;
      if (j > 0) {  // P.V of the previous tile is done: P is free, O is final for it
        if (unlikely(!wait_bounded(&o_done[t], (j - 1) & 1, abort_flag))) { ok = false; break; }
        tc_fence_after();
      }
      const float nb = kBias - (base > -INFINITY ? base : 0.f);
      float sum = 0.f;
      const auto exp_half = [&](int h) {
        uint64_t one_acc[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float pk[16];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int gi = 4 * h + 2 * half + q;
            const float2 fv = ONE ? held[0] : (NH == 1 ? held[2 * half + q] : group(gi));
            const float f = fv.x, off = nb + fv.y;
            const uint64_t f2 = f2_pack(f, f), o2 = f2_pack(off, off);
            uint64_t acc = ONE ? one_acc[q] : f2_pack(0.f, 0.f);
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              float t0, t1;
              f2_unpack(f2_fma(f2_pack(sv[half][16 * q + 2 * c], sv[half][16 * q + 2 * c + 1]), f2, o2), t0, t1);
              const float e0 = ex2_approx(t0), e1 = ex2_approx(t1);
              acc = f2_add(acc, f2_pack(e0, e1));
              const __half2 h2 = __floats2half2_rn(e0, e1);
              pk[8 * q + c] = *reinterpret_cast<const float *>(&h2);
            }
            if constexpr (ONE) {
              one_acc[q] = acc;
            } else {
              float a0, a1;
              f2_unpack(acc, a0, a1);
              sum = fmaf(a0 + a1, __uint_as_float(sc[gi].x << 16), sum);
            }
          }
          tmem_st16_async(tP + 32 * h + 16 * half, pk);
        }
        if constexpr (ONE) {
          float a0, a1;
          f2_unpack(f2_add(one_acc[0], one_acc[1]), a0, a1);
          sum = fmaf(a0 + a1, __uint_as_float(sc[0].x << 16), sum);
        }
      };
      if (busy) exp_half(NH - 1);
      if constexpr (SEL) {
        if (warp_live && !busy) {
          float zeros[16];
#pragma unroll
          for (int c = 0; c < 16; ++c) zeros[c] = 0.f;
#pragma unroll
          for (int c = 0; c < NK / 2; c += 16) tmem_st16_async(tP + c, zeros);
        }
      }
      if constexpr (NH == 2) {
        if (busy) tmem_ld32x2(tS, sv[0], sv[1]);
        release();
        if (busy) {
          if (unlikely(!dense)) mask_half(0);
          exp_half(0);
        }
      }
      if (warp_live) tmem_wait_st();
      l = fmaf(l, alpha, sum);
      if (unlikely(warp_live && j > 0 && __any_sync(0xffffffffu, raise))) {
#pragma unroll 1
        for (int c0 = 0; c0 < DH; c0 += 32) {
          float o[32];
          tmem_ld32(tO + c0, o);
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] *= alpha;
          tmem_st32(tO + c0, o);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[t]);
      __syncwarp();
    }
    if (ok && T > 0 && unlikely(!wait_bounded(&o_done[t], (T - 1) & 1, abort_flag))) ok = false;
    tc_fence_after();
    // tcgen05.ld is warp-collective: every lane executes it, rows past the last
    // node only skip the global writes
    const int h = g * a.G + hh;
    const int64_t orow = (static_cast<int64_t>(b) * n + i) * a.Hq + h;
    const bool have = ok && T > 0;
    if constexpr (SPLIT) {
      part_have = have;
      part_m = m;
      part_l = l;
    } else {
      const float inv = (have && l != 0.f) ? 1.f / l : 0.f;  // a NaN stays one
#pragma unroll
      for (int c0 = 0; c0 < DH; c0 += 32) {
        float o[32];
        if (have) {
          tmem_ld32(tO + c0, o);
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = 0.f;
        }
        if (!row_ok) continue;
        __nv_bfloat162 hv[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) hv[e] = __floats2bfloat162_rn(o[2 * e] * inv, o[2 * e + 1] * inv);
        uint4 *dst = reinterpret_cast<uint4 *>(a.out + orow * DH + c0);
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[e] = reinterpret_cast<const uint4 *>(hv)[e];
      }
      if (row_ok && a.lse) a.lse[orow] = (have && l != 0.f) ? (m - kBias + log2f(l)) * kLn2 : -INFINITY;
    }
  }

  pdl_trigger();
  // ---- teardown --------------------------------------------------------------
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // Equal shares again, only now that every warp has left its role: a warp that
  // took its registers back earlier would take them from the softmax warps'
  // share, which would then wait for ever.
  if (warp < kConvertWarp) regs_dec<Sh::kLaunchRegs>();
  else regs_inc<Sh::kLaunchRegs>();
  if (*abort_flag) {
    if (tid == 0) report(a.status, EAGLE_ERR_TIMEOUT);
    volatile int never = 0;
    if (warp == kMmaWarp) {
      __syncwarp();
      if (elect_one()) {  // the thread that issued the MMAs (the election is the same each time): a commit covers its own
        mma_commit(teardown);  // every MMA issued so far completes before tensor memory is released
        mbar_wait(teardown, 0, &never, 100000000ull);
      }
    }
    if (warp >= kProducerWarp && warp < kMmaWarp && lane == 0) {
      // copies still in flight complete before shared memory is released
      const uint64_t *full = bytes_full + (warp - kProducerWarp) * S8;
      for (int j = max(0, issued - S8); j < issued; ++j)
        mbar_wait(const_cast<uint64_t *>(&full[j % S8]), (j / S8) & 1, &never, 100000000ull);
    }
    __syncthreads();
  }
  const int r0 = mg * MT * 128, nr = max(0, min(rows_total, r0 + MT * 128) - r0);
  if constexpr (SPLIT) {
    if (warp < MT * 4) {
      // this CTA's O rows (fp32) into the f16 stages and its (m, l) pairs into
      // the Q buffer: every MMA and copy has completed.  Row r's 16-byte chunk c
      // sits at chunk c ^ (r & 7), so a warp's rows store to distinct banks.
      const int t = warp >> 2, qtr = warp & 3, rl = t * 128 + qtr * 32 + lane;
      const uint32_t tO = tmem + (static_cast<uint32_t>(qtr * 32) << 16) + Sh::kColO + t * DH;
      const bool have = part_have && !*abort_flag;
      float4 *prow = reinterpret_cast<float4 *>(sK) + rl * (DH / 4);
#pragma unroll
      for (int c0 = 0; c0 < DH; c0 += 32) {
        float o[32];
        if (__all_sync(0xffffffffu, have)) {
          tmem_ld32(tO + c0, o);
        } else {
#pragma unroll
          for (int c = 0; c < 32; ++c) o[c] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          prow[(c0 / 4 + e) ^ (rl & 7)] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
      }
      reinterpret_cast<float2 *>(sQ)[rl] = have ? make_float2(part_m, part_l) : make_float2(-INFINITY, 0.f);
    }
    tc_fence_before();
    __syncthreads();
    constexpr int NV = DH / 4;
    const int64_t cl = static_cast<int64_t>(bg) * mgroups + mg;
    float *slot = a.part + (cl * a.S + split) * static_cast<int64_t>(a.slot_rows) * (DH + 2);
    for (int idx = tid; idx < nr * NV; idx += Sh::kThreads) {
      const int r = idx / NV, c = idx % NV;
      reinterpret_cast<float4 *>(slot)[idx] = reinterpret_cast<const float4 *>(sK)[r * NV + (c ^ (r & 7))];
    }
    for (int r = tid; r < nr; r += Sh::kThreads)
      reinterpret_cast<float2 *>(slot + static_cast<int64_t>(a.slot_rows) * DH)[r] = reinterpret_cast<const float2 *>(sQ)[r];
  }
  if (warp == kMmaWarp) tmem_dealloc(tmem, Sh::kTmemCols);

  // ---- split merge across the cluster: CTA `rank` merges its share of the rows
  // from all S slots, read from L2
  if constexpr (MERGE == 1) {
    cluster_arrive_release();
    cluster_wait();
    if (*abort_flag) return;
    const int per = (nr + a.S - 1) / a.S;
    const int q0 = min(nr, static_cast<int>(cluster_ctarank()) * per), q1 = min(nr, q0 + per);
    for (int item = tid; item < (q1 - q0) * (DH / 4); item += Sh::kThreads)
      kv8_merge_item<DH>(a, bg, mg, mgroups, MT, q0 + item / (DH / 4), item % (DH / 4));
  }
}

// ---- host side ---------------------------------------------------------------

struct Kv8Plan {
  int MT, NK, QR, mgroups, S, ctas_per_sm;
  bool one_wave;
};

// M-tiles per CTA, key-tile width, and the KV split S that minimises (waves of
// CTAs) x (key tiles per CTA + what a CTA costs before its first and after its
// last tile, about six tiles, + the merge of partial results).  From three
// waves on the last one is hardly seen, ragged lengths spread it.
inline Kv8Plan kv8_plan(int B, int n, int Hq, int Hkv, int dh, int Lmax, int num_sms) {
  Kv8Plan p;
  const int G = Hq / Hkv, rows = n * G, tiles = (rows + 127) / 128;
  p.MT = tiles <= 1 ? 1 : 2;
  p.QR = rows <= 64 ? 64 : 128;
  p.NK = dh == 64 && p.MT == 2 ? 128 : 64;
  p.mgroups = (tiles + p.MT - 1) / p.MT;
  p.ctas_per_sm = p.MT == 1 && (dh == 64 || p.QR == 64) ? 2 : 1;
  const int64_t base = static_cast<int64_t>(B) * Hkv * p.mgroups;
  const int64_t slots = static_cast<int64_t>(num_sms) * p.ctas_per_sm;
  const int64_t ptiles = (static_cast<int64_t>(Lmax) + p.NK - 1) / p.NK;
  const double split_cost = static_cast<double>(rows) * 64.0 / p.NK / 32.0 / p.mgroups;
  p.S = 1;
  double best = 1e30;
  for (int S = 1; S <= kMaxClusterSplits8 && S <= ptiles; ++S) {
    const double load = static_cast<double>(base * S) / slots;
    const double waves = load < 3.0 ? static_cast<double>((base * S + slots - 1) / slots) : load + 0.5;
    const double cost = waves * (static_cast<double>((ptiles + S - 1) / S) + 6.0 + (S > 1 ? split_cost : 0.0));
    if (cost < best * 0.97) {  // prefer fewer splits unless clearly better
      best = cost;
      p.S = S;
    }
  }
  // A cluster merges its splits where two CTAs share an SM; clusters of CTAs that
  // fill an SM each find too few neighbours free (392 rows, dh 128, 8 heads of
  // 4096 keys: 59 us with clusters of eight, 35 with the merge kernel).
  p.one_wave = p.ctas_per_sm == 2 && base * p.S <= slots;
  return p;
}

// Rows of a split's workspace slot, rounded up to 8.
inline int kv8_slot_rows(const Kv8Plan &p, int rows) { return min((rows + 7) / 8 * 8, p.MT * 128); }

template <int DH, int MT, int NK, int SF, int S8, int QR, int OCC, bool ONE, int MERGE, bool SEL>
static cudaError_t launch_kv8_v(const CUtensorMap *maps, const typename Kv8KernelArgs<SEL>::type &a, const Kv8Plan &p, cudaStream_t st) {
  using Sh = Kv8Shape<DH, MT, NK, SF, S8, QR, OCC, ONE>;
  const auto kernel = tree_attn_kv8_kernel<DH, MT, NK, SF, S8, QR, OCC, ONE, MERGE, SEL>;
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = set_smem_limit_once(kernel, Sh::kSmem, configured);
  if (e != cudaSuccess) return e;
  // the warpgroups' shares add up only if a thread is launched with these
  static std::atomic<int> regs{0};
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, kernel);
    if (e != cudaSuccess) return e;
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) != Sh::kLaunchRegs) return cudaErrorInvalidConfiguration;
  const dim3 grid(p.S, SEL ? a.B * a.Hkv : p.mgroups, SEL ? p.mgroups : a.B * a.Hkv);
  if constexpr (MERGE == 2) {
    e = launch_chained(kernel, grid, dim3(Sh::kThreads), Sh::kSmem, st, maps[0], maps[1], a);
    if (e != cudaSuccess) return e;
    const dim3 mgrid((a.slot_rows * (DH / 4) + 255) / 256, p.mgroups, a.B * a.Hkv);
    return launch_chained(tree_attn_kv8_merge_kernel<DH>, mgrid, dim3(256), 0, st, static_cast<const Kv8Args &>(a), MT);
  }
  return launch_chained_cluster(kernel, grid, dim3(Sh::kThreads), Sh::kSmem, st, p.S, maps[0], maps[1], a);
}

template <bool SEL, int DH, int MT, int NK, int SF, int S8, int QR, int OCC, bool ONE>
static cudaError_t launch_kv8_t(const CUtensorMap *maps, const typename Kv8KernelArgs<SEL>::type &a, const Kv8Plan &p, cudaStream_t st) {
  if (p.S <= 1) return launch_kv8_v<DH, MT, NK, SF, S8, QR, OCC, ONE, 0, SEL>(maps, a, p, st);
  return p.one_wave ? launch_kv8_v<DH, MT, NK, SF, S8, QR, OCC, ONE, 1, SEL>(maps, a, p, st)
                    : launch_kv8_v<DH, MT, NK, SF, S8, QR, OCC, ONE, 2, SEL>(maps, a, p, st);
}

// The instance for a shape, with the plan's numbers.
template <bool SEL>
static cudaError_t launch_kv8(typename Kv8KernelArgs<SEL>::type a, const void *k_pages, const void *v_pages, int dh, const Kv8Plan &p,
                              void *part, cudaStream_t st) {
  if (p.S > 1 && !part) return cudaErrorInvalidValue;
  a.S = p.S;
  a.page_box = min(a.page_size, p.NK);
  a.part = p.S > 1 ? reinterpret_cast<float *>(part) : nullptr;
  a.slot_rows = kv8_slot_rows(p, a.n * a.G);
  CUtensorMap maps[2];
  const int64_t blocks = static_cast<int64_t>(a.num_pages) * a.Hkv;
  if (!make_pool_map(&maps[0], k_pages, blocks, a.page_size, dh, a.page_box, false) ||
      !make_pool_map(&maps[1], v_pages, blocks, a.page_size, dh, a.page_box, false))
    return cudaErrorInvalidValue;
  const bool one = a.page_size >= p.NK;
  if (dh == 64) {
    if (p.MT == 2)
      return one ? launch_kv8_t<SEL, 64, 2, 128, 2, 4, 128, 1, true>(maps, a, p, st) : launch_kv8_t<SEL, 64, 2, 128, 2, 4, 128, 1, false>(maps, a, p, st);
    return launch_kv8_t<SEL, 64, 1, 64, 3, 4, 128, 2, false>(maps, a, p, st);
  }
  if (p.MT == 2)
    return one ? launch_kv8_t<SEL, 128, 2, 64, 2, 5, 128, 1, true>(maps, a, p, st) : launch_kv8_t<SEL, 128, 2, 64, 2, 5, 128, 1, false>(maps, a, p, st);
  return p.QR == 64 ? launch_kv8_t<SEL, 128, 1, 64, 2, 2, 64, 2, false>(maps, a, p, st) : launch_kv8_t<SEL, 128, 1, 64, 3, 4, 128, 1, false>(maps, a, p, st);
}

}  // namespace eagle
