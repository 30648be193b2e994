// Attention over the 8-bit paged cache for few query rows a KV head (single
// tokens, small trees; rows are (node, grouped head) pairs): the mathematics of
// tree_attn_kv8.cu on warp-level f16 MMAs (m16n8k16), which take 16 rows.
//
// What bounds it: HBM for a batch of single tokens, latency for one sequence.
// With a row or two to a key, tcgen05's 128-row tiles and their hand-overs
// between warps (bytes, converters, MMA, softmax, MMA) cost more than the
// arithmetic; here a warp does all of it in registers, and only bytes pass
// through shared memory:
//   * the bytes of 16 keys (one group, one page) come by two TMA boxes into the
//     warp's ring; a lane's 16-byte pieces of K are B fragments once converted,
//     word by word, because the order of the head's columns in the dot product
//     is free: lane t of a quad takes columns 32t..32t+31 (16t..16t+15 for 64);
//   * V's fragments pair two keys of one column: a byte permute of two rows' words
//     and the same conversion; the order of output columns is free too;
//   * P stays in the accumulators' layout, which is the A operand's;
//   * the running maximum is looked at across a quad only when a lane's own
//     exceeds it by more than 2^8.
// Measured: 64 single tokens, 64 heads on 8, dh 128, 1024 to 8192 keys: 122 us
// (607 MB, 5.0 TB/s, 74 % of a copy's rate; 84 % at 8192 keys each, 93 % at
// 16384), against 237 us for the 16-bit cache; what is lost is each CTA's chain
// length - page number - bytes, and the last CTAs of the grid.
// A CTA of four warps is KG = 4 / RG groups of keys times RG = 1 or 2 tiles of 16
// rows; the RG warps of a key group share its ring.  Three CTAs an SM keep up
// to 192 KB of requests in flight.
#include "kv8_attn.cuh"

namespace eagle {

using namespace sm100;

constexpr int kRingBytes = 65536;
constexpr int kMaxSplitsFew = 32;

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 lds16(const unsigned char *p) { return *reinterpret_cast<const uint4 *>(p); }
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// Where 16-byte chunk c of the fp32 O row r of a warp's tile lies, so that the
// eight lanes of a store touch every bank once.
template <int DH>
__device__ __forceinline__ int o_chunk(int r, int c) {
  const int key = DH == 128 ? ((c >> 3) | ((r & 1) << 2)) : ((c >> 3) | ((r & 1) << 1));
  return r * (DH / 4) + (c ^ key);
}

template <bool SEL> struct FewArgs { using type = Kv8Args; };
template <> struct FewArgs<true> { using type = Kv8SelArgs; };

// SEL: a "sequence" is one node of a sequence, with the pages that its row of `sel`
// lists for the KV head in place of the whole prefix, and the nodes of its mask row;
// its rows are the head's grouped queries alone.
template <int DH, int RG, int MERGE, bool SEL>
__global__ void __launch_bounds__(128, 3)
    tree_attn_kv8_few_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map,
                             typename FewArgs<SEL>::type a) {
  constexpr int KG = 4 / RG;
  constexpr int STAGE = 32 * DH;                    // 16 keys' K, then V
  constexpr int DEPTH = kRingBytes / KG / STAGE;
  constexpr int STEPS = DH / 16, NT = DH / 8;       // k steps of Q K^T, column tiles of P V
  constexpr int KW = DH / 16, VW = DH / 32;         // words of a K row, of a V row a lane holds
  extern __shared__ __align__(1024) unsigned char few_smem[];
  unsigned char *ring0 = few_smem + ((1024 - (smem_u32(few_smem) & 1023)) & 1023);
  __shared__ uint64_t full[KG * DEPTH], empty[KG * DEPTH];
  __shared__ float2 s_ml[4 * 16];
  __shared__ int s_abort;
  volatile int *abort_flag = &s_abort;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gr = lane >> 2, t = lane & 3;
  const int kg = warp / RG, rg = warp % RG;
  const int split = SEL ? blockIdx.x % a.S : blockIdx.x, bg = SEL ? blockIdx.x / a.S : blockIdx.z;
  const int b = bg / a.Hkv, g = bg % a.Hkv;
  int seq = b, nodes = a.n;  // whose cache and tree, its nodes
  const int32_t *list = nullptr;
  if constexpr (SEL) {
    seq = b / a.nodes;
    nodes = a.nodes;
    list = a.sel + static_cast<int64_t>(bg) * a.top;
  }
  unsigned char *ring = ring0 + kg * DEPTH * STAGE;
  uint64_t *kfull = full + kg * DEPTH, *kempty = empty + kg * DEPTH;

  if (tid == 0) {
    prefetch_l2(a.kv_len + seq);
    prefetch_tmap(&k_map);
    prefetch_tmap(&v_map);
    for (int i = 0; i < KG * DEPTH; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], RG);
    }
    s_abort = 0;
    mbar_init_fence();
  }
  pdl_wait();
  // the query rows are requested first: kv_len, page numbers and bytes follow one another
  const int rows_total = a.n * a.G;
  uint4 xq[2][DH / 32];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int rho = rg * 16 + gr + 8 * r;
#pragma unroll
    for (int c = 0; c < DH / 32; ++c) {
      xq[r][c] = make_uint4(0, 0, 0, 0);
      if (rho < rows_total)
        xq[r][c] = *reinterpret_cast<const uint4 *>(
            a.q + ((static_cast<int64_t>(b) * a.n + rho / a.G) * a.Hq + g * a.G + rho % a.G) * DH + t * (DH / 4) + c * 8);
    }
  }
  const int L = static_cast<int>(min(static_cast<int64_t>(max(a.kv_len[seq], 0)), static_cast<int64_t>(a.max_pages) << a.log_page));
  int groups = (L + 15) >> 4;
  if constexpr (SEL) {  // of the entries before the first -1, the last one's page as far as the prefix goes
    int entries = 0;
    for (bool whole = true; whole && entries < a.top;) {
      const uint32_t on = __ballot_sync(0xffffffffu, entries + lane < a.top && list[entries + lane] >= 0);
      entries += on == 0xffffffffu ? 32 : __ffs(~on) - 1;
      whole = on == 0xffffffffu;
    }
    const int64_t tail = entries ? L - (static_cast<int64_t>(list[entries - 1]) << a.log_page) : 0;
    if (entries && tail <= 0) report(a.status, EAGLE_ERR_INVALID);  // past the prefix: nothing of it is read
    groups = entries ? ((entries - 1) << (a.log_page - 4)) +
                           ((static_cast<int>(min(max(tail, static_cast<int64_t>(0)), static_cast<int64_t>(a.page_size))) + 15) >> 4)
                     : 0;
  }
  const int per = (groups + a.S - 1) / a.S;
  const int g0 = min(groups, split * per) + kg, g1 = min(groups, split * per + per);
  const int n_it = g1 > g0 ? (g1 - g0 + KG - 1) / KG : 0;  // this warp's groups: g0, g0 + KG, ..

  // Lane i of batch k looks after iteration 32k + i: its page, then its scales.
  // SEL: `keys` becomes the prefix's positions from its group's first on (16 or more:
  // all of the group counts; 0: none does).
  const auto page_at = [&](int batch, int &keys) {
    const int it = batch * 32 + lane;
    keys = 0;
    if (it >= n_it) return 0;
    int lp = ((g0 + it * KG) << 4) >> a.log_page;
    if constexpr (SEL) {
      const int before = lp ? list[lp - 1] : -1;
      lp = list[lp];
      const int64_t first = (static_cast<int64_t>(lp) << a.log_page) + (((g0 + it * KG) << 4) & (a.page_size - 1));
      if (lp <= before || first >= L) {  // out of order, or past the prefix
        report(a.status, EAGLE_ERR_INVALID);
        return 0;
      }
      keys = L - static_cast<int>(first);
    }
    const int page = a.block_table[static_cast<int64_t>(seq) * a.max_pages + lp];
    if (page >= 0 && page < a.num_pages) return page;
    report(a.status, EAGLE_ERR_INVALID);  // outside the pool: read page 0
    return 0;
  };
  int keys = 0, keys_next = 0;
  int page = page_at(0, keys), page_next = page_at(1, keys_next);
  __syncthreads();
  const auto issue = [&](int it, int pg) {  // lane 0
    unsigned char *dst = ring + (it % DEPTH) * STAGE;
    const int row = ((g0 + it * KG) << 4) & (a.page_size - 1);
    uint64_t *bar = &kfull[it % DEPTH];
    mbar_arrive_expect_tx(bar, STAGE);
    tma_load_3d(dst, &k_map, 0, row, pg * a.Hkv + g, bar);
    tma_load_3d(dst + STAGE / 2, &v_map, 0, row, pg * a.Hkv + g, bar);
  };
  int issued = 0;
  if (rg == 0) {
    for (; issued < min(DEPTH, n_it); ++issued) {
      const int pg = __shfl_sync(0xffffffffu, page, issued);
      if (lane == 0) issue(issued, pg);
    }
    __syncwarp();
  }
  float ks = a.k_scale[static_cast<int64_t>(page) * a.Hkv + g], vs = a.v_scale[static_cast<int64_t>(page) * a.Hkv + g];

  // ---- this warp's 16 query rows, f16 over a power of two of the row ---------
  uint32_t qa[STEPS][4];
  float row_scale[2];
  int node[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int rho = rg * 16 + gr + 8 * r;
    node[r] = rho < rows_total ? rho / a.G : -1;
    const uint4 (&x)[DH / 32] = xq[r];
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < DH / 32; ++c) amax = fmaxf(amax, amax8(x[c]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int e = half_exponent(amax);
    const float f = pow2_clamped(-e);
    row_scale[r] = a.scale_log2 * pow2_clamped(e);
#pragma unroll
    for (int c = 0; c < DH / 32; ++c) {
      qa[2 * c][r] = bf16x2_to_half2(x[c].x, f);
      qa[2 * c][2 + r] = bf16x2_to_half2(x[c].y, f);
      qa[2 * c + 1][r] = bf16x2_to_half2(x[c].z, f);
      qa[2 * c + 1][2 + r] = bf16x2_to_half2(x[c].w, f);
    }
  }

  float acc[NT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[i][c] = 0.f;

  // Scores c of 16 keys (two tiles of eight; masked ones -inf) to P' as the A
  // operand, the running maximum and the sums.
  const auto softmax16 = [&](float (&c)[2][4], float kf, float ve, float vinv, uint32_t (&pa)[4]) {
    float f[2], top[2];
    bool high = false;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      f[r] = fminf(fmaxf(row_scale[r] * kf, 1.2e-38f), 1e38f);
      top[r] = fmaf(fmaxf(fmaxf(c[0][2 * r], c[0][2 * r + 1]), fmaxf(c[1][2 * r], c[1][2 * r + 1])), f[r], ve);
      high |= top[r] > m[r] + 8.f;
    }
    if (__any_sync(0xffffffffu, high)) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
        if (top[r] > m[r] + 8.f) {  // the same in the row's four lanes
          const float alpha = ex2_approx(m[r] - top[r]);  // m = -inf gives 0
          m[r] = top[r];
          l[r] *= alpha;
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            acc[i][2 * r] *= alpha;
            acc[i][2 * r + 1] *= alpha;
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float off = ve + kBias - (m[r] > -INFINITY ? m[r] : 0.f);
      float p[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) p[h][e] = ex2_approx(fmaf(c[h][2 * r + e], f[r], off));
      l[r] = fmaf((p[0][0] + p[0][1]) + (p[1][0] + p[1][1]), vinv, l[r]);
      pa[r] = pack_half2(p[0][0], p[0][1]);
      pa[2 + r] = pack_half2(p[1][0], p[1][1]);
    }
  };

  float ks_next = 1.f, vs_next = 1.f;
  int page_ahead = page_next;  // of iterations that are requested ahead of the batch at hand
  bool ok = true;
  for (int it = 0; it < n_it; ++it) {
    if ((it & 31) == 0) {
      if (it) {
        page = page_next; ks = ks_next; vs = vs_next;
        keys = keys_next;
        page_next = page_at((it >> 5) + 1, keys_next);
        page_ahead = page_next;
      }
      ks_next = a.k_scale[static_cast<int64_t>(page_next) * a.Hkv + g];
      vs_next = a.v_scale[static_cast<int64_t>(page_next) * a.Hkv + g];
    }
    const int st = it % DEPTH;
    if (!warp_wait(&kfull[st], (it / DEPTH) & 1, abort_flag)) { ok = false; break; }
    __syncwarp();
    const unsigned char *kst = ring + st * STAGE, *vst = kst + STAGE / 2;
    // below 16 in the prefix's last group only
    const int valid = SEL ? __shfl_sync(0xffffffffu, keys, it & 31) : L - ((g0 + it * KG) << 4);
    uint32_t kw[2][KW], vw[4][VW];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = gr + 8 * h;
      if constexpr (DH == 128) {
        const uint4 x = lds16(kst + r * 128 + (((2 * t) ^ (r & 7)) << 4)), y = lds16(kst + r * 128 + (((2 * t + 1) ^ (r & 7)) << 4));
        kw[h][0] = x.x; kw[h][1] = x.y; kw[h][2] = x.z; kw[h][3] = x.w;
        kw[h][4] = y.x; kw[h][5] = y.y; kw[h][6] = y.z; kw[h][7] = y.w;
      } else {
        const uint4 x = lds16(kst + r * 64 + ((t ^ ((r >> 1) & 3)) << 4));
        kw[h][0] = x.x; kw[h][1] = x.y; kw[h][2] = x.z; kw[h][3] = x.w;
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = 2 * t + (q & 1) + 8 * (q >> 1);
      if constexpr (DH == 128) {
        const uint4 x = lds16(vst + r * 128 + ((gr ^ (r & 7)) << 4));
        vw[q][0] = x.x; vw[q][1] = x.y; vw[q][2] = x.z; vw[q][3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2 *>(vst + r * 64 + (((gr >> 1) ^ ((r >> 1) & 3)) << 4) + (gr & 1) * 8);
        vw[q][0] = x.x; vw[q][1] = x.y;
      }
    }
    float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int s = 0; s < STEPS; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) mma16816(c[h], qa[s], e4m3_to_half2(kw[h][s] & 0xffffu), e4m3_to_half2(kw[h][s] >> 16));
    // the stage is in registers: the next request into it
    __syncwarp();
    if constexpr (RG == 1) {
      const int nx = it + DEPTH;
      const int pg = __shfl_sync(0xffffffffu, (nx >> 5) == (it >> 5) ? page : page_ahead, nx & 31);
      if (nx < n_it) {
        if (lane == 0) issue(nx, pg);
        issued = nx + 1;
      }
    } else {
      if (lane == 0) mbar_arrive(&kempty[st]);
      // the one before: its readers are likely done
      const int nx = it - 1 + DEPTH;
      if (rg == 0 && it > 0) {
        const int pg = __shfl_sync(0xffffffffu, (nx >> 5) == (it >> 5) ? page : page_ahead, nx & 31);
        if (nx < n_it) {
          if (!warp_wait(&kempty[(it - 1) % DEPTH], ((it - 1) / DEPTH) & 1, abort_flag)) { ok = false; break; }
          __syncwarp();
          if (lane == 0) issue(nx, pg);
          issued = nx + 1;
        }
      }
    }
    __syncwarp();
    if (valid < 16) {  // rows past the prefix: whatever the page holds
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (8 * h + 2 * t + (e & 1) >= valid) c[h][e] = -INFINITY;
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int w = 0; w < VW; ++w)
          if (2 * t + (q & 1) + 8 * (q >> 1) >= valid) vw[q][w] = 0;
    }
    const int ke = scale_exponent(__shfl_sync(0xffffffffu, ks, it & 31)), ve = scale_exponent(__shfl_sync(0xffffffffu, vs, it & 31));
    uint32_t pa[4];
    softmax16(c, exponent_scale(ke), static_cast<float>(ve), exponent_scale(-ve), pa);
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      const uint32_t a0 = __byte_perm(vw[0][w], vw[1][w], 0x5140), a1 = __byte_perm(vw[0][w], vw[1][w], 0x7362);
      const uint32_t b0 = __byte_perm(vw[2][w], vw[3][w], 0x5140), b1 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
      mma16816(acc[4 * w], pa, e4m3_to_half2(a0 & 0xffffu), e4m3_to_half2(b0 & 0xffffu));
      mma16816(acc[4 * w + 1], pa, e4m3_to_half2(a0 >> 16), e4m3_to_half2(b0 >> 16));
      mma16816(acc[4 * w + 2], pa, e4m3_to_half2(a1 & 0xffffu), e4m3_to_half2(b1 & 0xffffu));
      mma16816(acc[4 * w + 3], pa, e4m3_to_half2(a1 >> 16), e4m3_to_half2(b1 >> 16));
    }
  }

  // ---- the tree: groups of 16 nodes, bf16 over the group's powers of two -----
  if (ok && split == a.S - 1) {
    for (int n0 = kg * 16; n0 < nodes; n0 += KG * 16) {
      const int64_t tree = ((SEL ? static_cast<int64_t>(seq) * a.Hkv + g : bg) * static_cast<int64_t>(nodes) + n0) * DH;
      const __nv_bfloat16 *kt = a.k_tree + tree, *vt = a.v_tree + tree;
      uint4 x[2][DH / 32], y[4][DH / 64];
      float kmax = 0.f, vmax = 0.f;
      // the nodes that a row attends to (there are at most kFewRows rows of nodes, so
      // a lane each and one mask word); the others are zeros and decide nothing
      uint32_t attended = 0;
      if constexpr (SEL) {
        attended = static_cast<uint32_t>(a.mask[static_cast<int64_t>(b) * a.W + (n0 >> 6)] >> (n0 & 63)) & 0xffffu;
        if (n0 + 16 > nodes) attended &= (1u << (nodes - n0)) - 1u;
        if (!attended) continue;  // the same in the whole warp
      } else if (lane < a.n) attended = static_cast<uint32_t>(a.mask[static_cast<int64_t>(b) * a.n + lane] >> n0) & 0xffffu;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < DH / 32; ++i) {
          x[h][i] = make_uint4(0, 0, 0, 0);
          if (n0 + gr + 8 * h < nodes && (!SEL || ((attended >> (gr + 8 * h)) & 1u))) x[h][i] = *reinterpret_cast<const uint4 *>(kt + (gr + 8 * h) * DH + t * (DH / 4) + i * 8);
        }
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < DH / 64; ++i) {
          const int r = 2 * t + (q & 1) + 8 * (q >> 1);
          y[q][i] = make_uint4(0, 0, 0, 0);
          if (n0 + r < nodes && (!SEL || ((attended >> r) & 1u))) y[q][i] = *reinterpret_cast<const uint4 *>(vt + r * DH + gr * (DH / 8) + i * 8);
        }
      if constexpr (!SEL) attended = __reduce_or_sync(0xffffffffu, attended);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < DH / 32; ++i) {
          if (!((attended >> (gr + 8 * h)) & 1u)) x[h][i] = make_uint4(0, 0, 0, 0);
          kmax = fmaxf(kmax, amax8(x[h][i]));
        }
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < DH / 64; ++i) {
          if (!((attended >> (2 * t + (q & 1) + 8 * (q >> 1))) & 1u)) y[q][i] = make_uint4(0, 0, 0, 0);
          vmax = fmaxf(vmax, amax8(y[q][i]));
        }
      uint32_t bits[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        bits[r] = 0;
        if (SEL) {
          bits[r] = node[r] >= 0 ? attended : 0u;
          continue;
        }
        if (node[r] >= 0)
          bits[r] = static_cast<uint32_t>(a.mask[static_cast<int64_t>(b) * a.n + node[r]] >> n0) & 0xffffu;
        if (n0 + 16 > a.n) bits[r] &= (1u << (a.n - n0)) - 1u;
      }
      const int ke = half_exponent(warp_max(kmax)), ve = half_exponent(warp_max(vmax));
      const float kf = pow2_clamped(-ke), vf = pow2_clamped(-ve);
      float c[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int i = 0; i < DH / 32; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mma16816(c[h], qa[2 * i], bf16x2_to_half2(x[h][i].x, kf), bf16x2_to_half2(x[h][i].y, kf));
          mma16816(c[h], qa[2 * i + 1], bf16x2_to_half2(x[h][i].z, kf), bf16x2_to_half2(x[h][i].w, kf));
        }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!((bits[e >> 1] >> (8 * h + 2 * t + (e & 1))) & 1u)) c[h][e] = -INFINITY;
      uint32_t pa[4];
      softmax16(c, pow2_clamped(ke), static_cast<float>(ve), pow2_clamped(-ve), pa);
#pragma unroll
      for (int i = 0; i < DH / 64; ++i) {
        const uint32_t w[4][4] = {{y[0][i].x, y[0][i].y, y[0][i].z, y[0][i].w}, {y[1][i].x, y[1][i].y, y[1][i].z, y[1][i].w},
                                  {y[2][i].x, y[2][i].y, y[2][i].z, y[2][i].w}, {y[3][i].x, y[3][i].y, y[3][i].z, y[3][i].w}};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          mma16816(acc[8 * i + 2 * j], pa, bf16x2_to_half2(__byte_perm(w[0][j], w[1][j], 0x5410), vf),
                   bf16x2_to_half2(__byte_perm(w[2][j], w[3][j], 0x5410), vf));
          mma16816(acc[8 * i + 2 * j + 1], pa, bf16x2_to_half2(__byte_perm(w[0][j], w[1][j], 0x7632), vf),
                   bf16x2_to_half2(__byte_perm(w[2][j], w[3][j], 0x7632), vf));
        }
      }
    }
  }
  pdl_trigger();

  // ---- the CTA's key groups together ------------------------------------------
  if (!ok && rg == 0 && lane == 0) {
    // copies still in flight complete before shared memory is used again or released
    volatile int never = 0;
    for (int i = max(0, issued - DEPTH); i < issued; ++i) mbar_wait(&kfull[i % DEPTH], (i / DEPTH) & 1, &never, 100000000ull);
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
  }
  __syncthreads();  // every ring has been read
  float4 *o4 = reinterpret_cast<float4 *>(ring0) + warp * 16 * (DH / 4);
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = gr + 8 * r;
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < NT / 4; ++i)
        o4[o_chunk<DH>(row, (2 * t + e) * (NT / 4) + i)] =
            make_float4(acc[4 * i][2 * r + e], acc[4 * i + 1][2 * r + e], acc[4 * i + 2][2 * r + e], acc[4 * i + 3][2 * r + e]);
    if (t == 0) s_ml[warp * 16 + row] = make_float2(m[r], l[r]);
  }
  __syncthreads();
  if (*abort_flag && tid == 0) report(a.status, EAGLE_ERR_TIMEOUT);
  constexpr int NV = DH / 4;
  float *slot = a.part + (static_cast<int64_t>(bg) * a.S + split) * a.slot_rows * (DH + 2);
  for (int item = tid; item < rows_total * NV; item += 128) {
    const int rho = item / NV, cc = item % NV, row = rho & 15, w0 = rho >> 4;
    float M = -INFINITY, Ls = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < KG; ++k) M = fmaxf(M, s_ml[(k * RG + w0) * 16 + row].x);
#pragma unroll
    for (int k = 0; k < KG; ++k) {
      const float2 ml = s_ml[(k * RG + w0) * 16 + row];
      const float w = ml.x > -INFINITY ? ex2_approx(ml.x - M) : 0.f;
      const float4 x = reinterpret_cast<const float4 *>(ring0)[(k * RG + w0) * 16 * NV + o_chunk<DH>(row, cc)];
      Ls = fmaf(w, ml.y, Ls);
      o.x = fmaf(w, x.x, o.x); o.y = fmaf(w, x.y, o.y);
      o.z = fmaf(w, x.z, o.z); o.w = fmaf(w, x.w, o.w);
    }
    if constexpr (MERGE == 0) {
      kv8_write_out<DH>(a, bg, rho, cc, o, M, Ls);
    } else {
      reinterpret_cast<float4 *>(slot)[item] = o;
      if (cc == 0) reinterpret_cast<float2 *>(slot + static_cast<int64_t>(a.slot_rows) * DH)[rho] = make_float2(M, Ls);
    }
  }
  // one wave: the S splits are a cluster and share the merge
  if constexpr (MERGE == 1) {
    cluster_arrive_release();
    cluster_wait();
    if (*abort_flag) return;
    const int share = (rows_total * NV + a.S - 1) / a.S, i0 = static_cast<int>(cluster_ctarank()) * share;
    for (int item = i0 + tid; item < min(rows_total * NV, i0 + share); item += 128)
      kv8_merge_item<DH>(a, bg, 0, 1, 1, item / NV, item % NV);
  }
}

// ---- host side ---------------------------------------------------------------

struct FewPlan {
  int RG, S;
  bool cluster;
};

// Row tiles a CTA, and the KV split S that minimises (CTAs an SM slot) x (groups
// a warp + a CTA's fixed cost in groups).
static FewPlan few_plan(int B, int rows, int Hkv, int Lmax, int num_sms) {
  FewPlan p;
  p.RG = rows <= 16 ? 1 : 2;
  const int KG = 4 / p.RG;
  const int64_t base = static_cast<int64_t>(B) * Hkv, slots = 3ll * num_sms;
  const int64_t groups = (static_cast<int64_t>(Lmax) + 15) / 16;
  double best = 1e30;
  p.S = 1;
  for (int S = 1; S <= kMaxSplitsFew && (S == 1 || static_cast<int64_t>(S) * KG * 2 <= groups); ++S) {
    const double load = static_cast<double>(base * S) / slots;
    const double waves = load <= 1.0 ? 1.0 : (load <= 3.0 ? static_cast<double>((base * S + slots - 1) / slots) : load + 0.5);
    const double cost = waves * (static_cast<double>(groups) / (S * KG) + 12.0 + (S > 1 ? 4.0 : 0.0));
    if (cost < best * 0.97) {
      best = cost;
      p.S = S;
    }
  }
  p.cluster = p.S <= kMaxClusterSplits8 && base * p.S <= slots;
  return p;
}

size_t attn_kv8_few_workspace_bytes(int B, int n, int Hq, int Hkv, int dh, int Lmax, int num_sms) {
  const int rows = n * (Hq / Hkv);
  const FewPlan p = few_plan(B, rows, Hkv, Lmax, num_sms);
  return p.S <= 1 ? 0 : static_cast<size_t>(B) * Hkv * p.S * ((rows + 7) / 8 * 8) * (dh + 2) * sizeof(float);
}

template <int DH, int RG, int MERGE, bool SEL>
static cudaError_t launch_few_v(const CUtensorMap *maps, const typename FewArgs<SEL>::type &a, cudaStream_t st) {
  static std::atomic<unsigned long long> configured{0};
  constexpr int kSmem = kRingBytes + 1024;
  const auto kernel = tree_attn_kv8_few_kernel<DH, RG, MERGE, SEL>;
  cudaError_t e = set_smem_limit_once(kernel, kSmem, configured);
  if (e != cudaSuccess) return e;
  const dim3 grid(SEL ? a.S * a.B * a.Hkv : a.S, 1, SEL ? 1 : a.B * a.Hkv);
  if constexpr (MERGE == 1)
    return launch_chained_cluster(kernel, grid, dim3(128), kSmem, st, a.S, maps[0], maps[1], a);
  e = launch_chained(kernel, grid, dim3(128), kSmem, st, maps[0], maps[1], a);
  if (e != cudaSuccess || MERGE == 0) return e;
  if constexpr (SEL) {
    const int64_t items = static_cast<int64_t>(a.B) * a.Hkv * a.n * a.G * (DH / 4);
    return launch_chained(tree_attn_kv8_merge_flat_kernel<DH>, dim3(static_cast<unsigned>((items + 255) / 256)), dim3(256), 0,
                          st, static_cast<const Kv8Args &>(a));
  }
  return launch_chained(tree_attn_kv8_merge_kernel<DH>, dim3((a.slot_rows * (DH / 4) + 255) / 256, 1, a.B * a.Hkv), dim3(256), 0,
                        st, a, 1);
}

template <int DH, int RG, bool SEL>
static cudaError_t launch_few_t(const CUtensorMap *maps, const typename FewArgs<SEL>::type &a, const FewPlan &p, cudaStream_t st) {
  if (p.S == 1) return launch_few_v<DH, RG, 0, SEL>(maps, a, st);
  return p.cluster ? launch_few_v<DH, RG, 1, SEL>(maps, a, st) : launch_few_v<DH, RG, 2, SEL>(maps, a, st);
}

template <bool SEL>
static cudaError_t launch_few(typename FewArgs<SEL>::type a, const void *k_pages, const void *v_pages, int dh, int Lmax, void *ws,
                              int num_sms, cudaStream_t st) {
  const int rows = a.n * a.G;
  const FewPlan p = few_plan(a.B, rows, a.Hkv, Lmax, num_sms);
  if (p.S > 1 && !ws) return cudaErrorInvalidValue;
  a.S = p.S;
  a.page_box = 16;
  a.part = p.S > 1 ? reinterpret_cast<float *>(ws) : nullptr;
  a.slot_rows = (rows + 7) / 8 * 8;
  CUtensorMap maps[2];
  const int64_t blocks = static_cast<int64_t>(a.num_pages) * a.Hkv;
  if (!make_pool_map(&maps[0], k_pages, blocks, a.page_size, dh, 16, true) ||
      !make_pool_map(&maps[1], v_pages, blocks, a.page_size, dh, 16, true))
    return cudaErrorInvalidValue;
  if (dh == 64) {
    if (p.RG == 1) return launch_few_t<64, 1, SEL>(maps, a, p, st);
    return launch_few_t<64, 2, SEL>(maps, a, p, st);
  }
  if (p.RG == 1) return launch_few_t<128, 1, SEL>(maps, a, p, st);
  return launch_few_t<128, 2, SEL>(maps, a, p, st);
}

cudaError_t launch_tree_attn_kv8_few(Kv8Args a, const void *k_pages, const void *v_pages, int dh, void *ws, int num_sms,
                                     cudaStream_t st) {
  return launch_few<false>(a, k_pages, v_pages, dh, a.max_pages * a.page_size, ws, num_sms, st);
}

cudaError_t launch_tree_attn_kv8_pages_few(const Kv8SelArgs &a, const void *k_pages, const void *v_pages, int dh, int Lmax, void *ws,
                                           int num_sms, cudaStream_t st) {
  return launch_few<true>(a, k_pages, v_pages, dh, Lmax, ws, num_sms, st);
}

}  // namespace eagle
