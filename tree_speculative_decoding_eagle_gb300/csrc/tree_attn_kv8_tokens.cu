// Attention over selected pages of the 8-bit cache for up to eight query rows a node
// and KV head (heads grouped by eight or fewer): the few-row kernel of
// tree_attn_kv8_few.cu with the operands the other way round.
//
// m16n8k16 has 16 rows for its A operand and eight for B.  Eight query rows as A would
// leave half of each product and half of the accumulators empty; here keys are A in
// S^T = K Q^T and columns of V are A in O^T = V^T P^T, the query rows the eight of B.
// Half the MMAs, half the exponentials, and 32 accumulators a thread instead of 64, so
// four CTAs of four warps share an SM instead of three:
//   * a lane's 16-byte pieces of K are A fragments once converted, word by word,
//     because the order of the head's columns in the dot product is free; V's
//     fragments pair two keys of one column, and which column is which row is free;
//   * P^T leaves the first product with keys down the lanes and is wanted with keys
//     across them: two movmatrix transpositions of 8 x 8 weights;
//   * the running maximum is looked at across the warp only when a lane's own exceeds
//     it by more than 2^8.
// Everything else (rings of bytes by TMA, a warp a run of 16-key groups, the merge)
// and the arithmetic are as there.
//
// What bounds it: HBM for a batch of single tokens, each CTA's chain (length - list -
// page number - bytes) for one.  Measured, on the device: 64 tokens, 64 heads on 8 of
// 128, 32 pages of 64 each 51.4 us (261 MB, 79 % of the copy rate; 75.8 in the few-row
// kernel); one token, 32 heads of 128, 64 pages of 16 9.2 us.
#include "kv8_attn.cuh"

namespace eagle {

using namespace sm100;

constexpr int kTokenRing = 49152;     // bytes a CTA, a quarter each warp's
constexpr int kTokenCtas = 4;         // an SM
constexpr int kMaxSplitsTokens = 32;

__device__ __forceinline__ void mma_t(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 tile of 16-bit numbers, a lane's two of row lane / 4, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t half2_of(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint4 lds_vec(const unsigned char *p) { return *reinterpret_cast<const uint4 *>(p); }

template <int DH, int MERGE>
__global__ void __launch_bounds__(128, kTokenCtas)
    tree_attn_kv8_tokens_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map, Kv8SelArgs a) {
  constexpr int KG = 4;
  constexpr int STAGE = 32 * DH;                  // 16 keys' K, then V
  constexpr int DEPTH = kTokenRing / KG / STAGE;
  constexpr int STEPS = DH / 16, NT = DH / 16;    // k steps of K Q^T, 16-column tiles of V
  constexpr int KW = DH / 16, VW = DH / 32;       // words of a K row, of a V row a lane holds
  constexpr int NV = DH / 4;
  extern __shared__ __align__(1024) unsigned char token_smem[];
  unsigned char *ring0 = token_smem + ((1024 - (smem_u32(token_smem) & 1023)) & 1023);
  __shared__ uint64_t full[KG * DEPTH];
  __shared__ float2 s_ml[KG * 8];
  __shared__ int s_abort;
  volatile int *abort_flag = &s_abort;

  const int tid = threadIdx.x, kg = tid >> 5, lane = tid & 31, gr = lane >> 2, t = lane & 3;
  const int split = blockIdx.x % a.S, bg = blockIdx.x / a.S;
  const int b = bg / a.Hkv, g = bg % a.Hkv, seq = b / a.nodes;  // b: a node of a sequence
  unsigned char *ring = ring0 + kg * DEPTH * STAGE;
  uint64_t *kfull = full + kg * DEPTH;

  if (tid == 0) {
    prefetch_l2(a.kv_len + seq);
    prefetch_tmap(&k_map);
    prefetch_tmap(&v_map);
    for (int i = 0; i < KG * DEPTH; ++i) mbar_init(&full[i], 1);
    s_abort = 0;
    mbar_init_fence();
  }
  pdl_wait();
  // the list first: lengths, entries, page numbers and bytes follow one another
  const int32_t *list = a.sel + static_cast<int64_t>(bg) * a.top;
  const int L = static_cast<int>(min(static_cast<int64_t>(max(a.kv_len[seq], 0)), static_cast<int64_t>(a.max_pages) << a.log_page));
  int entries = 0;  // before the first that is negative
  for (bool whole = true; whole && entries < a.top;) {
    const uint32_t on = __ballot_sync(0xffffffffu, entries + lane < a.top && list[entries + lane] >= 0);
    entries += on == 0xffffffffu ? 32 : __ffs(~on) - 1;
    whole = on == 0xffffffffu;
  }
  uint4 xq[DH / 32];
#pragma unroll
  for (int c = 0; c < DH / 32; ++c) {
    xq[c] = make_uint4(0, 0, 0, 0);
    if (gr < a.G) xq[c] = *reinterpret_cast<const uint4 *>(a.q + (static_cast<int64_t>(b) * a.Hq + g * a.G + gr) * DH + t * (DH / 4) + c * 8);
  }
  const int64_t tail = entries ? L - (static_cast<int64_t>(list[entries - 1]) << a.log_page) : 0;
  if (entries && tail <= 0) report(a.status, EAGLE_ERR_INVALID);  // past the prefix: nothing of it is read
  const int groups = entries ? ((entries - 1) << (a.log_page - 4)) +
                                   ((static_cast<int>(min(max(tail, static_cast<int64_t>(0)), static_cast<int64_t>(a.page_size))) + 15) >> 4)
                             : 0;
  const int per = (groups + a.S - 1) / a.S;
  const int g0 = min(groups, split * per) + kg, g1 = min(groups, split * per + per);
  const int n_it = g1 > g0 ? (g1 - g0 + KG - 1) / KG : 0;  // this warp's groups: g0, g0 + KG, ..

  // Lane i of batch k looks after iteration 32k + i: its page, and `keys`, the
  // prefix's positions from the group's first on (16 or more: all of the group
  // counts; 0: none does).
  const auto page_at = [&](int batch, int &keys) {
    const int it = batch * 32 + lane;
    keys = 0;
    if (it >= n_it) return 0;
    const int at = (g0 + it * KG) << 4, entry = at >> a.log_page;
    const int before = entry ? list[entry - 1] : -1, lp = list[entry];
    const int64_t first = (static_cast<int64_t>(lp) << a.log_page) + (at & (a.page_size - 1));
    if (lp <= before || first >= L) {  // out of order, or past the prefix
      report(a.status, EAGLE_ERR_INVALID);
      return 0;
    }
    keys = L - static_cast<int>(first);
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
  for (; issued < min(DEPTH, n_it); ++issued) {
    const int pg = __shfl_sync(0xffffffffu, page, issued);
    if (lane == 0) issue(issued, pg);
  }
  __syncwarp();
  float ks = a.k_scale[static_cast<int64_t>(page) * a.Hkv + g], vs = a.v_scale[static_cast<int64_t>(page) * a.Hkv + g];

  // ---- the query rows as B, f16 over a power of two of the row -------------------
  uint32_t qb[STEPS][2];
  float row_scale[2];  // of rows 2t, 2t + 1
  {
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < DH / 32; ++c) amax = fmaxf(amax, amax8(xq[c]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int e = half_exponent(amax);
    const float f = pow2_clamped(-e), own = a.scale_log2 * pow2_clamped(e);
#pragma unroll
    for (int r = 0; r < 2; ++r) row_scale[r] = __shfl_sync(0xffffffffu, own, (2 * t + r) * 4);
#pragma unroll
    for (int c = 0; c < DH / 32; ++c) {
      qb[2 * c][0] = bf16x2_to_half2(xq[c].x, f);
      qb[2 * c][1] = bf16x2_to_half2(xq[c].y, f);
      qb[2 * c + 1][0] = bf16x2_to_half2(xq[c].z, f);
      qb[2 * c + 1][1] = bf16x2_to_half2(xq[c].w, f);
    }
  }

  // acc[i]: columns 2i (elements 0, 1) and 2i + 1 (2, 3) of the lane's DH / 8, rows 2t, 2t + 1
  float acc[NT][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[i][c] = 0.f;

  // Scores c of 16 keys (elements 0, 1: key gr, rows 2t, 2t + 1; 2, 3: key gr + 8;
  // masked ones -inf) to P^T as the B operand, the running maximum and the sums.
  const auto softmax16 = [&](const float (&c)[4], float kf, float ve, float vinv, uint32_t &p0, uint32_t &p1) {
    float f[2], top[2];
    bool high = false;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      f[r] = fminf(fmaxf(row_scale[r] * kf, 1.2e-38f), 1e38f);
      top[r] = fmaf(fmaxf(c[r], c[2 + r]), f[r], ve);
      high |= top[r] > m[r] + 8.f;
    }
    if (__any_sync(0xffffffffu, high)) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], o));
        if (top[r] > m[r] + 8.f) {  // the same in the row's eight lanes
          const float alpha = ex2_approx(m[r] - top[r]);  // m = -inf gives 0
          m[r] = top[r];
          l[r] *= alpha;
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            acc[i][r] *= alpha;
            acc[i][2 + r] *= alpha;
          }
        }
      }
    }
    float p[2][2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float off = ve + kBias - (m[r] > -INFINITY ? m[r] : 0.f);
#pragma unroll
      for (int h = 0; h < 2; ++h) p[h][r] = ex2_approx(fmaf(c[2 * h + r], f[r], off));
      l[r] = fmaf(p[0][r] + p[1][r], vinv, l[r]);
    }
    p0 = transposed(half2_of(p[0][0], p[0][1]));
    p1 = transposed(half2_of(p[1][0], p[1][1]));
  };

  float ks_next = 1.f, vs_next = 1.f;
  int page_ahead = page_next;  // of iterations that are requested ahead of the batch at hand
  bool ok = true;
  for (int it = 0; it < n_it; ++it) {
    if ((it & 31) == 0) {
      if (it) {
        page = page_next; ks = ks_next; vs = vs_next; keys = keys_next;
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
    const int valid = __shfl_sync(0xffffffffu, keys, it & 31);  // below 16 in the last page's last group
    uint32_t kw[2][KW], vw[4][VW];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = gr + 8 * h;
      if constexpr (DH == 128) {
        const uint4 x = lds_vec(kst + r * 128 + (((2 * t) ^ (r & 7)) << 4)), y = lds_vec(kst + r * 128 + (((2 * t + 1) ^ (r & 7)) << 4));
        kw[h][0] = x.x; kw[h][1] = x.y; kw[h][2] = x.z; kw[h][3] = x.w;
        kw[h][4] = y.x; kw[h][5] = y.y; kw[h][6] = y.z; kw[h][7] = y.w;
      } else {
        const uint4 x = lds_vec(kst + r * 64 + ((t ^ ((r >> 1) & 3)) << 4));
        kw[h][0] = x.x; kw[h][1] = x.y; kw[h][2] = x.z; kw[h][3] = x.w;
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = 2 * t + (q & 1) + 8 * (q >> 1);
      if constexpr (DH == 128) {
        const uint4 x = lds_vec(vst + r * 128 + ((gr ^ (r & 7)) << 4));
        vw[q][0] = x.x; vw[q][1] = x.y; vw[q][2] = x.z; vw[q][3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2 *>(vst + r * 64 + (((gr >> 1) ^ ((r >> 1) & 3)) << 4) + (gr & 1) * 8);
        vw[q][0] = x.x; vw[q][1] = x.y;
      }
    }
    float c[4] = {0.f, 0.f, 0.f, 0.f}, c2[4] = {0.f, 0.f, 0.f, 0.f};  // two chains
#pragma unroll
    for (int s = 0; s < STEPS; s += 2) {
      mma_t(c, e4m3_to_half2(kw[0][s] & 0xffffu), e4m3_to_half2(kw[1][s] & 0xffffu), e4m3_to_half2(kw[0][s] >> 16),
            e4m3_to_half2(kw[1][s] >> 16), qb[s][0], qb[s][1]);
      mma_t(c2, e4m3_to_half2(kw[0][s + 1] & 0xffffu), e4m3_to_half2(kw[1][s + 1] & 0xffffu), e4m3_to_half2(kw[0][s + 1] >> 16),
            e4m3_to_half2(kw[1][s + 1] >> 16), qb[s + 1][0], qb[s + 1][1]);
    }
    // the stage is in registers: the next request into it
    __syncwarp();
    {
      const int nx = it + DEPTH;
      const int pg = __shfl_sync(0xffffffffu, (nx >> 5) == (it >> 5) ? page : page_ahead, nx & 31);
      if (nx < n_it) {
        if (lane == 0) issue(nx, pg);
        issued = nx + 1;
      }
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < 4; ++e) c[e] += c2[e];
    if (valid < 16) {  // rows past the prefix: whatever the page holds
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (gr + 8 * (e >> 1) >= valid) c[e] = -INFINITY;
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int w = 0; w < VW; ++w)
          if (2 * t + (q & 1) + 8 * (q >> 1) >= valid) vw[q][w] = 0;
    }
    const int ke = scale_exponent(__shfl_sync(0xffffffffu, ks, it & 31)), ve = scale_exponent(__shfl_sync(0xffffffffu, vs, it & 31));
    uint32_t p0, p1;
    softmax16(c, exponent_scale(ke), static_cast<float>(ve), exponent_scale(-ve), p0, p1);
#pragma unroll
    for (int w = 0; w < VW; ++w) {
      const uint32_t a0 = __byte_perm(vw[0][w], vw[1][w], 0x5140), a1 = __byte_perm(vw[0][w], vw[1][w], 0x7362);
      const uint32_t b0 = __byte_perm(vw[2][w], vw[3][w], 0x5140), b1 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
      mma_t(acc[2 * w], e4m3_to_half2(a0 & 0xffffu), e4m3_to_half2(a0 >> 16), e4m3_to_half2(b0 & 0xffffu), e4m3_to_half2(b0 >> 16), p0, p1);
      mma_t(acc[2 * w + 1], e4m3_to_half2(a1 & 0xffffu), e4m3_to_half2(a1 >> 16), e4m3_to_half2(b1 & 0xffffu), e4m3_to_half2(b1 >> 16), p0, p1);
    }
  }

  // ---- the tree: groups of 16 nodes, bf16 over the group's powers of two -----
  if (ok && split == a.S - 1) {
    for (int n0 = kg * 16; n0 < a.nodes; n0 += KG * 16) {
      uint32_t attended = static_cast<uint32_t>(a.mask[static_cast<int64_t>(b) * a.W + (n0 >> 6)] >> (n0 & 63)) & 0xffffu;
      if (n0 + 16 > a.nodes) attended &= (1u << (a.nodes - n0)) - 1u;
      if (!attended) continue;  // the same in the whole warp
      const int64_t tree = ((static_cast<int64_t>(seq) * a.Hkv + g) * a.nodes + n0) * DH;
      const __nv_bfloat16 *kt = a.k_tree + tree, *vt = a.v_tree + tree;
      // nodes that the row does not name are zeros, whatever they hold
      float kmax = 0.f, vmax = 0.f;
      float c[4] = {0.f, 0.f, 0.f, 0.f};
      {
        uint4 x[2][DH / 32];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < DH / 32; ++i) {
            x[h][i] = make_uint4(0, 0, 0, 0);
            if ((attended >> (gr + 8 * h)) & 1u) x[h][i] = *reinterpret_cast<const uint4 *>(kt + (gr + 8 * h) * DH + t * (DH / 4) + i * 8);
            kmax = fmaxf(kmax, amax8(x[h][i]));
          }
        kmax = warp_max(kmax);
        const float kf = pow2_clamped(-half_exponent(kmax));
#pragma unroll
        for (int i = 0; i < DH / 32; ++i) {
          mma_t(c, bf16x2_to_half2(x[0][i].x, kf), bf16x2_to_half2(x[1][i].x, kf), bf16x2_to_half2(x[0][i].y, kf),
                bf16x2_to_half2(x[1][i].y, kf), qb[2 * i][0], qb[2 * i][1]);
          mma_t(c, bf16x2_to_half2(x[0][i].z, kf), bf16x2_to_half2(x[1][i].z, kf), bf16x2_to_half2(x[0][i].w, kf),
                bf16x2_to_half2(x[1][i].w, kf), qb[2 * i + 1][0], qb[2 * i + 1][1]);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (!((attended >> (gr + 8 * (e >> 1))) & 1u)) c[e] = -INFINITY;
      uint4 y[4][DH / 64];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < DH / 64; ++i) {
          const int r = 2 * t + (q & 1) + 8 * (q >> 1);
          y[q][i] = make_uint4(0, 0, 0, 0);
          if ((attended >> r) & 1u) y[q][i] = *reinterpret_cast<const uint4 *>(vt + r * DH + gr * (DH / 8) + i * 8);
          vmax = fmaxf(vmax, amax8(y[q][i]));
        }
      const int ve = half_exponent(warp_max(vmax));
      const float vf = pow2_clamped(-ve);
      uint32_t p0, p1;
      softmax16(c, pow2_clamped(half_exponent(kmax)), static_cast<float>(ve), pow2_clamped(-ve), p0, p1);
#pragma unroll
      for (int i = 0; i < DH / 64; ++i) {
        const uint32_t w[4][4] = {{y[0][i].x, y[0][i].y, y[0][i].z, y[0][i].w}, {y[1][i].x, y[1][i].y, y[1][i].z, y[1][i].w},
                                  {y[2][i].x, y[2][i].y, y[2][i].z, y[2][i].w}, {y[3][i].x, y[3][i].y, y[3][i].z, y[3][i].w}};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma_t(acc[4 * i + j], bf16x2_to_half2(__byte_perm(w[0][j], w[1][j], 0x5410), vf),
                bf16x2_to_half2(__byte_perm(w[0][j], w[1][j], 0x7632), vf), bf16x2_to_half2(__byte_perm(w[2][j], w[3][j], 0x5410), vf),
                bf16x2_to_half2(__byte_perm(w[2][j], w[3][j], 0x7632), vf), p0, p1);
      }
    }
  }
  pdl_trigger();

  // ---- the CTA's warps together -----------------------------------------------
  if (!ok && lane == 0) {
    // copies still in flight complete before shared memory is used again or released
    volatile int never = 0;
    for (int i = max(0, issued - DEPTH); i < issued; ++i) mbar_wait(&kfull[i % DEPTH], (i / DEPTH) & 1, &never, 100000000ull);
  }
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
  __syncthreads();  // every ring has been read
  // 16-byte chunk c of row r lies at chunk c ^ (r / 2), so eight lanes of a store touch every bank once
  float4 *o4 = reinterpret_cast<float4 *>(ring0) + kg * 8 * NV;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
#pragma unroll
    for (int w = 0; w < VW; ++w)
      o4[(2 * t + r) * NV + ((gr * VW + w) ^ t)] = make_float4(acc[2 * w][r], acc[2 * w][2 + r], acc[2 * w + 1][r], acc[2 * w + 1][2 + r]);
    if (gr == 0) s_ml[kg * 8 + 2 * t + r] = make_float2(m[r], l[r]);
  }
  __syncthreads();
  if (*abort_flag && tid == 0) report(a.status, EAGLE_ERR_TIMEOUT);
  float *slot = a.part + (static_cast<int64_t>(bg) * a.S + split) * a.slot_rows * (DH + 2);
  for (int item = tid; item < a.G * NV; item += 128) {
    const int rho = item / NV, cc = item % NV;
    float M = -INFINITY, Ls = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < KG; ++k) M = fmaxf(M, s_ml[k * 8 + rho].x);
#pragma unroll
    for (int k = 0; k < KG; ++k) {
      const float2 ml = s_ml[k * 8 + rho];
      const float w = ml.x > -INFINITY ? ex2_approx(ml.x - M) : 0.f;
      const float4 x = reinterpret_cast<const float4 *>(ring0)[(k * 8 + rho) * NV + (cc ^ (rho >> 1))];
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
    const int share = (a.G * NV + a.S - 1) / a.S, i0 = static_cast<int>(cluster_ctarank()) * share;
    for (int item = i0 + tid; item < min(a.G * NV, i0 + share); item += 128)
      kv8_merge_item<DH>(a, bg, 0, 1, 1, item / NV, item % NV);
  }
}

// ---- host side ---------------------------------------------------------------

struct TokenPlan {
  int S;
  bool cluster;
};

// The KV split that minimises (CTAs an SM slot) x (groups a warp + a CTA's fixed
// cost in groups).
static TokenPlan token_plan(int64_t base, int positions, int num_sms) {
  TokenPlan p = {1, false};
  const int64_t slots = static_cast<int64_t>(kTokenCtas) * num_sms, groups = (static_cast<int64_t>(positions) + 15) / 16;
  double best = 1e30;
  for (int S = 1; S <= kMaxSplitsTokens && (S == 1 || S * 8ll <= groups); ++S) {
    const double load = static_cast<double>(base * S) / slots;
    const double waves = load <= 1.0 ? 1.0 : (load <= 3.0 ? static_cast<double>((base * S + slots - 1) / slots) : load + 0.5);
    const double cost = waves * (static_cast<double>(groups) / (S * 4) + 12.0 + (S > 1 ? 4.0 : 0.0));
    if (cost < best * 0.97) {
      best = cost;
      p.S = S;
    }
  }
  p.cluster = p.S <= kMaxClusterSplits8 && base * p.S <= slots;
  return p;
}

size_t attn_kv8_tokens_workspace_bytes(int64_t nodes, int Hkv, int dh, int positions, int num_sms) {
  const TokenPlan p = token_plan(nodes * Hkv, positions, num_sms);
  return p.S <= 1 ? 0 : static_cast<size_t>(nodes) * Hkv * p.S * 8 * (dh + 2) * sizeof(float);
}

template <int DH, int MERGE>
static cudaError_t launch_tokens_v(const CUtensorMap *maps, const Kv8SelArgs &a, cudaStream_t st) {
  static std::atomic<unsigned long long> configured{0};
  constexpr int kSmem = kTokenRing + 1024;
  const auto kernel = tree_attn_kv8_tokens_kernel<DH, MERGE>;
  cudaError_t e = set_smem_limit_once(kernel, kSmem, configured);
  if (e != cudaSuccess) return e;
  const dim3 grid(a.S * a.B * a.Hkv);
  if constexpr (MERGE == 1) return launch_chained_cluster(kernel, grid, dim3(128), kSmem, st, a.S, maps[0], maps[1], a);
  e = launch_chained(kernel, grid, dim3(128), kSmem, st, maps[0], maps[1], a);
  if (e != cudaSuccess || MERGE == 0) return e;
  const int64_t items = static_cast<int64_t>(a.B) * a.Hkv * a.G * (DH / 4);
  return launch_chained(tree_attn_kv8_merge_flat_kernel<DH>, dim3(static_cast<unsigned>((items + 255) / 256)), dim3(256), 0, st,
                        static_cast<const Kv8Args &>(a));
}

template <int DH>
static cudaError_t launch_tokens_t(const CUtensorMap *maps, const Kv8SelArgs &a, const TokenPlan &p, cudaStream_t st) {
  if (p.S == 1) return launch_tokens_v<DH, 0>(maps, a, st);
  return p.cluster ? launch_tokens_v<DH, 1>(maps, a, st) : launch_tokens_v<DH, 2>(maps, a, st);
}

cudaError_t launch_tree_attn_kv8_tokens(Kv8SelArgs a, const void *k_pages, const void *v_pages, int dh, int positions, void *ws,
                                        int num_sms, cudaStream_t st) {
  const TokenPlan p = token_plan(static_cast<int64_t>(a.B) * a.Hkv, positions, num_sms);
  if (p.S > 1 && !ws) return cudaErrorInvalidValue;
  a.S = p.S;
  a.page_box = 16;
  a.part = p.S > 1 ? reinterpret_cast<float *>(ws) : nullptr;
  a.slot_rows = 8;
  CUtensorMap maps[2];
  const int64_t blocks = static_cast<int64_t>(a.num_pages) * a.Hkv;
  if (!make_pool_map(&maps[0], k_pages, blocks, a.page_size, dh, 16, true) ||
      !make_pool_map(&maps[1], v_pages, blocks, a.page_size, dh, 16, true))
    return cudaErrorInvalidValue;
  return dh == 64 ? launch_tokens_t<64>(maps, a, p, st) : launch_tokens_t<128>(maps, a, p, st);
}

}  // namespace eagle
