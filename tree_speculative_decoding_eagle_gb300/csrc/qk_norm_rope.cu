// Norms of queries and keys for each head, their weight and the rotary position in
// one pass, into the tree attention's layouts (rope.cu without the norm).
//
// A head x of dh columns becomes y_c = x_c r (w_c + offset), r = 1 / sqrt(mean of
// x^2 + eps), and its pairs then turn as in rope.cu: y' = factor * R(position) y.
// Everything from the element as loaded to the turned one is float32, rounded once
// to the output type; the sum of squares runs over a lane's columns, then over the
// head's lanes in a fixed order, so a head's result does not depend on the launch.
//
// What bounds it: HBM (each element read once and written once), latency for one
// tree.  Heads are numbered node by node and a CTA takes a run of them, whatever
// their nodes: no place for a head stays empty, and the turns of the two or three
// nodes in the run are computed by all threads while the heads' vectors are on
// their way.  A group of lanes holds a head's 16-byte vectors in registers between
// the sum and the rotation, so the head is read once.
#include "rope.cuh"

namespace eagle {

constexpr int kNormThreads = 256;

struct NormArgs {
  RopeArgs r;
  const void *q_weight, *k_weight;  // [dh] of the same type, or NULL: ones
  float eps, offset;
  int64_t heads;  // B * n * (Hq + Hkv, and Hkv of v)
};

// The run of heads a CTA takes: its first node, the first head's place in that
// node, and the nodes it touches.
struct HeadRun {
  int H, node0, rem, nodes;
  int64_t base;
  __device__ __forceinline__ HeadRun(const NormArgs &a, int count) {
    H = a.r.Hq + (a.r.v ? 2 : 1) * a.r.Hkv;
    base = static_cast<int64_t>(blockIdx.x) * count;
    node0 = static_cast<int>(base / H);
    rem = static_cast<int>(base - static_cast<int64_t>(node0) * H);
    const int64_t last = min(base + count, a.heads) - 1;
    nodes = static_cast<int>(last / H) - node0 + 1;
  }
};
// cos and sin of the run's nodes: node k's pair j at cs[k * half + j].
__device__ __forceinline__ void run_turns(const RopeArgs &a, const HeadRun &run, float2 *cs) {
  for (int idx = threadIdx.x; idx < run.nodes * a.half; idx += kNormThreads) {
    const int k = idx / a.half, node = run.node0 + k, b = node / a.n;
    cs[idx] = turn_of(a, position_of(a, node, b, node - b * a.n), idx - k * a.half);
  }
}

// 16-byte vectors, `lanes` threads a head, NI items a lane (an item as in rope.cu:
// two vectors half of rot_dim apart, one vector of whole pairs, or one that does
// not turn), U heads a thread with their loads in flight together.
template <typename T, bool INTER, int NI>
__global__ void __launch_bounds__(kNormThreads) norm_rope_vec_kernel(NormArgs a, int log_lanes, int items) {
  constexpr int E = VecTraits<T>::kElems, U = NI == 1 ? 2 : 1;
  extern __shared__ float2 norm_cs[];
  const int lanes = 1 << log_lanes, slots = kNormThreads >> log_lanes;
  const int lane = threadIdx.x & (lanes - 1), slot = threadIdx.x >> log_lanes;
  const HeadRun run(a, U * slots);
  const int dh = a.r.dh, half = a.r.half;
  const int turning = INTER ? 2 * half / E : half / E;  // items that turn
  pdl_wait();
  uint4 x[U][NI][2], w[U][NI][2];
  T *dst[U];
  int near[U];  // the head's node within the run
  bool normed[U], weighted[U];
  // columns of item number it: c1 < 0 for an item of one vector
  const auto columns = [&](int it, bool is_v, int &c0, int &c1) {
    c1 = -1;
    if (is_v) {
      c0 = it * E;
      if ((it + items) * E < dh) c1 = (it + items) * E;
    } else if (it < turning) {
      c0 = it * E;
      if (!INTER) c1 = half + it * E;
    } else {
      c0 = 2 * half + (it - turning) * E;
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int at = run.rem + u * slots + slot;
    dst[u] = nullptr;
    normed[u] = weighted[u] = false;
    near[u] = 0;
    if (run.base + u * slots + slot >= a.heads) continue;
    near[u] = at / run.H;
    const int h = at - near[u] * run.H, node = run.node0 + near[u], b = node / a.r.n;
    const T *src;
    normed[u] = head_of(a.r, node, b, node - b * a.r.n, h, src, dst[u]);
    const T *wt = reinterpret_cast<const T *>(h < a.r.Hq ? a.q_weight : a.k_weight);
    weighted[u] = normed[u] && wt;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int it = lane + i * lanes;
      if (it >= items) continue;
      int c0, c1;
      columns(it, !normed[u], c0, c1);
      x[u][i][0] = __ldcs(reinterpret_cast<const uint4 *>(src + c0));  // coherent: q may be turned in place
      if (c1 >= 0) x[u][i][1] = __ldcs(reinterpret_cast<const uint4 *>(src + c1));
      if (weighted[u]) {
        w[u][i][0] = __ldg(reinterpret_cast<const uint4 *>(wt + c0));
        if (c1 >= 0) w[u][i][1] = __ldg(reinterpret_cast<const uint4 *>(wt + c1));
      }
    }
  }
  run_turns(a.r, run, norm_cs);
  __syncthreads();
  pdl_trigger();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    // the head's sum of squares: every lane of the warp takes part in the exchange
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int it = lane + i * lanes;
      if (!dst[u] || !normed[u] || it >= items) continue;
      float f[E];
      VecTraits<T>::unpack(x[u][i][0], f);
#pragma unroll
      for (int e = 0; e < E; ++e) sum = fmaf(f[e], f[e], sum);
      if (!INTER && it < turning) {
        VecTraits<T>::unpack(x[u][i][1], f);
#pragma unroll
        for (int e = 0; e < E; ++e) sum = fmaf(f[e], f[e], sum);
      }
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (!dst[u]) continue;
    const float r = rsqrtf(sum / static_cast<float>(dh) + a.eps);
    const float2 *cs = norm_cs + near[u] * half;
    const auto scaled = [&](const uint4 &xv, const uint4 &wv, float (&y)[E]) {
      VecTraits<T>::unpack(xv, y);
      float f[E];
      VecTraits<T>::unpack(wv, f);
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = y[e] * r * (weighted[u] ? f[e] + a.offset : 1.f);
    };
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int it = lane + i * lanes;
      if (it >= items) continue;
      int c0, c1;
      columns(it, !normed[u], c0, c1);
      if (normed[u]) {
        float f0[E], f1[E];
        scaled(x[u][i][0], w[u][i][0], f0);
        if (it >= turning) {
          x[u][i][0] = pack_vec<T>(f0);
        } else if constexpr (INTER) {
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const float2 t = cs[c0 / 2 + e / 2];
            f1[e] = f0[e] * t.x - f0[e + 1] * t.y;
            f1[e + 1] = f0[e + 1] * t.x + f0[e] * t.y;
          }
          x[u][i][0] = pack_vec<T>(f1);
        } else {
          scaled(x[u][i][1], w[u][i][1], f1);
          float r0[E], r1[E];
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float2 t = cs[c0 + e];
            r0[e] = f0[e] * t.x - f1[e] * t.y;
            r1[e] = f1[e] * t.x + f0[e] * t.y;
          }
          x[u][i][0] = pack_vec<T>(r0);
          x[u][i][1] = pack_vec<T>(r1);
        }
      }
      *reinterpret_cast<uint4 *>(dst[u] + c0) = x[u][i][0];
      if (c1 >= 0) *reinterpret_cast<uint4 *>(dst[u] + c1) = x[u][i][1];
    }
  }
}

// Any even rot_dim: a warp a head, one pair (or two elements that do not turn) a
// lane and step; the head is read twice, the second time from L1.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_rope_pair_kernel(NormArgs a) {
  constexpr int E = VecTraits<T>::kElems, kWarps = kNormThreads / 32;
  extern __shared__ float2 norm_cs[];
  const HeadRun run(a, kWarps);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  run_turns(a.r, run, norm_cs);
  __syncthreads();
  pdl_trigger();
  if (run.base + warp >= a.heads) return;
  const int at = run.rem + warp, near = at / run.H, h = at - near * run.H, node = run.node0 + near, b = node / a.r.n;
  const T *src;
  T *dst;
  const bool normed = head_of(a.r, node, b, node - b * a.r.n, h, src, dst);
  const T *wt = reinterpret_cast<const T *>(h < a.r.Hq ? a.q_weight : a.k_weight);
  float r = 1.f;
  if (normed) {
    float sum = 0.f;
    for (int c = lane * E; c < a.r.dh; c += 32 * E) {
      float f[E];
      VecTraits<T>::unpack(*reinterpret_cast<const uint4 *>(src + c), f);
#pragma unroll
      for (int e = 0; e < E; ++e) sum = fmaf(f[e], f[e], sum);
    }
    r = rsqrtf(warp_sum(sum) / static_cast<float>(a.r.dh) + a.eps);
  }
  const float2 *cs = norm_cs + near * a.r.half;
  for (int j = lane; j < a.r.dh / 2; j += 32) {
    const bool rot = normed && j < a.r.half;
    const int c0 = rot ? (a.r.interleaved ? 2 * j : j) : 2 * j;
    const int c1 = rot && !a.r.interleaved ? j + a.r.half : c0 + 1;
    const T x0 = src[c0], x1 = src[c1];
    if (!normed) {
      dst[c0] = x0;
      dst[c1] = x1;
      continue;
    }
    float f0 = static_cast<float>(x0) * r, f1 = static_cast<float>(x1) * r;
    if (wt) {
      f0 *= static_cast<float>(wt[c0]) + a.offset;
      f1 *= static_cast<float>(wt[c1]) + a.offset;
    }
    const float2 t = rot ? cs[j] : make_float2(1.f, 0.f);
    dst[c0] = static_cast<T>(rot ? f0 * t.x - f1 * t.y : f0);
    dst[c1] = static_cast<T>(rot ? f1 * t.x + f0 * t.y : f1);
  }
}

// Shared memory for the turns of `count` neighbouring heads.
static size_t turns_bytes(int count, int H, int half) {
  return static_cast<size_t>((count + H - 2) / H + 1) * half * sizeof(float2);
}

template <typename T, bool INTER>
static cudaError_t launch_norm_vec(const NormArgs &a, int items, int H, cudaStream_t st) {
  int log_lanes = 0;
  while (log_lanes < 5 && (1 << log_lanes) < items) ++log_lanes;
  const int ni = (items + (1 << log_lanes) - 1) >> log_lanes, count = (ni == 1 ? 2 : 1) * (kNormThreads >> log_lanes);
  const dim3 grid(static_cast<unsigned>((a.heads + count - 1) / count));
  const size_t smem = turns_bytes(count, H, a.r.half);
  if (ni == 1) return launch_chained(norm_rope_vec_kernel<T, INTER, 1>, grid, dim3(kNormThreads), smem, st, a, log_lanes, items);
  if (ni == 2) return launch_chained(norm_rope_vec_kernel<T, INTER, 2>, grid, dim3(kNormThreads), smem, st, a, log_lanes, items);
  return launch_chained(norm_rope_vec_kernel<T, INTER, 4>, grid, dim3(kNormThreads), smem, st, a, log_lanes, items);
}

template <typename T>
static cudaError_t launch_norm_t(const NormArgs &a, cudaStream_t st) {
  constexpr int E = VecTraits<T>::kElems;
  const int H = a.r.Hq + (a.r.v ? 2 : 1) * a.r.Hkv, half = a.r.half;
  // whole vectors turn: in two halves rot_dim/2, interleaved rot_dim divides into vectors
  if ((a.r.interleaved ? 2 * half : half) % E == 0)
    return a.r.interleaved ? launch_norm_vec<T, true>(a, a.r.dh / E, H, st)
                           : launch_norm_vec<T, false>(a, half / E + (a.r.dh - 2 * half) / E, H, st);
  constexpr int kWarps = kNormThreads / 32;
  const dim3 grid(static_cast<unsigned>((a.heads + kWarps - 1) / kWarps));
  return launch_chained(norm_rope_pair_kernel<T>, grid, dim3(kNormThreads), turns_bytes(kWarps, H, half), st, a);
}

cudaError_t launch_qk_norm_rope(const void *q, const void *k, const void *v, int dtype, int B, int n, int Hq, int Hkv,
                                int dh, int64_t ld_q, int64_t ld_k, int64_t ld_v, const void *q_weight,
                                const void *k_weight, float weight_offset, float eps, const double *inv_freq,
                                int rot_dim, int interleaved, float factor, const int32_t *pos_base,
                                const int32_t *pos_off, int shift, void *q_out, void *k_tree, void *v_tree,
                                cudaStream_t st) {
  NormArgs a = {{q, k, v, q_out, k_tree, v_tree, B, n, Hq, Hkv, dh, rot_dim / 2, interleaved, shift, ld_q, ld_k, ld_v,
                 inv_freq, pos_base, pos_off, factor},
                q_weight, k_weight, eps, weight_offset,
                static_cast<int64_t>(B) * n * (Hq + static_cast<int64_t>(v ? 2 : 1) * Hkv)};
  return dtype == EAGLE_BF16 ? launch_norm_t<__nv_bfloat16>(a, st) : launch_norm_t<float>(a, st);
}

}  // namespace eagle
