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
// their nodes: no place for a head stays empty.  A group of lanes holds a head's
// 16-byte vectors in registers between the sum and the rotation, so the head is
// read once; a thread has up to four heads' vectors on their way while the turns of
// the run's nodes and the weights are made ready in shared memory.
#include "rope.cuh"

namespace eagle {

constexpr int kNormThreads = 256;

// x / d for x < 2^31 by a product: s = ceil(log2 d), m = floor(2^32 (2^s - d) / d) + 1.
struct Divisor {
  uint32_t d, m;
  int s;
  explicit Divisor(uint32_t of) : d(of), s(0) {
    while ((1ull << s) < d) ++s;
    m = static_cast<uint32_t>(((1ull << 32) * ((1ull << s) - d)) / d + 1);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t x) const { return (__umulhi(m, x) + x) >> s; }
};

struct NormArgs {
  RopeArgs r;
  const void *q_weight, *k_weight;  // [dh] of the same type, or NULL: ones
  float eps, offset, mean;          // mean: 1 / dh
  uint32_t heads;                   // B * n * (Hq + Hkv, and Hkv of v), below 2^31
  Divisor per_node, per_seq;        // heads of a node, nodes of a sequence
};

// The run of heads a CTA takes: its first node, the first head's place in that
// node, and the nodes it touches.
struct HeadRun {
  uint32_t base, node0, rem, nodes;
  __device__ __forceinline__ HeadRun(const NormArgs &a, uint32_t count) {
    base = blockIdx.x * count;
    node0 = a.per_node(base);
    rem = base - node0 * a.per_node.d;
    nodes = a.per_node(min(base + count, a.heads) - 1) - node0 + 1;
  }
};
// cos and sin of the run's nodes (node k's pair j at cs[k * half + j]).  A thread
// keeps its pair: the float64 operations are once a pair and CTA.
__device__ __forceinline__ void run_turns(const NormArgs &a, const HeadRun &run, float2 *cs) {
  for (int j = threadIdx.x; j < a.r.half; j += kNormThreads) {
    const uint64_t inc = turn_step(a.r.inv_freq[j]);
    for (uint32_t k = 0; k < run.nodes; ++k) {
      const uint32_t node = run.node0 + k, b = a.per_seq(node);
      cs[k * a.r.half + j] = turn_at(inc, position_of(a.r, node, b, node - b * a.per_seq.d), a.r.factor);
    }
  }
}

// 16-byte vectors, `lanes` threads a head, NI items a lane (an item as in rope.cu:
// two vectors half of rot_dim apart, one vector of whole pairs, or one that does
// not turn), U heads a thread with their loads in flight together.
template <typename T, bool INTER, int NI, int U>
__global__ void __launch_bounds__(kNormThreads) norm_rope_vec_kernel(NormArgs a, int log_lanes, int items) {
  constexpr int E = VecTraits<T>::kElems;
  extern __shared__ float4 norm_smem[];
  float *ws = reinterpret_cast<float *>(norm_smem);  // q's weights, then k's
  const int dh = a.r.dh, half = a.r.half;
  float2 *turns = reinterpret_cast<float2 *>(ws + 2 * dh);
  const int lanes = 1 << log_lanes, slots = kNormThreads >> log_lanes;
  const int lane = threadIdx.x & (lanes - 1), slot = threadIdx.x >> log_lanes;
  const HeadRun run(a, U * slots);
  const int turning = INTER ? 2 * half / E : half / E;  // items that turn
  pdl_wait();
  uint4 x[U][NI][2];
  T *dst[U];
  uint32_t near[U];  // the head's node within the run
  bool normed[U], is_q[U];
  // columns of item number it: c1 < 0 for an item of one vector
  const auto columns = [&](int it, bool is_v, int &c0, int &c1) {
    c1 = -1;
    if (is_v) {
      c0 = it * E;
      if (!INTER && (it + items) * E < dh) c1 = (it + items) * E;  // interleaved, the items are the vectors
    } else if (it < turning) {
      c0 = it * E;
      if (!INTER) c1 = half + it * E;
    } else {
      c0 = 2 * half + (it - turning) * E;
    }
  };
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t at = run.rem + u * slots + slot;
    dst[u] = nullptr;
    normed[u] = is_q[u] = false;
    near[u] = 0;
    if (run.base + u * slots + slot >= a.heads) continue;
    near[u] = a.per_node(at);
    const int h = at - near[u] * a.per_node.d, node = run.node0 + near[u], b = a.per_seq(node);
    const T *src;
    normed[u] = head_of(a.r, node, b, node - b * a.r.n, h, src, dst[u]);
    is_q[u] = h < a.r.Hq;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int it = lane + i * lanes;
      if (it >= items) continue;
      int c0, c1;
      columns(it, !normed[u], c0, c1);
      x[u][i][0] = __ldcs(reinterpret_cast<const uint4 *>(src + c0));  // coherent: q may be turned in place
      if (!INTER && c1 >= 0) x[u][i][1] = __ldcs(reinterpret_cast<const uint4 *>(src + c1));
    }
  }
  for (int c = threadIdx.x; c < 2 * dh; c += kNormThreads) {
    const T *wt = reinterpret_cast<const T *>(c < dh ? a.q_weight : a.k_weight);
    ws[c] = wt ? static_cast<float>(wt[c < dh ? c : c - dh]) + a.offset : 1.f;
  }
  run_turns(a, run, turns);
  __syncthreads();
  pdl_trigger();
#pragma unroll
  for (int u = 0; u < U; ++u) {
    // the head's sum of squares: every lane of the warp takes part in the exchange
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int it = lane + i * lanes;
      if (!normed[u] || it >= items) continue;
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
    const float r = rsqrtf(fmaf(sum, a.mean, a.eps));
    const float2 *cs = turns + near[u] * half;
    const float *w = ws + (is_q[u] ? 0 : dh);
    const auto scaled = [&](const uint4 &xv, int c, float (&y)[E]) {
      VecTraits<T>::unpack(xv, y);
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(w + c + e);
        y[e] *= r * f.x; y[e + 1] *= r * f.y; y[e + 2] *= r * f.z; y[e + 3] *= r * f.w;
      }
    };
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int it = lane + i * lanes;
      if (it >= items) continue;
      int c0, c1;
      columns(it, !normed[u], c0, c1);
      if (normed[u]) {
        float f0[E], f1[E];
        scaled(x[u][i][0], c0, f0);
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
          scaled(x[u][i][1], c1, f1);
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
      if (!INTER && c1 >= 0) *reinterpret_cast<uint4 *>(dst[u] + c1) = x[u][i][1];
    }
  }
}

// Any even rot_dim: a warp a head, one pair (or two elements that do not turn) a
// lane and step; the head is read twice, the second time from L1.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_rope_pair_kernel(NormArgs a) {
  constexpr int E = VecTraits<T>::kElems, kWarps = kNormThreads / 32;
  extern __shared__ float4 norm_smem[];
  float2 *turns = reinterpret_cast<float2 *>(norm_smem);
  const HeadRun run(a, kWarps);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  run_turns(a, run, turns);
  __syncthreads();
  pdl_trigger();
  if (run.base + warp >= a.heads) return;
  const uint32_t at = run.rem + warp, near = a.per_node(at);
  const int h = at - near * a.per_node.d, node = run.node0 + near, b = a.per_seq(node);
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
    r = rsqrtf(fmaf(warp_sum(sum), a.mean, a.eps));
  }
  const float2 *cs = turns + near * a.r.half;
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
    const float w0 = wt ? static_cast<float>(wt[c0]) + a.offset : 1.f, w1 = wt ? static_cast<float>(wt[c1]) + a.offset : 1.f;
    const float f0 = static_cast<float>(x0) * (r * w0), f1 = static_cast<float>(x1) * (r * w1);
    const float2 t = rot ? cs[j] : make_float2(1.f, 0.f);
    dst[c0] = static_cast<T>(rot ? f0 * t.x - f1 * t.y : f0);
    dst[c1] = static_cast<T>(rot ? f1 * t.x + f0 * t.y : f1);
  }
}

// Shared memory for the turns of `count` neighbouring heads.
static size_t turns_bytes(int count, int H, int half) {
  return static_cast<size_t>((count + H - 2) / H + 1) * half * sizeof(float2);
}

template <typename T, bool INTER, int NI, int U>
static cudaError_t launch_norm_v(const NormArgs &a, int log_lanes, int items, cudaStream_t st) {
  const int count = U * (kNormThreads >> log_lanes);
  const size_t smem = 2 * a.r.dh * sizeof(float) + turns_bytes(count, a.per_node.d, a.r.half);
  return launch_chained(norm_rope_vec_kernel<T, INTER, NI, U>, dim3((a.heads + count - 1) / count), dim3(kNormThreads), smem, st,
                        a, log_lanes, items);
}

template <typename T, bool INTER>
static cudaError_t launch_norm_vec(const NormArgs &a, int items, int num_sms, cudaStream_t st) {
  int log_lanes = 0;
  while (log_lanes < 5 && (1 << log_lanes) < items) ++log_lanes;
  const int ni = (items + (1 << log_lanes) - 1) >> log_lanes;
  if (ni > 2) return launch_norm_v<T, INTER, 4, 1>(a, log_lanes, items, st);
  if (ni > 1) return launch_norm_v<T, INTER, 2, 1>(a, log_lanes, items, st);
  // four heads a thread where that leaves each SM two CTAs or more, else one
  const uint32_t slots = kNormThreads >> log_lanes;
  return a.heads >= 8u * slots * num_sms ? launch_norm_v<T, INTER, 1, 4>(a, log_lanes, items, st)
                                         : launch_norm_v<T, INTER, 1, 1>(a, log_lanes, items, st);
}

template <typename T>
static cudaError_t launch_norm_t(const NormArgs &a, int num_sms, cudaStream_t st) {
  constexpr int E = VecTraits<T>::kElems;
  const int half = a.r.half;
  // whole vectors turn: in two halves rot_dim/2, interleaved rot_dim divides into vectors
  if ((a.r.interleaved ? 2 * half : half) % E == 0)
    return a.r.interleaved ? launch_norm_vec<T, true>(a, a.r.dh / E, num_sms, st)
                           : launch_norm_vec<T, false>(a, half / E + (a.r.dh - 2 * half) / E, num_sms, st);
  constexpr int kWarps = kNormThreads / 32;
  return launch_chained(norm_rope_pair_kernel<T>, dim3((a.heads + kWarps - 1) / kWarps), dim3(kNormThreads),
                        turns_bytes(kWarps, a.per_node.d, half), st, a);
}

cudaError_t launch_qk_norm_rope(const void *q, const void *k, const void *v, int dtype, int B, int n, int Hq, int Hkv,
                                int dh, int64_t ld_q, int64_t ld_k, int64_t ld_v, const void *q_weight,
                                const void *k_weight, float weight_offset, float eps, const double *inv_freq,
                                int rot_dim, int interleaved, float factor, const int32_t *pos_base,
                                const int32_t *pos_off, int shift, void *q_out, void *k_tree, void *v_tree, int num_sms,
                                cudaStream_t st) {
  const uint32_t H = Hq + (v ? 2 : 1) * Hkv;
  const NormArgs a = {{q, k, v, q_out, k_tree, v_tree, B, n, Hq, Hkv, dh, rot_dim / 2, interleaved, shift, ld_q, ld_k, ld_v,
                       inv_freq, pos_base, pos_off, factor},
                      q_weight, k_weight, eps, weight_offset, 1.f / static_cast<float>(dh),
                      static_cast<uint32_t>(B) * n * H, Divisor(H), Divisor(n)};
  return dtype == EAGLE_BF16 ? launch_norm_t<__nv_bfloat16>(a, num_sms, st) : launch_norm_t<float>(a, num_sms, st);
}

}  // namespace eagle
