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
// tree.  A group of lanes holds a head's 16-byte vectors in registers between the sum
// and the rotation, so the head is read once.  A thread stays with one node and takes
// up to four of its heads, their vectors on their way together while the node's turns
// and the weights are made ready in shared memory; the block is as large as the
// node's heads need.
// Measured, on the device: 8191 nodes of 40 + 40 heads of 128, a quarter turned, f32,
// 184 us (1.0 GB, 82 % of the copy rate); 64 x 61 nodes of 64 + 8 heads of 64, bf16, 21.3
// us (80 MB, 56 %; rope.cu without the norm 17.6: four tenths more instructions, and the
// barrier before the turns is waited at twice as long); 61 nodes of 32 + 32 heads of 128
// 3.5 us; 8191 nodes of 64 + 8 heads of 128, all of it turned in two halves, bf16, 78 us
// (336 MB, 65 %), of 32 + 32 heads 95 us (63 %).  The arithmetic in packed pairs (f32x2): 20.7 and 3.3 us, but 191 in f32.
#include "rope.cuh"

namespace eagle {

constexpr int kNormThreads = 256;

struct NormArgs {
  RopeArgs r;
  const void *q_weight, *k_weight;  // [dh] of the same type, or NULL: ones
  float eps, offset, mean;          // mean: 1 / dh
  int nodes, heads;                 // B * n; of a node: Hq + Hkv, and Hkv of v
};

// cos and sin of `count` neighbouring nodes (node k's pair j at cs[k * half + j]).  A
// thread keeps its pair: the float64 operations are once a pair and CTA.
__device__ __forceinline__ void run_turns(const NormArgs &a, int node0, int count, float2 *cs) {
  for (int j = threadIdx.x; j < a.r.half; j += blockDim.x) {
    const uint64_t inc = turn_step(a.r.inv_freq[j]);
    for (int k = 0; k < count && node0 + k < a.nodes; ++k) {
      const int node = node0 + k, b = node / a.r.n;
      cs[k * a.r.half + j] = turn_at(inc, position_of(a.r, node, b, node - b * a.r.n), a.r.factor);
    }
  }
}

// 16-byte vectors, `lanes` threads a head, NI items a lane (an item as in rope.cu:
// two vectors half of rot_dim apart, one vector of whole pairs, or one that does
// not turn), U heads a thread with their loads in flight together.  blockIdx.x: nb
// nodes, each with `per_node` threads; blockIdx.y: a run of U * per_node / lanes heads.
template <typename T, bool INTER, int NI, int U>
__global__ void __launch_bounds__(512) norm_rope_vec_kernel(NormArgs a, int log_lanes, int items, int per_node, int nb) {
  constexpr int E = VecTraits<T>::kElems;
  extern __shared__ float4 norm_smem[];
  float *ws = reinterpret_cast<float *>(norm_smem);  // q's weights, then k's
  const int dh = a.r.dh, half = a.r.half, Hq = a.r.Hq, Hkv = a.r.Hkv;
  float2 *turns = reinterpret_cast<float2 *>(ws + 2 * dh);
  const int lanes = 1 << log_lanes, slots = per_node >> log_lanes;
  const int near = threadIdx.x / per_node, slot = (threadIdx.x - near * per_node) >> log_lanes, lane = threadIdx.x & (lanes - 1);
  const int node = blockIdx.x * nb + near, h0 = blockIdx.y * U * slots + slot;
  // heads of this thread: none in the last warp's spare lanes and the last CTA's spare nodes
  const int heads = near < nb && node < a.nodes ? a.heads : 0;
  // An item's columns from c[k] and, where it turns in two halves, c[k] + half; v is
  // copied in the same pieces.
  int c[NI];
  bool live[NI], turns_here[NI];
#pragma unroll
  for (int k = 0; k < NI; ++k) {
    const int it = lane + k * lanes, turning = INTER ? 2 * half / E : half / E;
    live[k] = it < items;
    turns_here[k] = it < turning;
    c[k] = INTER || it < turning ? it * E : 2 * half + (it - turning) * E;
  }
  pdl_wait();
  const int b = node / a.r.n, i = node - b * a.r.n;
  const T *src_q = reinterpret_cast<const T *>(a.r.q) + node * a.r.ld_q, *src_k = reinterpret_cast<const T *>(a.r.k) + node * a.r.ld_k,
          *src_v = reinterpret_cast<const T *>(a.r.v) + node * a.r.ld_v;
  const int64_t tree = (static_cast<int64_t>(b) * Hkv * a.r.n + i) * dh, per_head = static_cast<int64_t>(a.r.n) * dh;
  T *dst_q = reinterpret_cast<T *>(a.r.q_out) + static_cast<int64_t>(node) * Hq * dh, *dst_k = reinterpret_cast<T *>(a.r.k_tree) + tree,
    *dst_v = reinterpret_cast<T *>(a.r.v_tree) + tree;
  uint4 x[U][NI][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * slots;
    if (h >= heads) continue;
    const T *src = h < Hq ? src_q + h * dh : h < Hq + Hkv ? src_k + (h - Hq) * dh : src_v + (h - Hq - Hkv) * dh;
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      if (!live[k]) continue;
      x[u][k][0] = __ldcs(reinterpret_cast<const uint4 *>(src + c[k]));  // coherent: q may be turned in place
      if (!INTER && turns_here[k]) x[u][k][1] = __ldcs(reinterpret_cast<const uint4 *>(src + c[k] + half));
    }
  }
  for (int e = threadIdx.x; e < 2 * dh; e += blockDim.x) {
    const T *wt = reinterpret_cast<const T *>(e < dh ? a.q_weight : a.k_weight);
    ws[e] = wt ? static_cast<float>(wt[e < dh ? e : e - dh]) + a.offset : 1.f;
  }
  run_turns(a, blockIdx.x * nb, nb, turns);
  __syncthreads();
  pdl_trigger();
  const float2 *cs = turns + near * half;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * slots;
    const bool normed = h < Hq + Hkv;
    // the head's sum of squares: every lane of the warp takes part in the exchange
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      if (!live[k] || h >= heads) continue;
      float f[E];
      VecTraits<T>::unpack(x[u][k][0], f);
#pragma unroll
      for (int e = 0; e < E; ++e) sum = fmaf(f[e], f[e], sum);
      if (!INTER && turns_here[k]) {
        VecTraits<T>::unpack(x[u][k][1], f);
#pragma unroll
        for (int e = 0; e < E; ++e) sum = fmaf(f[e], f[e], sum);
      }
    }
    for (int o = lanes >> 1; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (h >= heads) continue;
    const float r = rsqrtf(fmaf(sum, a.mean, a.eps));
    const float *w = ws + (h < Hq ? 0 : dh);
    T *dst = h < Hq ? dst_q + h * dh : (normed ? dst_k + (h - Hq) * per_head : dst_v + (h - Hq - Hkv) * per_head);
    const auto scaled = [&](const uint4 &xv, int col, float (&y)[E]) {
      VecTraits<T>::unpack(xv, y);
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        const float4 f = *reinterpret_cast<const float4 *>(w + col + e);
        y[e] *= r * f.x; y[e + 1] *= r * f.y; y[e + 2] *= r * f.z; y[e + 3] *= r * f.w;
      }
    };
#pragma unroll
    for (int k = 0; k < NI; ++k) {
      if (!live[k]) continue;
      if (normed) {
        float f0[E], f1[E];
        scaled(x[u][k][0], c[k], f0);
        if (!turns_here[k]) {
          x[u][k][0] = pack_vec<T>(f0);
        } else if constexpr (INTER) {
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const float2 t = cs[c[k] / 2 + e / 2];
            f1[e] = f0[e] * t.x - f0[e + 1] * t.y;
            f1[e + 1] = f0[e + 1] * t.x + f0[e] * t.y;
          }
          x[u][k][0] = pack_vec<T>(f1);
        } else {
          scaled(x[u][k][1], c[k] + half, f1);
          float r0[E], r1[E];
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float2 t = cs[c[k] + e];
            r0[e] = f0[e] * t.x - f1[e] * t.y;
            r1[e] = f1[e] * t.x + f0[e] * t.y;
          }
          x[u][k][0] = pack_vec<T>(r0);
          x[u][k][1] = pack_vec<T>(r1);
        }
      }
      *reinterpret_cast<uint4 *>(dst + c[k]) = x[u][k][0];
      if (!INTER && turns_here[k]) *reinterpret_cast<uint4 *>(dst + c[k] + half) = x[u][k][1];
    }
  }
}

// Any even rot_dim: a warp a head, one pair (or two elements that do not turn) a
// lane and step; the head is read twice, the second time from L1.  Measured, on the
// device, 20 columns turned, bf16: 8191 nodes of 64 + 8 heads of 128 192 us (26 % of the
// copy rate; whole vectors 78), 64 x 61 nodes of 64 + 8 heads of 64 75 us, 61 nodes of 32
// + 32 heads 4.0 us: element-wise accesses, a warp's 64 bytes a request.
template <typename T>
__global__ void __launch_bounds__(kNormThreads) norm_rope_pair_kernel(NormArgs a) {
  constexpr int E = VecTraits<T>::kElems, kWarps = kNormThreads / 32;
  extern __shared__ float4 norm_smem[];
  float2 *cs = reinterpret_cast<float2 *>(norm_smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int node = blockIdx.x, b = node / a.r.n, h = blockIdx.y * kWarps + warp;
  pdl_wait();
  run_turns(a, node, 1, cs);
  __syncthreads();
  pdl_trigger();
  if (h >= a.heads) return;
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

template <typename T, bool INTER, int NI, int U>
static cudaError_t launch_norm_v(const NormArgs &a, int log_lanes, int items, int most_threads, cudaStream_t st) {
  // a node's heads over runs (blockIdx.y) of equal size, several nodes to a CTA where
  // one has fewer than 128 threads to do
  const int lanes = 1 << log_lanes, runs = (a.heads * lanes + U * most_threads - 1) / (U * most_threads);
  const int slots = (a.heads + U * runs - 1) / (U * runs), per_node = slots * lanes;
  const int nb = per_node >= 128 ? 1 : 128 / per_node;
  const int threads = (nb * per_node + 31) / 32 * 32;
  const size_t smem = 2 * a.r.dh * sizeof(float) + static_cast<size_t>(nb) * a.r.half * sizeof(float2);
  const dim3 grid((a.nodes + nb - 1) / nb, (a.heads + U * slots - 1) / (U * slots));
  return launch_chained(norm_rope_vec_kernel<T, INTER, NI, U>, grid, dim3(threads), smem, st, a, log_lanes, items, per_node, nb);
}

template <typename T, bool INTER>
static cudaError_t launch_norm_vec(const NormArgs &a, int items, int num_sms, cudaStream_t st) {
  int log_lanes = 0;
  while (log_lanes < 5 && (1 << log_lanes) < items) ++log_lanes;
  const int ni = (items + (1 << log_lanes) - 1) >> log_lanes;
  if (ni > 2) return launch_norm_v<T, INTER, 4, 1>(a, log_lanes, items, 512, st);
  if (ni > 1) return launch_norm_v<T, INTER, 2, 1>(a, log_lanes, items, 512, st);
  // several heads a thread where that leaves each SM four warps' worth of threads or
  // more, else one and smaller blocks: latency counts
  const int64_t work = static_cast<int64_t>(a.nodes) * a.heads << log_lanes;
  constexpr int MANY = INTER ? 4 : 2;  // (f32, 120 heads of 128: 249, 208, 186, 183 us with one to four of one vector)
  return work >= 512ll * MANY * num_sms ? launch_norm_v<T, INTER, 1, MANY>(a, log_lanes, items, INTER ? 256 : 512, st)
                                        : launch_norm_v<T, INTER, 1, 1>(a, log_lanes, items, 256, st);
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
  return launch_chained(norm_rope_pair_kernel<T>, dim3(a.nodes, (a.heads + kWarps - 1) / kWarps), dim3(kNormThreads),
                        half * sizeof(float2), st, a);
}

cudaError_t launch_qk_norm_rope(const void *q, const void *k, const void *v, int dtype, int B, int n, int Hq, int Hkv,
                                int dh, int64_t ld_q, int64_t ld_k, int64_t ld_v, const void *q_weight,
                                const void *k_weight, float weight_offset, float eps, const double *inv_freq,
                                int rot_dim, int interleaved, float factor, const int32_t *pos_base,
                                const int32_t *pos_off, int shift, void *q_out, void *k_tree, void *v_tree, int num_sms,
                                cudaStream_t st) {
  const NormArgs a = {{q, k, v, q_out, k_tree, v_tree, B, n, Hq, Hkv, dh, rot_dim / 2, interleaved, shift, ld_q, ld_k, ld_v,
                       inv_freq, pos_base, pos_off, factor},
                      q_weight, k_weight, eps, weight_offset, 1.f / static_cast<float>(dh), B * n,
                      Hq + (v ? 2 : 1) * Hkv};
  return dtype == EAGLE_BF16 ? launch_norm_t<__nv_bfloat16>(a, num_sms, st) : launch_norm_t<float>(a, num_sms, st);
}

}  // namespace eagle
