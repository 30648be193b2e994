// Rotary positions of q and k, and v, into the tree attention's layouts.
//
// Pair j of a head at position p turns by the angle p * f_j.  The angle is
// wanted modulo a turn for positions up to 2^31: f_j / 2pi is taken as a 64-bit
// fixed-point fraction of a turn, and p * that, wrapping, reduces it without
// another rounding; its top 32 bits are the turns that sincospi gets (a float's 24
// bits of them).  The angle is off by at most 2^-25 half turns, 1e-7, and what the
// rounding of f_j / 2pi in float64 grows to, p f_j 2^-52 (the product's half step
// and the constant's): 5e-7 at 2^31.  That product and its fraction, a handful of
// float64 operations, are done once a pair and CTA, the float64 reduction of p f_j
// itself never.
//
// What bounds it: HBM (each element read once and written once), and latency
// for one tree.  A CTA takes one node and a run of its heads; the node's cos and
// sin are computed once per CTA into shared memory, while the heads' 16-byte
// vectors are on their way.  Measured: 8191 nodes of 120 heads of 128 in f32
// 175 us (5.8 TB/s, 86 % of a copy's rate); 3904 nodes of 80 heads of 64 in
// bf16 16.9 us (4.7 TB/s, 71 %); 61 nodes of 96 heads of 128 3.3 us.
#include <math.h>

#include "common.cuh"

namespace eagle {

constexpr int kRopeThreads = 256;

struct RopeArgs {
  const void *q, *k, *v;
  void *q_out, *k_tree, *v_tree;
  int B, n, Hq, Hkv, dh, half, interleaved, shift;
  int64_t ld_q, ld_k, ld_v;
  const double *inv_freq;
  const int32_t *pos_base, *pos_off;
  float factor;
};

// cos and sin (times the factor) of the node's angles into shared memory.
__device__ __forceinline__ void node_turns(const RopeArgs &a, int pos, float2 *cs) {
  for (int j = threadIdx.x; j < a.half; j += kRopeThreads) {
    double t = a.inv_freq[j] * 0.15915494309189533577;  // turns per position
    t -= rint(t);
    const uint64_t inc = static_cast<uint64_t>(static_cast<int64_t>(t * 18446744073709551616.0));
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * inc;
    float sn, c;
    sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &sn, &c);
    cs[j] = make_float2(c * a.factor, sn * a.factor);
  }
}
__device__ __forceinline__ int position_of(const RopeArgs &a, int node, int b, int i) {
  return (a.pos_base ? a.pos_base[b] : 0) + (a.pos_off ? a.pos_off[node] : i) + a.shift;
}
// Head h of a node: where it is read and written, and whether it turns.
template <typename T>
__device__ __forceinline__ bool head_of(const RopeArgs &a, int node, int b, int i, int h, const T *&src, T *&dst) {
  if (h < a.Hq) {
    src = reinterpret_cast<const T *>(a.q) + node * a.ld_q + static_cast<int64_t>(h) * a.dh;
    dst = reinterpret_cast<T *>(a.q_out) + (static_cast<int64_t>(node) * a.Hq + h) * a.dh;
    return true;
  }
  const bool is_k = h < a.Hq + a.Hkv;
  const int g = h - a.Hq - (is_k ? 0 : a.Hkv);
  src = reinterpret_cast<const T *>(is_k ? a.k : a.v) + node * (is_k ? a.ld_k : a.ld_v) + static_cast<int64_t>(g) * a.dh;
  dst = reinterpret_cast<T *>(is_k ? a.k_tree : a.v_tree) + ((static_cast<int64_t>(b) * a.Hkv + g) * a.n + i) * a.dh;
  return is_k;
}

template <typename T> __device__ __forceinline__ uint4 pack_vec(const float (&x)[VecTraits<T>::kElems]);
template <> __device__ __forceinline__ uint4 pack_vec<float>(const float (&x)[4]) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}
template <> __device__ __forceinline__ uint4 pack_vec<__nv_bfloat16>(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16-byte vectors.  An item of a head is what one thread turns: two vectors half
// of rot_dim apart, or (interleaved) one vector of whole pairs, or one vector
// that is copied; a head of v is copied up to two vectors an item.  `lanes` (a
// power of two) threads share a head, kRopeItems heads' items are requested
// before the turns are computed, so their latencies overlap.
constexpr int kRopeItems = 2;

template <typename T, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_vec_kernel(RopeArgs a, int log_lanes, int items) {
  constexpr int E = VecTraits<T>::kElems;
  __shared__ float2 cs[256];
  const int node = blockIdx.x, b = node / a.n, i = node % a.n;
  const int it = threadIdx.x & ((1 << log_lanes) - 1);
  const int H = a.Hq + (a.v ? 2 : 1) * a.Hkv;
  const int step = kRopeThreads >> log_lanes, h0 = blockIdx.y * kRopeItems * step + (threadIdx.x >> log_lanes);
  pdl_wait();
  const int pos = position_of(a, node, b, i);
  const int turning = INTER ? 2 * a.half / E : a.half / E;  // items that turn
  uint4 x[kRopeItems][2];
  T *dst[kRopeItems];
  int c0[kRopeItems], c1[kRopeItems];  // the item's columns; c1 < 0: one vector
  bool turn[kRopeItems];
#pragma unroll
  for (int u = 0; u < kRopeItems; ++u) {
    const int h = h0 + u * step;
    dst[u] = nullptr;
    if (h >= H || it >= items) continue;
    const T *src;
    turn[u] = head_of(a, node, b, i, h, src, dst[u]);
    c1[u] = -1;
    if (!turn[u]) {
      c0[u] = it * E;
      if ((it + items) * E < a.dh) c1[u] = (it + items) * E;
    } else if (it < turning) {
      c0[u] = it * E;
      if (!INTER) c1[u] = a.half + it * E;
    } else {
      c0[u] = 2 * a.half + (it - turning) * E;
      turn[u] = false;
    }
    x[u][0] = __ldcs(reinterpret_cast<const uint4 *>(src + c0[u]));  // coherent: q may be turned in place
    if (c1[u] >= 0) x[u][1] = __ldcs(reinterpret_cast<const uint4 *>(src + c1[u]));
  }
  node_turns(a, pos, cs);
  __syncthreads();
  pdl_trigger();
#pragma unroll
  for (int u = 0; u < kRopeItems; ++u) {
    if (!dst[u]) continue;
    if (turn[u]) {
      float f0[E], f1[E];
      VecTraits<T>::unpack(x[u][0], f0);
      if constexpr (INTER) {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 w = cs[c0[u] / 2 + e / 2];
          f1[e] = f0[e] * w.x - f0[e + 1] * w.y;
          f1[e + 1] = f0[e + 1] * w.x + f0[e] * w.y;
        }
        x[u][0] = pack_vec<T>(f1);
      } else {
        VecTraits<T>::unpack(x[u][1], f1);
        float r0[E], r1[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float2 w = cs[c0[u] + e];
          r0[e] = f0[e] * w.x - f1[e] * w.y;
          r1[e] = f1[e] * w.x + f0[e] * w.y;
        }
        x[u][0] = pack_vec<T>(r0);
        x[u][1] = pack_vec<T>(r1);
      }
    }
    *reinterpret_cast<uint4 *>(dst[u] + c0[u]) = x[u][0];
    if (c1[u] >= 0) *reinterpret_cast<uint4 *>(dst[u] + c1[u]) = x[u][1];
  }
}

// Any even rot_dim: one pair (or two copied elements) a thread step.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_pair_kernel(RopeArgs a) {
  __shared__ float2 cs[256];
  const int node = blockIdx.x, b = node / a.n, i = node % a.n;
  pdl_wait();
  node_turns(a, position_of(a, node, b, i), cs);
  __syncthreads();
  pdl_trigger();
  const int H = a.Hq + (a.v ? 2 : 1) * a.Hkv, pairs = a.dh / 2;
  for (int idx = blockIdx.y * kRopeThreads + threadIdx.x; idx < H * pairs; idx += gridDim.y * kRopeThreads) {
    const int h = idx / pairs, j = idx % pairs;
    const T *src;
    T *dst;
    const bool turn = head_of(a, node, b, i, h, src, dst);
    const bool rot = turn && j < a.half;
    const int c0 = rot ? (a.interleaved ? 2 * j : j) : 2 * j;
    const int c1 = rot && !a.interleaved ? j + a.half : c0 + 1;
    const T x0 = src[c0], x1 = src[c1];
    if (rot) {
      const float2 w = cs[j];
      const float f0 = static_cast<float>(x0), f1 = static_cast<float>(x1);
      dst[c0] = static_cast<T>(f0 * w.x - f1 * w.y);
      dst[c1] = static_cast<T>(f1 * w.x + f0 * w.y);
    } else {
      dst[c0] = x0;
      dst[c1] = x1;
    }
  }
}

template <typename T>
static cudaError_t launch_rope_t(const RopeArgs &a, cudaStream_t st) {
  constexpr int E = VecTraits<T>::kElems;
  const int H = a.Hq + (a.v ? 2 : 1) * a.Hkv;
  // whole vectors turn: in two halves rot_dim/2, interleaved rot_dim divides into vectors
  if ((a.interleaved ? 2 * a.half : a.half) % E == 0) {
    const int items = a.interleaved ? a.dh / E : a.half / E + (a.dh - 2 * a.half) / E;
    int log_lanes = 0;
    while ((1 << log_lanes) < items) ++log_lanes;
    const int heads = kRopeItems * (kRopeThreads >> log_lanes);  // a CTA
    const dim3 grid(a.B * a.n, (H + heads - 1) / heads);
    return a.interleaved ? launch_chained(rope_vec_kernel<T, true>, grid, dim3(kRopeThreads), 0, st, a, log_lanes, items)
                         : launch_chained(rope_vec_kernel<T, false>, grid, dim3(kRopeThreads), 0, st, a, log_lanes, items);
  }
  const dim3 grid(a.B * a.n, (H * a.dh / 2 + kRopeThreads * 8 - 1) / (kRopeThreads * 8));
  return launch_chained(rope_pair_kernel<T>, grid, dim3(kRopeThreads), 0, st, a);
}

cudaError_t launch_rope(const void *q, const void *k, const void *v, int dtype, int B, int n, int Hq, int Hkv, int dh,
                        int64_t ld_q, int64_t ld_k, int64_t ld_v, const double *inv_freq, int rot_dim,
                        int interleaved, float factor, const int32_t *pos_base, const int32_t *pos_off, int shift,
                        void *q_out, void *k_tree, void *v_tree, cudaStream_t st) {
  RopeArgs a = {q, k, v, q_out, k_tree, v_tree, B, n, Hq, Hkv, dh, rot_dim / 2, interleaved, shift,
                ld_q, ld_k, ld_v, inv_freq, pos_base, pos_off, factor};
  return dtype == EAGLE_BF16 ? launch_rope_t<__nv_bfloat16>(a, st) : launch_rope_t<float>(a, st);
}

// Host: the frequencies.
void rope_freqs(int rot_dim, double theta, int kind, double stretch, int orig_len, double low, double high,
                double *inv_freq, float *factor) {
  const double two_pi = 6.283185307179586476925;
  const int half = rot_dim / 2;
  // the pair index (not rounded) that makes r turns over the trained context
  auto index_of = [&](double r) { return rot_dim * log(orig_len / (r * two_pi)) / (2.0 * log(theta)); };
  const double lo = kind == EAGLE_ROPE_YARN ? fmax(floor(index_of(high)), 0.0) : 0.0;
  const double hi = kind == EAGLE_ROPE_YARN ? fmin(ceil(index_of(low)), rot_dim - 1.0) : 0.0;
  for (int j = 0; j < half; ++j) {
    const double f = pow(theta, -2.0 * j / rot_dim);
    double keep = 1.0;  // share of the unstretched frequency
    if (kind == EAGLE_ROPE_LINEAR) keep = 0.0;
    if (kind == EAGLE_ROPE_BANDS) keep = (orig_len * f / two_pi - low) / (high - low);
    if (kind == EAGLE_ROPE_YARN) keep = 1.0 - (j - lo) / fmax(hi - lo, 1e-3);
    keep = fmin(fmax(keep, 0.0), 1.0);
    inv_freq[j] = f * keep + f / stretch * (1.0 - keep);
    if (kind == EAGLE_ROPE_PLAIN) inv_freq[j] = f;
  }
  if (factor) *factor = kind == EAGLE_ROPE_YARN ? static_cast<float>(0.1 * log(stretch) + 1.0) : 1.f;
}

}  // namespace eagle
