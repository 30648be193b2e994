// Rotary positions of q and k, and v, into the tree attention's layouts.
//
// Pair j of a head at position p turns by the angle p * f_j.  The angle is
// wanted modulo a turn for positions up to 2^31: f_j / 2pi is taken as a 64-bit
// fixed-point fraction of a turn, and p * that, wrapping, is the reduced phase
// exactly; its top 32 bits are the turns that sincospi gets (a float's 24 bits
// of them: the angle is off by at most 2^-25 half turns, 1e-7).  No float64
// arithmetic is done per position.
//
// What bounds it: HBM (each element read once and written once).  A
// CTA takes one node and a run of its heads; the node's cos and sin are
// computed once per CTA into shared memory.
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

template <typename T> __device__ __forceinline__ float load_f(const T *p) { return static_cast<float>(*p); }

// One pair (or one copied element pair) per thread step: any rot_dim.
template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a) {
  __shared__ float2 cs[256];
  const int node = blockIdx.x, b = node / a.n, i = node % a.n;
  pdl_wait();
  const int pos = (a.pos_base ? a.pos_base[b] : 0) + (a.pos_off ? a.pos_off[node] : i) + a.shift;
  for (int j = threadIdx.x; j < a.half; j += kRopeThreads) {
    double t = a.inv_freq[j] * 0.15915494309189533577;  // turns per position
    t -= rint(t);
    const uint64_t inc = static_cast<uint64_t>(static_cast<int64_t>(t * 18446744073709551616.0));
    const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * inc;
    float sn, c;
    sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &sn, &c);
    cs[j] = make_float2(c * a.factor, sn * a.factor);
  }
  __syncthreads();
  pdl_trigger();
  const int H = a.Hq + 2 * a.Hkv, pairs = a.dh / 2;
  for (int idx = blockIdx.y * kRopeThreads + threadIdx.x; idx < H * pairs; idx += gridDim.y * kRopeThreads) {
    const int h = idx / pairs, j = idx % pairs;
    const T *src;
    T *dst;
    bool turn = true;
    if (h < a.Hq) {
      src = reinterpret_cast<const T *>(a.q) + node * a.ld_q + static_cast<int64_t>(h) * a.dh;
      dst = reinterpret_cast<T *>(a.q_out) + (static_cast<int64_t>(node) * a.Hq + h) * a.dh;
    } else if (h < a.Hq + a.Hkv) {
      const int g = h - a.Hq;
      src = reinterpret_cast<const T *>(a.k) + node * a.ld_k + static_cast<int64_t>(g) * a.dh;
      dst = reinterpret_cast<T *>(a.k_tree) + ((static_cast<int64_t>(b) * a.Hkv + g) * a.n + i) * a.dh;
    } else {
      if (!a.v) continue;
      const int g = h - a.Hq - a.Hkv;
      src = reinterpret_cast<const T *>(a.v) + node * a.ld_v + static_cast<int64_t>(g) * a.dh;
      dst = reinterpret_cast<T *>(a.v_tree) + ((static_cast<int64_t>(b) * a.Hkv + g) * a.n + i) * a.dh;
      turn = false;
    }
    const bool rot = turn && j < a.half;
    const int c0 = rot ? (a.interleaved ? 2 * j : j) : (turn ? 2 * a.half + 2 * (j - a.half) : 2 * j);
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

cudaError_t launch_rope(const void *q, const void *k, const void *v, int dtype, int B, int n, int Hq, int Hkv, int dh,
                        int64_t ld_q, int64_t ld_k, int64_t ld_v, const double *inv_freq, int rot_dim,
                        int interleaved, float factor, const int32_t *pos_base, const int32_t *pos_off, int shift,
                        void *q_out, void *k_tree, void *v_tree, cudaStream_t st) {
  RopeArgs a = {q, k, v, q_out, k_tree, v_tree, B, n, Hq, Hkv, dh, rot_dim / 2, interleaved, shift,
                ld_q, ld_k, ld_v, inv_freq, pos_base, pos_off, factor};
  const int items = (Hq + 2 * Hkv) * dh / 2;
  const dim3 grid(B * n, (items + kRopeThreads * 8 - 1) / (kRopeThreads * 8));
  return dtype == EAGLE_BF16 ? launch_chained(rope_kernel<__nv_bfloat16>, grid, dim3(kRopeThreads), 0, st, a)
                             : launch_chained(rope_kernel<float>, grid, dim3(kRopeThreads), 0, st, a);
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
