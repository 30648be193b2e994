// What the rotation kernels share: arguments, a position's turns, where a head is
// read and written.
#pragma once

#include "common.cuh"

namespace eagle {

struct RopeArgs {
  const void *q, *k, *v;
  void *q_out, *k_tree, *v_tree;
  int B, n, Hq, Hkv, dh, half, interleaved, shift;
  int64_t ld_q, ld_k, ld_v;
  const double *inv_freq;
  const int32_t *pos_base, *pos_off;
  float factor;
};

// A frequency as turns a position, in 64-bit fixed point.
__device__ __forceinline__ uint64_t turn_step(double inv_freq) {
  double t = inv_freq * 0.15915494309189533577;  // turns per position
  t -= rint(t);
  return static_cast<uint64_t>(static_cast<int64_t>(t * 18446744073709551616.0));
}
// cos and sin (times the factor) at a position.
__device__ __forceinline__ float2 turn_at(uint64_t step, int pos, float factor) {
  const uint64_t phase = static_cast<uint64_t>(static_cast<int64_t>(pos)) * step;
  float sn, c;
  sincospif(static_cast<float>(static_cast<int32_t>(phase >> 32)) * 4.656612873077393e-10f, &sn, &c);
  return make_float2(c * factor, sn * factor);
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

}  // namespace eagle
