// Device pieces that the rotation's kernels share: angles as fractions of a turn, 16-byte chunks of
// values as fp32.
#pragma once
#include "rope.h"

namespace laga {

using ll = long long;

inline bool aligned_to_16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(bf16 v) { return __bfloat162float(v); }

// cos and sin of position p times `turns` (a frequency as a 64-bit fraction of a turn).
__device__ __forceinline__ float2 cos_sin(ll p, uint64_t turns) {
  const uint64_t turn = static_cast<uint64_t>(p) * turns;
  const float half_turns = static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f;  // [-1, 1]
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c, s);
}

// cos and sin of the CTA's tokens x pairs into shared memory.
template <int THREADS>
__device__ __forceinline__ void fill_angles(const RopeArgs& a, const RopeTable& t, ll first, int tokens, float2* cs) {
  const int n = a.d_rope / 2;
  for (int e = threadIdx.x; e < tokens * n; e += THREADS) {
    const int k = e / n, i = e - k * n;
    const ll at = t.axis[i] * a.tokens + first + k;
    const ll p = a.pos64 ? static_cast<const ll*>(a.pos)[at] : static_cast<ll>(static_cast<const int*>(a.pos)[at]);
    const float2 v = cos_sin(p, t.turns[i]);
    cs[e] = make_float2(v.x, a.inverse ? -v.y : v.y);
  }
}

template <typename T>
struct Vec;
template <>
struct Vec<bf16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[2 * k] = __uint_as_float(w[k] << 16);
      x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * k], x[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(uint4 v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
};

}  // namespace laga
