// Per-score arithmetic of the masked attention kernels, in the log2 domain: with x the raw
// product q . K, a score's exponent is
//   t2 = log2(e) * (cap tanh(scale x / cap) - slope |position - key|)
// without a cap: scale x in place of cap tanh(.); without slopes: no second term.
#pragma once
#include "internal.h"
#include "ptx.cuh"

namespace laga {

struct ModParams {
  float u_scale;        // scale / cap
  float cap_log2;       // cap * log2(e)
  const float* slopes;  // [n_h]
};

inline ModParams mod_params(const Dims& d, const ScoreMods& m) {
  ModParams p{};
  if (m.cap > 0.f) {
    p.u_scale = d.scale / m.cap;
    p.cap_log2 = m.cap * 1.4426950408889634f;
  }
  p.slopes = m.slopes;
  return p;
}

// tanh(u) = 1 - 2 / (1 + e^(2u)), to ~1e-7 absolute: it is multiplied by the cap, so the
// absolute error is the one that counts. e^(2u) = inf gives 1, 0 gives -1. Two of the
// special-function unit's instructions a score, beside the softmax's own.
__device__ __forceinline__ float tanh_abs(float u) {
  return 1.f - __fdividef(2.f, 1.f + ex2_approx(u * 2.8853900817779268f));
}

// The same for caps so large that 1e-7 of them shows (kModFar): the first terms of tanh's series
// for small u, exact there to 1e-7 of tanh(u) itself.
__device__ __forceinline__ float tanh_rel(float u) {
  const float w = u * u;
  return fabsf(u) < 0.1f ? u * fmaf(w, fmaf(w, 2.f / 15.f, -1.f / 3.f), 1.f) : tanh_abs(u);
}

// Bit k of 32: key k of a run is visible, for the visible interval [first, end) relative to the run.
// Testing a bit a key costs less than comparing each key's index (2 x 4096 rows in 5 documents,
// capped: forward 141 -> 134 us, dq 151 -> 147). Only where a tile is partly masked: made for every
// tile, the bits cost dq 3% of a long walk.
__device__ __forceinline__ uint32_t visible_bits(int first, int end) {
  const int a = min(max(first, 0), 32), e = min(max(end, 0), 32);
  uint32_t below_a, below_e;  // shl gives 0 for 32, and 0 - 1 all bits
  asm("shl.b32 %0, 1, %1;" : "=r"(below_a) : "r"(a));
  asm("shl.b32 %0, 1, %1;" : "=r"(below_e) : "r"(e));
  return (below_e - 1u) & ~(below_a - 1u);
}

// Bit j of lane i becomes bit i of lane j.
__device__ __forceinline__ uint32_t transpose_bits(uint32_t x, int lane) {
  constexpr uint32_t low[5] = {0x0000ffffu, 0x00ff00ffu, 0x0f0f0f0fu, 0x33333333u, 0x55555555u};
#pragma unroll
  for (int s = 0; s < 5; ++s) {
    const int j = 16 >> s;
    const uint32_t y = __shfl_xor_sync(0xffffffffu, x, j);
    x = lane & j ? ((y >> j) & low[s]) | (x & ~low[s]) : (x & low[s]) | ((y & low[s]) << j);
  }
  return x;
}

// a * 0 + c on both halves: c, or a NaN where a is not finite.
__device__ __forceinline__ uint32_t times_zero_plus_bf16x2(uint32_t a, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(0u), "r"(c));
  return r;
}

// Two fp32 values in one 64-bit register: products and sums of pairs are one instruction.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ F2 f2(float x) { return f2(x, x); }
__device__ __forceinline__ float2 parts(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// tanh(u) / u for |u| <= 1 as a polynomial in w = u^2 (a least-squares fit at Chebyshev
// points): tanh to 7e-7 relative in fp32, on the multiply-add units instead of the special
// functions, two scores per instruction. Scores rarely come near the cap, and a thread whose
// visible scores of a tile all stay within it takes this form (a capped forward of 2048 rows
// of 128 heads over 16384 keys: 2.32 ms with tanh_abs for every score, 1.89 with this). Which form a score takes depends on
// nothing but its own row (or key): masked scores are set to 0 before the question is asked.
__device__ __forceinline__ F2 tanh_over_u(F2 w) {
  F2 p = fma(f2(-0.00308040925f), w, f2(0.0167767762f));
  p = fma(p, w, f2(-0.0516354587f));
  p = fma(p, w, f2(0.132825138f));
  p = fma(p, w, f2(-0.333291803f));
  return fma(p, w, f2(0.999999442f));
}

// The bias of N consecutive keys (or query rows) added to exponents: -slope2 |dist + sign * k|
// for k < N, as pairs. Where the distance keeps its sign over the run it is linear in k.
template <int N, int SIGN, class Get, class Put>
__device__ __forceinline__ void add_bias(float slope2, float dist, Get&& get, Put&& put) {
  const float last = dist + static_cast<float>(SIGN * (N - 1));
  const bool up = dist >= 0.f && last >= 0.f, down = dist <= 0.f && last <= 0.f;
  if (__all_sync(0xffffffffu, up || down)) {
    const float s = up ? -slope2 : slope2;
    const F2 step = f2(s), base = f2(s * dist);
#pragma unroll
    for (int k = 0; k < N; k += 2)
      put(k, add(get(k), fma(f2(static_cast<float>(SIGN * k), static_cast<float>(SIGN * (k + 1))), step, base)));
  } else {
#pragma unroll
    for (int k = 0; k < N; k += 2) {
      const F2 d = f2(fabsf(dist + static_cast<float>(SIGN * k)), fabsf(dist + static_cast<float>(SIGN * (k + 1))));
      put(k, fma(d, f2(-slope2), get(k)));
    }
  }
}

// Whether this thread's N raw scores (bit patterns) stay within |u| <= 1.
template <int N>
__device__ __forceinline__ bool all_small(const uint32_t (&x)[N], float u_scale) {
  float a = fabsf(__uint_as_float(x[0])), b = fabsf(__uint_as_float(x[1]));
#pragma unroll
  for (int k = 2; k < N; k += 2) {
    a = fmaxf(a, fabsf(__uint_as_float(x[k])));
    b = fmaxf(b, fabsf(__uint_as_float(x[k + 1])));
  }
  return fmaxf(a, b) * u_scale <= 1.f;
}

}  // namespace laga
