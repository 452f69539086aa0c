// Rotary positions with several axes: pair i of a head's RoPE part turns by the angle
// pos[axis(i)] * f(i). Its gradient is the turn back (inverse).
//
// The angle is kept in turns as a 64-bit fraction: f(i) / (2 pi) rounded to 2^-64 times the
// integer position, modulo one turn by the multiplication's own wrap-around. So it is off by
// at most |position| 2^-65 turns, where at position 2^20 an fp32 product would be off by up to
// 0.06 rad. Its top 32 bits (2^-32 turns more) then go, rounded to fp32's 24 (2^-26 turns),
// to the fp32 sine and cosine of a multiple of pi.
//
// Memory bound: q is read and written once (the no-RoPE part is copied, or left alone in
// place). One CTA takes a few tokens: it computes their cosines and sines once, in shared
// memory, and all heads of the token use them. 2048 tokens of 128 bf16 heads of 192 (202 MB):
// 34.5 us, 5.85 TB/s, 86% of a plain copy's rate.
#include "rope.h"

#include <algorithm>
#include <type_traits>

namespace laga {
namespace {

using ll = long long;
constexpr int THREADS = 256;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(bf16 v) { return __bfloat162float(v); }

// cos and sin of the CTA's tokens x pairs into shared memory.
__device__ __forceinline__ void fill_angles(const RopeArgs& a, const RopeTable& t, ll first, int tokens, float2* cs) {
  const int n = a.d_rope / 2;
  for (int e = threadIdx.x; e < tokens * n; e += THREADS) {
    const int k = e / n, i = e - k * n;
    const ll at = t.axis[i] * a.tokens + first + k;
    const ll p = a.pos64 ? static_cast<const ll*>(a.pos)[at] : static_cast<ll>(static_cast<const int*>(a.pos)[at]);
    const uint64_t turn = static_cast<uint64_t>(p) * t.turns[i];
    const float half_turns = static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f;  // [-1, 1]
    float s, c;
    sincospif(half_turns, &s, &c);
    cs[e] = make_float2(c, a.inverse ? -s : s);
  }
}

// One value at a time: any widths and alignment. q is [token][head][d_nope + d_rope].
template <typename T>
__global__ void __launch_bounds__(THREADS) rope_any_kernel(const RopeArgs a, const RopeTable t, int per_cta) {
  extern __shared__ float2 cs[];
  after_previous();
  const ll first = static_cast<ll>(blockIdx.x) * per_cta;
  const int tokens = static_cast<int>(min(static_cast<ll>(per_cta), a.tokens - first));
  const int n = a.d_rope / 2, heads = a.q ? a.n_h : 0, rows = heads + (a.k ? 1 : 0);
  fill_angles(a, t, first, tokens, cs);
  __syncthreads();
  // a unit is one pair, or one value of the no-RoPE part when it has to be copied
  const int copy = a.q_out != a.q ? a.d_nope : 0;
  const int per_row = copy + n;
  for (int e = threadIdx.x; e < tokens * rows * per_row; e += THREADS) {
    const int k = e / (rows * per_row);
    const int r = (e - k * rows * per_row) / per_row;
    const int u = e - (k * rows + r) * per_row;
    const bool is_q = r < heads;
    const ll row = is_q ? ((first + k) * a.n_h + r) * (a.d_nope + a.d_rope) : (first + k) * a.d_rope;
    const T* src = static_cast<const T*>(is_q ? a.q : a.k) + row;
    T* dst = static_cast<T*>(is_q ? a.q_out : a.k_out) + row;
    if (u >= n) {
      if (is_q) dst[u - n] = src[u - n];
      continue;
    }
    const int base = is_q ? a.d_nope : 0;
    const int i0 = base + (a.interleaved ? 2 * u : u), i1 = base + (a.interleaved ? 2 * u + 1 : n + u);
    const float2 c = cs[k * n + u];
    const float x = to_f(src[i0]), y = to_f(src[i1]);
    dst[i0] = static_cast<T>(x * c.x - y * c.y);
    dst[i1] = static_cast<T>(x * c.y + y * c.x);
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

// Exact division of 0 <= e < 2^26 by a fixed 1 <= d < 2^17.
struct Div {
  uint64_t mul;
  int shift;
  uint32_t d;
};
Div make_div(uint32_t d) {
  int bits = 0;
  while ((1u << bits) < d) ++bits;
  const int shift = 26 + bits;
  return Div{((uint64_t{1} << shift) + d - 1) / d, shift, d};
}
__device__ __forceinline__ int div_by(const Div& v, int e) {
  return static_cast<int>((static_cast<uint64_t>(e) * v.mul) >> v.shift);
}

// 16-byte units: rows and their RoPE part aligned to 16 bytes. A unit is a chunk of the
// no-RoPE part, an interleaved chunk, or a chunk of the first half with its partner in the
// second (the halves a multiple of the chunk). A thread loads UNROLL units before it works on
// the first: with one at a time 128 heads of 2048 tokens took 60 us, half the copy's rate.
template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS) rope_vec_kernel(const RopeArgs a, const RopeTable t, int per_cta,
                                                           const Div per_head) {
  extern __shared__ float2 cs[];
  using V = Vec<T>;
  constexpr int N = V::N;
  constexpr int UNROLL = INTERLEAVED ? 4 : 2;
  after_previous();
  const ll first = static_cast<ll>(blockIdx.x) * per_cta;
  const int tokens = static_cast<int>(min(static_cast<ll>(per_cta), a.tokens - first));
  const int n = a.d_rope / 2, heads = a.q ? a.n_h : 0;
  fill_angles(a, t, first, tokens, cs);
  __syncthreads();
  const int rope_units = INTERLEAVED ? a.d_rope / N : n / N;
  const int copy = a.q_out != a.q ? a.d_nope / N : 0;
  const int q_units = heads * static_cast<int>(per_head.d), units = q_units + (a.k ? rope_units : 0);
  const int q_row = (a.d_nope + a.d_rope) / N, half = n / N;  // chunks
  for (int k = 0; k < tokens; ++k) {
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const T*>(a.q)) + (first + k) * a.n_h * q_row;
    uint4* q_out = reinterpret_cast<uint4*>(static_cast<T*>(a.q_out)) + (first + k) * a.n_h * q_row;
    const uint4* kr = reinterpret_cast<const uint4*>(static_cast<const T*>(a.k)) + (first + k) * (a.d_rope / N);
    uint4* k_out = reinterpret_cast<uint4*>(static_cast<T*>(a.k_out)) + (first + k) * (a.d_rope / N);
    const float2* c = cs + k * n;
    for (int e0 = threadIdx.x; e0 < units; e0 += THREADS * UNROLL) {
      uint4 x[UNROLL], y[UNROLL];
      uint4* dst[UNROLL];
      int unit[UNROLL];  // < 0: a copy
#pragma unroll
      for (int j = 0; j < UNROLL; ++j) {
        const int e = e0 + THREADS * j;
        dst[j] = nullptr;
        if (e >= units) continue;
        const uint4* src;
        if (e < q_units) {
          const int h = div_by(per_head, e);
          int u = e - h * static_cast<int>(per_head.d);
          const bool rotated = u >= copy;
          if (rotated) u += a.d_nope / N - copy;
          src = q + h * q_row + u;
          dst[j] = q_out + h * q_row + u;
          unit[j] = rotated ? u - a.d_nope / N : -1;
        } else {
          unit[j] = e - q_units;
          src = kr + unit[j];
          dst[j] = k_out + unit[j];
        }
        x[j] = __ldcs(src);
        if (!INTERLEAVED && unit[j] >= 0) y[j] = __ldcs(src + half);
      }
#pragma unroll
      for (int j = 0; j < UNROLL; ++j) {
        if (!dst[j]) continue;
        if (unit[j] < 0) {
          *dst[j] = x[j];
          continue;
        }
        if constexpr (INTERLEAVED) {
          const float2* w = c + unit[j] * (N / 2);
          float v[N];
          V::get(x[j], v);
#pragma unroll
          for (int i = 0; i < N / 2; ++i) {
            const float p = v[2 * i], r = v[2 * i + 1];
            v[2 * i] = p * w[i].x - r * w[i].y;
            v[2 * i + 1] = p * w[i].y + r * w[i].x;
          }
          *dst[j] = V::put(v);
        } else {
          const float2* w = c + unit[j] * N;
          float v[N], z[N];
          V::get(x[j], v);
          V::get(y[j], z);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const float p = v[i], r = z[i];
            v[i] = p * w[i].x - r * w[i].y;
            z[i] = p * w[i].y + r * w[i].x;
          }
          *dst[j] = V::put(v);
          dst[j][half] = V::put(z);
        }
      }
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename T>
cudaError_t launch(const RopeArgs& a, const RopeTable& t, cudaStream_t st) {
  constexpr int N = Vec<T>::N;
  const bool vec = a.d_nope % N == 0 && a.d_rope % N == 0 && (a.interleaved || (a.d_rope / 2) % N == 0) &&
                   aligned16(a.q) && aligned16(a.q_out) && aligned16(a.k) && aligned16(a.k_out);
  const int n = a.d_rope / 2;
  const ll work = static_cast<ll>((a.q ? a.n_h : 0)) * (a.d_nope + a.d_rope) + (a.k ? a.d_rope : 0);  // values a token
  // a few tokens per CTA when a token is little work, but no fewer CTAs than two per SM
  ll per = work > 0 ? 4096 / work : 1;
  const ll spread = a.tokens / (2 * static_cast<ll>(sm_count()));
  if (per > spread) per = spread;
  if (per > 16) per = 16;
  if (per < 1) per = 1;
  const unsigned grid = static_cast<unsigned>((a.tokens + per - 1) / per);
  const size_t smem = static_cast<size_t>(per) * n * sizeof(float2);
  const int copy = a.q_out != a.q ? a.d_nope / N : 0;
  const Div head = make_div(static_cast<uint32_t>(std::max(1, copy + (a.interleaved ? a.d_rope : n) / N)));
  if (!vec)
    return launch_next(rope_any_kernel<T>, grid, THREADS, smem, st, a, t, static_cast<int>(per));
  return launch_next(a.interleaved ? rope_vec_kernel<T, true> : rope_vec_kernel<T, false>, grid, THREADS, smem, st, a, t,
                     static_cast<int>(per), head);
}

}  // namespace

LaunchResult rope(const RopeArgs& a, const RopeTable& t, cudaStream_t st) {
  LaunchResult r;
  r.err = a.is_bf16 ? launch<bf16>(a, t, st) : launch<float>(a, t, st);
  if (r.err != cudaSuccess) r.what = "rope";
  return r;
}

}  // namespace laga
