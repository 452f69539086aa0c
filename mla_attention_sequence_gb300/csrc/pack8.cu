// Activation checkpoints in 8 bits: per block of 32 values of a row one power of two,
// the smallest that brings the block's largest finite size to at most 448, and 32 e4m3
// codes. A power of two costs no rounding of its own and divides exactly, so the only
// error is the code's (half a step: 2^-4 of the value, or 2^-10 of the scale for values
// more than 2^14 below the block's largest). Infinities and NaN become the NaN code and
// do not set the scale.
//
// Memory bound: a bf16 value is 2 bytes read and 1 + 1/32 written. Where a row's length is
// a multiple of 32 the whole tensor is one run of blocks and a thread owns 16 consecutive
// bytes of input (8 bf16 or 4 fp32), so a block's maximum is two or three shuffles. Other
// lengths take one warp per block, a value per lane. Saving q of 2048 tokens of 128 bf16 heads
// of 192 (153 MB moved): 27.5 us, 5.56 TB/s, 82% of a plain copy's rate.
#include "mask.h"

#include <cuda_fp8.h>

namespace laga {
namespace {

using ll = long long;

// Biased exponent of a block's scale from the bits of its largest finite size.
__device__ __forceinline__ uint32_t scale_exponent(uint32_t top) {
  if (top == 0u) return 127u;
  const int e = static_cast<int>(top >> 23) - ((top & 0x7fffffu) <= 0x600000u ? 8 : 7);  // 448 = 1.75 * 2^8
  return static_cast<uint32_t>(max(e, 0));
}
// 2^(127 - e): e <= 247, so never a subnormal
__device__ __forceinline__ float inverse_scale(uint32_t e) { return __uint_as_float((254u - e) << 23); }

// bits of |x|, 0 for an infinity or NaN
__device__ __forceinline__ uint32_t size_bits(float x) {
  const uint32_t u = __float_as_uint(x) & 0x7fffffffu;
  return u >= 0x7f800000u ? 0u : u;
}

// Two codes; x * 0 adds a NaN for an infinity (the conversion saturates it otherwise).
__device__ __forceinline__ uint32_t codes2(float a, float b, float inv) {
  const float2 v = make_float2(fmaf(a, 0.f, a * inv), fmaf(b, 0.f, b * inv));
  return __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
}

template <typename T>
struct Chunk;  // 16 bytes of input as floats
template <>
struct Chunk<bf16> {
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
struct Chunk<float> {
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

// Chunks a thread of the aligned kernels takes, 256 apart, all loads issued before the first
// use: one 16-byte load per thread in flight (32 KB an SM) leaves the memory partly idle.
constexpr int UNROLL = 4;

template <typename T>
__global__ void __launch_bounds__(256) pack8_kernel(ll chunks, const T* __restrict__ x, uint8_t* __restrict__ codes,
                                                    uint8_t* __restrict__ scales) {
  after_previous();
  using C = Chunk<T>;
  constexpr int PER = kPackBlock / C::N;  // threads per block
  const ll first = static_cast<ll>(blockIdx.x) * (256 * UNROLL) + threadIdx.x;
  uint4 raw[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const ll i = first + 256 * u;
    raw[u] = i < chunks ? __ldcs(reinterpret_cast<const uint4*>(x) + i) : make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const ll i = first + 256 * u;
    float v[C::N];
    C::get(raw[u], v);
    uint32_t top = 0u;
#pragma unroll
    for (int k = 0; k < C::N; ++k) top = max(top, size_bits(v[k]));
#pragma unroll
    for (int o = PER / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t e = scale_exponent(top);
    const float inv = inverse_scale(e);
    if (i >= chunks) continue;
    if constexpr (C::N == 8) {
      reinterpret_cast<uint2*>(codes)[i] = make_uint2(codes2(v[0], v[1], inv) | codes2(v[2], v[3], inv) << 16,
                                                      codes2(v[4], v[5], inv) | codes2(v[6], v[7], inv) << 16);
    } else {
      reinterpret_cast<uint32_t*>(codes)[i] = codes2(v[0], v[1], inv) | codes2(v[2], v[3], inv) << 16;
    }
    if (i % PER == 0) scales[i / PER] = static_cast<uint8_t>(e);
  }
}

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(bf16 v) { return __bfloat162float(v); }

// Rows whose length is no multiple of 32 (or an unaligned tensor): a warp per block.
template <typename T>
__global__ void __launch_bounds__(256) pack8_any_kernel(ll rows, int cols, int blocks, const T* __restrict__ x,
                                                        uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  after_previous();
  const ll w = (static_cast<ll>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (w >= rows * blocks) return;
  const ll row = w / blocks;
  const int col = static_cast<int>(w - row * blocks) * kPackBlock + (threadIdx.x & 31);
  const bool in = col < cols;
  const float v = in ? as_float(x[row * cols + col]) : 0.f;
  const uint32_t e = scale_exponent(__reduce_max_sync(0xffffffffu, size_bits(v)));
  if (in) codes[row * cols + col] = static_cast<uint8_t>(codes2(v, 0.f, inverse_scale(e)) & 0xffu);
  if ((threadIdx.x & 31) == 0) scales[w] = static_cast<uint8_t>(e);
}

template <typename T>
__global__ void __launch_bounds__(256) unpack8_kernel(ll chunks, const uint8_t* __restrict__ codes,
                                                      const uint8_t* __restrict__ scales, T* __restrict__ x) {
  after_previous();
  using C = Chunk<T>;
  constexpr int PER = kPackBlock / C::N;
  constexpr int W = C::N / 4;
  const ll first = static_cast<ll>(blockIdx.x) * (256 * UNROLL) + threadIdx.x;
  uint32_t w[UNROLL][W];
  uint8_t e[UNROLL];
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const ll i = first + 256 * u;
    if (i >= chunks) continue;
    e[u] = scales[i / PER];
    if constexpr (W == 2) {
      const uint2 c = __ldcs(reinterpret_cast<const uint2*>(codes) + i);
      w[u][0] = c.x;
      w[u][W - 1] = c.y;
    } else {
      w[u][0] = __ldcs(reinterpret_cast<const uint32_t*>(codes) + i);
    }
  }
#pragma unroll
  for (int u = 0; u < UNROLL; ++u) {
    const ll i = first + 256 * u;
    if (i >= chunks) continue;
    const float s = scale_value(e[u]);
    float v[C::N];
#pragma unroll
    for (int k = 0; k < C::N / 2; ++k) {
      const float2 f = e4m3x2_to_float2(static_cast<uint16_t>(w[u][k / 2] >> (16 * (k & 1))));
      v[2 * k] = f.x * s;
      v[2 * k + 1] = f.y * s;
    }
    reinterpret_cast<uint4*>(x)[i] = C::put(v);
  }
}

template <typename T>
__global__ void __launch_bounds__(256) unpack8_any_kernel(ll rows, int cols, const Packed p, T* __restrict__ x) {
  after_previous();
  const ll i = static_cast<ll>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= rows * cols) return;
  const ll row = i / cols;
  x[i] = static_cast<T>(unpack8_value(p, row, cols, static_cast<int>(i - row * cols)));
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <typename T>
cudaError_t pack(ll rows, int cols, const T* x, uint8_t* codes, uint8_t* scales, cudaStream_t st) {
  const int blocks = (cols + kPackBlock - 1) / kPackBlock;
  if (cols % kPackBlock == 0 && aligned(x, 16) && aligned(codes, 8)) {
    const ll chunks = rows * cols / Chunk<T>::N;
    const unsigned grid = static_cast<unsigned>((chunks + 256 * UNROLL - 1) / (256 * UNROLL));
    return launch_next(pack8_kernel<T>, grid, 256, 0, st, chunks, x, codes, scales);
  }
  const unsigned grid = static_cast<unsigned>((rows * blocks + 7) / 8);
  return launch_next(pack8_any_kernel<T>, grid, 256, 0, st, rows, cols, blocks, x, codes, scales);
}

template <typename T>
cudaError_t unpack(ll rows, int cols, const Packed& p, T* x, cudaStream_t st) {
  if (cols % kPackBlock == 0 && aligned(x, 16) && aligned(p.codes, 8)) {
    const ll chunks = rows * cols / Chunk<T>::N;
    const unsigned grid = static_cast<unsigned>((chunks + 256 * UNROLL - 1) / (256 * UNROLL));
    return launch_next(unpack8_kernel<T>, grid, 256, 0, st, chunks, p.codes, p.scales, x);
  }
  const unsigned grid = static_cast<unsigned>((rows * cols + 255) / 256);
  return launch_next(unpack8_any_kernel<T>, grid, 256, 0, st, rows, cols, p, x);
}

}  // namespace

LaunchResult pack8(bool is_bf16, ll rows, int cols, const void* x, uint8_t* codes, uint8_t* scales, cudaStream_t st) {
  LaunchResult r;
  r.err = is_bf16 ? pack(rows, cols, static_cast<const bf16*>(x), codes, scales, st)
                  : pack(rows, cols, static_cast<const float*>(x), codes, scales, st);
  if (r.err != cudaSuccess) r.what = "pack8";
  return r;
}

LaunchResult unpack8(bool is_bf16, ll rows, int cols, const Packed& p, void* x, cudaStream_t st) {
  LaunchResult r;
  r.err = is_bf16 ? unpack(rows, cols, p, static_cast<bf16*>(x), st) : unpack(rows, cols, p, static_cast<float*>(x), st);
  if (r.err != cudaSuccess) r.what = "unpack8";
  return r;
}

}  // namespace laga
