// The paged 4-bit latent cache: rows written and read, the sharing out of an attention call's key
// tiles and the joining of its pieces, and the attention on the CUDA cores for any widths.
//
// Writing and reading are bound by latency: a launch; a row's place behind its start and its table's
// entry; writing, a row's chain of a sum over the warp, a root and a cosine (500 instructions a row, issued
// in 45% of the cycles). A warp takes a row, a lane a block of 16 latents (at d_c = 512 each lane exactly
// one) and a pair of the RoPE key, so that the only thing that lanes exchange is the key's sum of squares.
// 12288 rows of 512 + 64 in bf16 (events around the launch, 6 us of it the launch's
// own): 18 us written, 10 read, 3 of DRAM either way. Codes by comparisons with the borders for bf16 too
// instead of the conversion: 25 written; with 4, 6 and 12 CTAs' shares an SM 18 .. 19 and 11 .. 12.
#include "cache4.h"
#include "rope_device.cuh"

#include <cuda_fp16.h>
#include <cuda_fp4.h>

#include <algorithm>

namespace laga {
namespace {

constexpr int ROW_WARPS = 8, ROW_CTAS = 3;  // CTAs an SM holds at once

__device__ __forceinline__ float scale_of(int byte) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7)));
}

// What a stored scale byte stands for: those past the grid are blocks that are not finite.
__device__ __forceinline__ float value_scale(int byte) {
  return byte > kCacheTopScale ? __int_as_float(0x7fc00000) : scale_of(byte);
}

// The smallest scale s of the grid with 6 s >= top (the largest scale if there is none), exactly: a
// first guess from top / 6 rounded up to the grid, then at most a step either way by the products,
// which are exact.
__device__ __forceinline__ int scale_for(float top) {
  if (!(top > 0.f)) return 0;
  const float q = fminf(top * (1.f / 6.f), 10240.f);
  int e;
  if (q >= 0x1p-14f)
    e = static_cast<int>((__float_as_uint(q) + 0xfffffu) >> 20) - ((127 - 15) << 3);
  else
    e = static_cast<int>(ceilf(q * 0x1p17f));
  e = min(max(e, 1), kCacheTopScale);
  if (e < kCacheTopScale && 6.f * scale_of(e) < top) ++e;
  if (e > 1 && 6.f * scale_of(e - 1) >= top) --e;
  return e;
}

// The code of v: its nearest multiple of s, ties to the even code; s > 0. Bit by bit: the borders of one
// level are two or four of the halves between neighbours, which are few-bit multiples of s, exact in fp32.
__device__ __forceinline__ uint32_t code_for(float v, float s) {
  const float a = fabsf(v);
  const bool b2 = a >= 1.75f * s;
  const bool b1 = a >= (b2 ? 3.5f * s : 0.75f * s);
  const bool b0 = a > (b1 ? (b2 ? 5.f * s : 1.25f * s) : (b2 ? 2.5f * s : 0.25f * s));
  return (v < 0.f ? 8u : 0u) | (b2 ? 4u : 0u) | (b1 ? 2u : 0u) | (b0 ? 1u : 0u);
}

__device__ __forceinline__ float2 codes_to_float2(uint32_t byte) {
  const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(byte), __NV_E2M1);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// The 16 values of one block -> 8 bytes of codes and a scale byte.
__device__ __forceinline__ uint2 encode_block(const float (&v)[16], int* scale) {
  float top = 0.f;
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    finite = finite && fabsf(v[i]) <= 3.402823466e38f;
    top = fmaxf(top, fabsf(v[i]));
  }
  const int e = finite ? scale_for(top) : kCacheNanScale;
  const float s = finite && e > 0 ? scale_of(e) : 1.f;  // e = 0: zeros only
  uint2 w = make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w.x |= code_for(v[i], s) << (4 * i);
    w.y |= code_for(v[8 + i], s) << (4 * i);
  }
  *scale = e;
  return finite ? w : make_uint2(0, 0);
}

// The same for 16 bf16 values in two chunks, by the conversion instruction on v / s. That is exact although
// 1 / s is not: a border between two codes is a number of 3 bits times s, s one of 4, so v of 8 bits is
// either on it or more than 2^-9 of it away. v (1 / s) is within 2^-22 of v / s, and rounded to 12 bits it
// is the border in the first case (the conversion sends ties to the even code) and on v's side of it in the
// other. A sum with +0 turns -0 into +0, whose code has no sign.
__device__ __forceinline__ uint2 encode_block(const uint4 (&held)[2], int* scale) {
  const uint32_t x[8] = {held[0].x, held[0].y, held[0].z, held[0].w, held[1].x, held[1].y, held[1].z, held[1].w};
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {  // sizes compare as integers; what is not finite comes out on top
    const uint32_t a = x[i] & 0x7fff7fffu;
    most = __vmaxu2(most, a);
  }
  const uint32_t top = max(most & 0xffffu, most >> 16);
  const bool finite = top < 0x7f80u;
  const int e = finite ? scale_for(__uint_as_float(top << 16)) : kCacheNanScale;
  const float inv = finite && e > 0 ? 1.f / scale_of(e) : 0.f;
  auto near = [&](float v) {
    return __uint_as_float((__float_as_uint(fmaf(v, inv, 0.f)) + 0x800u) & 0xfffff000u);
  };
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    b[i] = __nv_cvt_float2_to_fp4x2(make_float2(near(__uint_as_float(x[i] << 16)), near(__uint_as_float(x[i] & 0xffff0000u))),
                                    __NV_E2M1, cudaRoundNearest);
  *scale = e;
  const uint2 w = make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                             __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
  return finite ? w : make_uint2(0, 0);
}

// The rows of the padded batch that a warp takes: `per` (at most 32) consecutive ones. Lane j finds the
// place of the j-th, so that the loads behind each other that this takes are waited for once.
struct WarpRows {
  ll first;
  int n;     // rows; 0 past the batch
  ll p;      // lane's row: its position, and its slot in the pool (-1: none)
  ll slot;
  bool stored;  // i < counts[b]
};
__device__ __forceinline__ WarpRows warp_rows(const CacheRows& at, int per) {
  WarpRows r;
  r.first = (static_cast<ll>(blockIdx.x) * ROW_WARPS + (threadIdx.x >> 5)) * per;
  r.n = static_cast<int>(max(0ll, min(static_cast<ll>(per), static_cast<ll>(at.pages.B) * at.rows - r.first)));
  return r;
}
__device__ __forceinline__ void find_slots(const CacheView& c, const CacheRows& at, int* status, int where, WarpRows& r) {
  const int j = threadIdx.x & 31;
  r.p = 0;
  r.slot = -1;
  r.stored = false;
  if (j >= r.n) return;
  const ll row = r.first + j;
  const int b = static_cast<int>(row / at.rows), i = static_cast<int>(row - static_cast<ll>(b) * at.rows);
  r.stored = !at.counts || i < __ldg(at.counts + b);
  r.p = static_cast<ll>(__ldg(at.starts + b)) + i;
  if (!r.stored) return;
  r.slot = cache_slot(c, at.pages, b, r.p);
  if (r.slot < 0) report_page(status, where);
}

// VEC: d_c a multiple of 16 and the latents 16-byte aligned. The next row's first block and key are
// loaded before the row at hand is worked on; a lane's frequency, weights and first block of columns are
// the same in every row (read once: lanes that index the kernel's arguments differently are served one
// after the other).
template <typename T, bool VEC>
__global__ void __launch_bounds__(ROW_WARPS * 32, ROW_CTAS) append_kernel(const CacheAppend a, const RopeTable t, int per) {
  constexpr int N = Vec<T>::N, V = VEC ? 16 / N : 1;
  after_previous();
  WarpRows rows = warp_rows(a.at, per);
  if (rows.n == 0) return;
  const int lane = threadIdx.x & 31, d_c = a.cache.d_c, bytes = a.cache.code_bytes(), blocks = a.cache.blocks();
  const int dr = a.cache.d_rope, n = (dr + 1) / 2;  // odd only without a rotation
  const T* w = static_cast<const T*>(a.w_k);
  // a lane's pair of the key: of the rotation, and without one any two
  const bool between = a.turn && a.rope.interleaved;
  auto first = [&](int u) { return between ? 2 * u : u; };
  auto second = [&](int u) { return between ? 2 * u + 1 : n + u; };
  struct Pair {
    float x0, x1;
  };
  auto pair_of = [&](const T* x, int u) {
    return Pair{to_f(x[first(u)]), second(u) < dr ? to_f(x[second(u)]) : 0.f};
  };
  auto latents = [&](ll row) { return static_cast<const T*>(a.c_kv) + row * d_c; };
  auto key = [&](ll row) { return static_cast<const T*>(a.k_rope) + row * dr; };
  auto load = [&](ll row, int k, uint4 (&to)[V]) {
#pragma unroll
    for (int j = 0; j < V; ++j) to[j] = __ldcs(reinterpret_cast<const uint4*>(latents(row) + k * 16) + j);
  };
  uint4 held[V], ahead[V];
  Pair x{0.f, 0.f}, nx{0.f, 0.f}, wk{1.f, 1.f};
  auto fetch = [&](ll row) {
    if constexpr (VEC)
      if (lane < blocks) load(row, lane, ahead);
    if (lane < n) nx = pair_of(key(row), lane);
  };
  fetch(rows.first);
  find_slots(a.cache, a.at, a.status, 301, rows);
  if (w && lane < n) wk = pair_of(w, lane);
  uint64_t turns = 0;
  int axis = 0;
  if (a.turn && lane < n) {
    turns = t.turns[lane];
    axis = t.axis[lane];
  }

#pragma unroll 1
  for (int j = 0; j < rows.n; ++j) {
    const ll row = rows.first + j, p = __shfl_sync(0xffffffffu, rows.p, j), slot = __shfl_sync(0xffffffffu, rows.slot, j);
#pragma unroll
    for (int i = 0; i < V; ++i) held[i] = ahead[i];
    x = nx;
    if (j + 1 < rows.n) fetch(row + 1);
    if (slot < 0) continue;
    uint8_t* codes = a.cache.codes + slot * bytes;
    uint8_t* scales = a.cache.scales + slot * blocks;
    for (int k = lane; k < blocks; k += 32) {
      int e;
      uint2 q;
      if constexpr (VEC)
        if (k != lane) load(row, k, held);
      if constexpr (VEC && N == 8) {
        q = encode_block(held, &e);
      } else {
        float v[16];
        if constexpr (VEC) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float y[N];
            Vec<T>::get(held[i], y);
#pragma unroll
            for (int m = 0; m < N; ++m) v[i * N + m] = y[m];
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = k * 16 + i < d_c ? to_f(latents(row)[k * 16 + i]) : 0.f;
        }
        q = encode_block(v, &e);
      }
      scales[k] = static_cast<uint8_t>(e);
      if constexpr (VEC) {
        *reinterpret_cast<uint2*>(codes + k * 8) = q;
      } else {
        for (int i = 0; i < 8 && k * 8 + i < bytes; ++i)
          codes[k * 8 + i] = static_cast<uint8_t>((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
      }
    }
    if (dr == 0) continue;
    T* out = static_cast<T*>(a.cache.keys) + slot * dr;
    float down = 1.f, f = 1.f;
    if (w) {
      auto squares = [&](float by) {
        float sum = 0.f;
        for (int u = lane; u < n; u += 32) {
          const Pair y = u == lane ? x : pair_of(key(row), u);
          sum = fmaf(y.x0 * by, y.x0 * by, fmaf(y.x1 * by, y.x1 * by, sum));
        }
        return warp_sum(sum);
      };
      float sum = squares(1.f);
      if (!(sum < 0x1p120f)) {  // squares that may have left fp32
        down = 0x1p-70f;
        sum = squares(down);
      }
      f = rsqrtf(fmaf(sum, 1.f / dr, a.eps * down * down));
    }
    for (int u = lane; u < n; u += 32) {
      const int i0 = first(u), i1 = second(u);
      Pair y = u == lane ? x : pair_of(key(row), u);
      if (w) {
        const Pair by = u == lane ? wk : pair_of(w, u);
        y.x0 = y.x0 * down * f * by.x0;
        y.x1 = y.x1 * down * f * by.x1;
      }
      if (a.turn) {
        ll pos = p;
        if (a.own_pos) {
          const ll at = (u == lane ? axis : t.axis[u]) * a.rope.tokens + row;
          pos = a.rope.pos64 ? static_cast<const ll*>(a.rope.pos)[at] : static_cast<ll>(static_cast<const int*>(a.rope.pos)[at]);
        }
        const float2 cs = cos_sin(pos, u == lane ? turns : t.turns[u]);
        y = {y.x0 * cs.x - y.x1 * cs.y, y.x0 * cs.y + y.x1 * cs.x};
      }
      out[i0] = static_cast<T>(y.x0);
      if (i1 < dr) out[i1] = static_cast<T>(y.x1);
    }
  }
}

// The next row's first block and key values are loaded before the row at hand is written.
template <typename T, bool VEC>
__global__ void __launch_bounds__(ROW_WARPS * 32, ROW_CTAS) read_kernel(const CacheRead a, int per) {
  constexpr int N = Vec<T>::N, KEYS = 2;  // key values of a lane that are loaded ahead
  after_previous();
  WarpRows rows = warp_rows(a.at, per);
  if (rows.n == 0) return;
  find_slots(a.cache, a.at, a.status, 302, rows);
  const int lane = threadIdx.x & 31, d_c = a.cache.d_c, dr = a.cache.d_rope, blocks = a.cache.blocks();
  uint2 w = make_uint2(0, 0), nw = w;
  int e = 0, ne = 0;
  T x[KEYS], nx[KEYS];
  auto codes_of = [&](ll slot) { return a.cache.codes + slot * a.cache.code_bytes(); };
  auto scales_of = [&](ll slot) { return a.cache.scales + slot * blocks; };
  auto key_of = [&](ll slot) { return static_cast<const T*>(a.cache.keys) + slot * dr; };
  auto fetch = [&](ll slot) {
    if (slot < 0) return;
    if constexpr (VEC) {
      if (lane < blocks) {
        nw = __ldcg(reinterpret_cast<const uint2*>(codes_of(slot)) + lane);
        ne = __ldcg(scales_of(slot) + lane);
      }
    }
#pragma unroll
    for (int i = 0; i < KEYS; ++i)
      if (lane + 32 * i < dr) nx[i] = __ldcg(key_of(slot) + lane + 32 * i);
  };
  ll next = __shfl_sync(0xffffffffu, rows.slot, 0);
  fetch(next);
#pragma unroll 1
  for (int j = 0; j < rows.n; ++j) {
    const ll row = rows.first + j, slot = next;
    const bool stored = __shfl_sync(0xffffffffu, rows.stored, j);
    w = nw;
    e = ne;
#pragma unroll
    for (int i = 0; i < KEYS; ++i) x[i] = nx[i];
    if (j + 1 < rows.n) {
      next = __shfl_sync(0xffffffffu, rows.slot, j + 1);
      fetch(next);
    }
    T* c = static_cast<T*>(a.c_kv) + row * d_c;
    T* key = static_cast<T*>(a.k_rope) + row * dr;
    if (slot < 0) {
      const float fill = stored ? __int_as_float(0x7fc00000) : 0.f;  // a row that the table has no page for: NaN
      for (int i = lane; i < d_c; i += 32) c[i] = static_cast<T>(fill);
      for (int i = lane; i < dr; i += 32) key[i] = static_cast<T>(fill);
      continue;
    }
#pragma unroll
    for (int i = 0; i < KEYS; ++i)
      if (lane + 32 * i < dr) key[lane + 32 * i] = x[i];
    for (int i = lane + 32 * KEYS; i < dr; i += 32) key[i] = __ldcg(key_of(slot) + i);
    if constexpr (VEC) {
      for (int k = lane; k < blocks; k += 32) {
        if (k != lane) {
          w = __ldcg(reinterpret_cast<const uint2*>(codes_of(slot)) + k);
          e = __ldcg(scales_of(slot) + k);
        }
        const float s = value_scale(e);
        float v[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 f = codes_to_float2(((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 0xffu);
          v[2 * i] = f.x * s;
          v[2 * i + 1] = f.y * s;
        }
#pragma unroll
        for (int m = 0; m < 16 / N; ++m) {
          float y[N];
#pragma unroll
          for (int i = 0; i < N; ++i) y[i] = v[m * N + i];
          reinterpret_cast<uint4*>(c + k * 16)[m] = Vec<T>::put(y);
        }
      }
    } else {
      for (int i = lane; i < d_c; i += 32) {
        const float2 f = codes_to_float2(__ldcg(codes_of(slot) + (i >> 1)));
        c[i] = static_cast<T>((i & 1 ? f.y : f.x) * value_scale(__ldcg(scales_of(slot) + i / kCacheBlock)));
      }
    }
  }
}

// ---------------------------------------------------------------- sharing out and joining

// Rows blockIdx.y, + gridDim.y, .. of item blockIdx.x. The pieces' weights first, in shared memory (128
// pieces at a time), then the columns, four a thread, all of a batch's loads before its sums.
constexpr int JOIN_THREADS = 128;
__global__ void __launch_bounds__(JOIN_THREADS) join_kernel(const CacheAttn a, float* ctx) {
  constexpr float to_log = 1.4426950408889634f;
  __shared__ float weights[JOIN_THREADS];
  __shared__ float2 red[JOIN_THREADS / 32];
  after_previous();
  const int item = blockIdx.x, b = item / a.row_tiles, r0 = (item - b * a.row_tiles) * a.tile;
  const int begin = __ldcg(a.first + item), end = __ldcg(a.first + item + 1);
  const CacheShare share = cache_share(a, 0);
  const int p0 = begin / share.quota, p1 = end > begin ? (end - 1) / share.quota : p0;
  if (end > begin && p0 == p1) return;  // written by the part that had it all
  const int rows = min(a.tile, a.rows - r0), d_c = a.cache.d_c, pieces = p1 - p0 + 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    const ll row = static_cast<ll>(b) * a.rows + r0 + r;
    const int i = (r0 + r) / a.n_h, h = (r0 + r) - i * a.n_h;
    float* out = ctx + row * d_c;
    float* lse = a.lse + (static_cast<ll>(b) * a.n_h + h) * a.Sq + i;
    if (end == begin) {
      const float v = lost_row(cache_row_bounds(a, b, i));
      for (int c = threadIdx.x; c < d_c; c += JOIN_THREADS) out[c] = v;
      if (threadIdx.x == 0) *lse = v != v ? v : -INFINITY;
      continue;
    }
    // piece k is part p0 + k's; the first began the item
    auto slot = [&](int k) { return static_cast<ll>(2 * (p0 + k) + (k == 0 ? 1 : 0)) * a.tile + r; };
    // each thread its pieces' maximum and sum, then the CTA's, in a fixed order
    float m = -INFINITY, l = 0.f;
    auto add = [&](float2 v) {
      const float to = fmaxf(m, v.x);
      const float from = to == -INFINITY ? 0.f : to;
      l = l * exp2f((m - from) * to_log) + v.y * exp2f((v.x - from) * to_log);  // 2^-inf = 0; a NaN sum stays one
      m = to;
    };
    for (int k = threadIdx.x; k < pieces; k += JOIN_THREADS) add(__ldcg(a.part_ml + slot(k)));
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) add(make_float2(__shfl_down_sync(0xffffffffu, m, k), __shfl_down_sync(0xffffffffu, l, k)));
    __syncthreads();  // red and weights of the row before
    if (lane == 0) red[warp] = make_float2(m, l);
    __syncthreads();
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int k = 0; k < JOIN_THREADS / 32; ++k) add(red[k]);
    l = row_sum(l, cache_row_bounds(a, b, i));
    const float inv = l != l ? l : l == 0.f ? 0.f : 1.f / l, from = m == -INFINITY ? 0.f : m;
    if (threadIdx.x == 0) *lse = l == 0.f ? -INFINITY : m + logf(l);
    for (int c0 = 0; c0 < d_c; c0 += 4 * JOIN_THREADS) {
      const int c = c0 + 4 * threadIdx.x;
      const bool vec = d_c % 4 == 0;
      float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k0 = 0; k0 < pieces; k0 += JOIN_THREADS) {
        const int n = min(JOIN_THREADS, pieces - k0);
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < n)
          weights[threadIdx.x] = exp2f((__ldcg(a.part_ml + slot(k0 + threadIdx.x)).x - from) * to_log);
        __syncthreads();
        if (c < d_c && vec) {
#pragma unroll 8
          for (int k = 0; k < n; ++k) {
            const float w = weights[k];
            const float4 o = __ldcg(reinterpret_cast<const float4*>(a.part_o + slot(k0 + k) * d_c + c));
            sum.x = fmaf(w, o.x, sum.x);
            sum.y = fmaf(w, o.y, sum.y);
            sum.z = fmaf(w, o.z, sum.z);
            sum.w = fmaf(w, o.w, sum.w);
          }
        } else if (c < d_c) {
          for (int k = 0; k < n; ++k) {
            const float w = weights[k];
            const float* o = a.part_o + slot(k0 + k) * d_c + c;
            sum.x = fmaf(w, __ldcg(o), sum.x);
            if (c + 1 < d_c) sum.y = fmaf(w, __ldcg(o + 1), sum.y);
            if (c + 2 < d_c) sum.z = fmaf(w, __ldcg(o + 2), sum.z);
            if (c + 3 < d_c) sum.w = fmaf(w, __ldcg(o + 3), sum.w);
          }
        }
      }
      if (c < d_c) out[c] = sum.x * inv;
      if (c + 1 < d_c) out[c + 1] = sum.y * inv;
      if (c + 2 < d_c) out[c + 2] = sum.z * inv;
      if (c + 3 < d_c) out[c + 3] = sum.w * inv;
    }
  }
}

// ---------------------------------------------------------------- CUDA cores, any widths

// q_lat[token][h][c] = sum over k of q[token][h][k] W_UK[c][h d_nope + k]: 32 tokens x 32 columns a CTA.
// One more CTA makes the plan.
template <typename T>
__global__ void __launch_bounds__(256) simt_prepare_kernel(const CacheAttn a, int d_nope, const T* q, const T* W, float* q_lat) {
  __shared__ float sq[32][33], sw[32][33];
  after_previous();
  if (blockIdx.x == gridDim.x - 1) {
    if (blockIdx.y == 0 && blockIdx.z == 0) cache4_plan_items<256>(a);
    return;
  }
  const int tokens = a.pages.B * a.Sq, n_h = a.n_h, d_c = a.cache.d_c, d_qk = d_nope + a.cache.d_rope;
  const int c0 = blockIdx.x * 32, h = blockIdx.y, x = threadIdx.x & 31, y = threadIdx.x >> 5;
  for (int t0 = blockIdx.z * 32; t0 < tokens; t0 += gridDim.z * 32) {
    float acc[4] = {};
    for (int k0 = 0; k0 < d_nope; k0 += 32) {
      for (int j = y; j < 32; j += 8) {
        const bool k = k0 + x < d_nope;
        sq[j][x] = k && t0 + j < tokens ? to_f(q[(static_cast<ll>(t0 + j) * n_h + h) * d_qk + k0 + x]) : 0.f;
        sw[j][x] = k && c0 + j < d_c ? to_f(W[static_cast<ll>(c0 + j) * n_h * d_nope + h * d_nope + k0 + x]) : 0.f;
      }
      __syncthreads();
#pragma unroll 8
      for (int k = 0; k < 32; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = fmaf(sq[y + 8 * j][k], sw[x][k], acc[j]);
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (t0 + y + 8 * j < tokens && c0 + x < d_c)
        q_lat[(static_cast<ll>(t0 + y + 8 * j) * n_h + h) * d_c + c0 + x] = acc[j];
  }
}

// out[token][h][v] = sum over c of ctx[token][h][c] W_UV[c][h d_v + v].
template <typename T>
__global__ void __launch_bounds__(256) simt_out_kernel(int tokens, int n_h, int d_c, int d_v, const float* ctx, const T* W,
                                                       T* out) {
  __shared__ float sc[32][33], sw[32][33];
  after_previous();
  const int v0 = blockIdx.x * 32, h = blockIdx.y, x = threadIdx.x & 31, y = threadIdx.x >> 5;
  for (int t0 = blockIdx.z * 32; t0 < tokens; t0 += gridDim.z * 32) {
    float acc[4] = {};
    for (int c0 = 0; c0 < d_c; c0 += 32) {
      for (int j = y; j < 32; j += 8) {
        sc[j][x] = t0 + j < tokens && c0 + x < d_c ? __ldcg(ctx + (static_cast<ll>(t0 + j) * n_h + h) * d_c + c0 + x) : 0.f;
        sw[j][x] = c0 + j < d_c && v0 + x < d_v ? to_f(W[static_cast<ll>(c0 + j) * n_h * d_v + h * d_v + v0 + x]) : 0.f;
      }
      __syncthreads();
#pragma unroll 8
      for (int k = 0; k < 32; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = fmaf(sc[y + 8 * j][k], sw[k][x], acc[j]);
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (t0 + y + 8 * j < tokens && v0 + x < d_v)
        out[(static_cast<ll>(t0 + y + 8 * j) * n_h + h) * d_v + v0 + x] = static_cast<T>(acc[j]);
  }
}

// A part walks its key tiles, 32 keys of 8 rows at a time: the tile's values in shared memory (rows of
// an odd stride, so that lanes on neighbouring keys meet no bank twice), two rows' scores a warp with a
// key a lane, then the context with columns on threads.
constexpr int SIMT_THREADS = 128;
constexpr int SIMT_COLS = 8;  // columns of a thread: d_c <= 1024
template <typename T>
__global__ void __launch_bounds__(SIMT_THREADS) simt_attn_kernel(const CacheAttn a, int d_nope, const T* q,
                                                                 const float* q_lat, float* ctx) {
  extern __shared__ float smem[];
  const int d_c = a.cache.d_c, dr = a.cache.d_rope, D = d_c + dr, stride = D | 1;
  float* sq = smem;                                 // [8][D]
  float* sk = sq + kSimtRows * D;                   // [32][stride]
  float* sp = sk + kSimtKeys * stride;              // [8][32]
  float* sa = sp + kSimtRows * kSimtKeys;           // [8] what the sums so far are scaled by
  float* sl = sa + kSimtRows;                       // [8] sums
  int2* bounds = reinterpret_cast<int2*>(sl + kSimtRows);  // [8]; an even number of floats before it
  int* bad = reinterpret_cast<int*>(bounds + kSimtRows);  // [32] a key that is not finite
  after_previous();
  const int part = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const CacheShare share = cache_share(a, part);
  if (share.begin >= share.end) return;
  int item = __ldcg(a.part_item + part);
  for (int t = share.begin; t < share.end; ++item) {
    const int item_begin = __ldcg(a.first + item), item_end = __ldcg(a.first + item + 1);
    if (item_end <= t) continue;  // no keys
    const int b = item / a.row_tiles, r0 = (item - b * a.row_tiles) * kSimtRows, rows = min(kSimtRows, a.rows - r0);
    const int2 hull = __ldcg(a.hull + item);
    const bool begins = t == item_begin, ends = item_end <= share.end;
    const int stop = min(item_end, share.end);
    __syncthreads();
    for (int e = threadIdx.x; e < kSimtRows * D; e += SIMT_THREADS) {
      const int r = e / D, k = e - r * D;
      float v = 0.f;
      if (r < rows) {
        const ll row = static_cast<ll>(b) * a.rows + r0 + r;
        v = k < d_c ? __ldcg(q_lat + row * d_c + k) : to_f(q[row * (d_nope + dr) + d_nope + k - d_c]);
      }
      sq[e] = v;
    }
    if (threadIdx.x < kSimtRows) {
      const int r = threadIdx.x;
      bounds[r] = r < rows ? cache_row_bounds(a, b, (r0 + r) / a.n_h) : make_int2(0, 0);
    }
    float acc[kSimtRows][SIMT_COLS] = {};
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    for (; t < stop; ++t) {
      const int key0 = (hull.x / kSimtKeys + (t - item_begin)) * kSimtKeys;
      __syncthreads();
      // Eight keys a warp, a lane finds the place of one; all eight's loads are under way at once.
      const int p = key0 + 8 * warp + (lane & 7);
      const bool wanted = p >= hull.x && p < hull.y;
      const ll mine = wanted ? cache_slot(a.cache, a.pages, b, p) : -1;
      uint32_t strange = wanted && mine < 0 ? 1u << (lane & 7) : 0u;  // a bit a key: it is not finite
      if (strange && lane < 8) report_page(a.status, 304);
      float* to = sk + 8 * warp * stride;
      const int bytes = a.cache.code_bytes(), blocks = a.cache.blocks();
      for (int i0 = 0; i0 < bytes; i0 += 32) {
        const int i = i0 + lane;
        uint32_t code[8], e[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const ll slot = __shfl_sync(0xffffffffu, mine, k);
          code[k] = e[k] = 0;
          if (slot >= 0 && i < bytes) {
            code[k] = __ldcg(a.cache.codes + slot * bytes + i);
            e[k] = __ldcg(a.cache.scales + slot * blocks + i / (kCacheBlock / 2));
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const bool number = e[k] <= kCacheTopScale;
          if (!number) strange |= 1u << k;
          const float2 f = codes_to_float2(code[k]);
          const float by = number ? scale_of(e[k]) : 0.f;
          if (2 * i < d_c) to[k * stride + 2 * i] = f.x * by;
          if (2 * i + 1 < d_c) to[k * stride + 2 * i + 1] = f.y * by;
        }
      }
      for (int i0 = 0; i0 < dr; i0 += 32) {
        const int i = i0 + lane;
        float x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const ll slot = __shfl_sync(0xffffffffu, mine, k);
          x[k] = slot >= 0 && i < dr ? to_f(__ldcg(static_cast<const T*>(a.cache.keys) + slot * dr + i)) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const bool number = fabsf(x[k]) <= 3.402823466e38f;
          if (!number) strange |= 1u << k;
          if (i < dr) to[k * stride + d_c + i] = number ? x[k] : 0.f;
        }
      }
      strange = __reduce_or_sync(0xffffffffu, strange);
      if (lane < 8) bad[8 * warp + lane] = (strange >> lane) & 1u;
      __syncthreads();
      float both[2] = {0.f, 0.f};
      {
        const float *x = sq + 2 * warp * D, *y = sk + lane * stride;
#pragma unroll 8
        for (int k = 0; k < D; ++k) {
          both[0] = fmaf(x[k], y[k], both[0]);
          both[1] = fmaf(x[D + k], y[k], both[1]);
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = warp * 2 + j, p = key0 + lane;
        const int2 seen = bounds[r];
        float s = both[j] * a.scale;
        if (a.mods.cap > 0.f) s = a.mods.cap * tanhf(s / a.mods.cap);
        if (a.mods.slopes) {
          const int i = (r0 + r) / a.n_h, h = (r0 + r) - i * a.n_h;
          const int at = __ldg(a.lengths + b) - a.Sq + i;
          if (r < rows) s -= __ldg(a.mods.slopes + h) * fabsf(static_cast<float>(at - p));
        }
        const bool visible = p >= seen.x && p < seen.y;
        if (visible && bad[lane]) s = __int_as_float(0x7fc00000);
        if (!visible) s = -INFINITY;
        float top = s;
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
        const float to = fmaxf(m[j], top);
        const float from = to == -INFINITY ? 0.f : to;
        const float w = visible ? expf(s - from) : 0.f;
        const float alpha = m[j] == -INFINITY ? 0.f : expf(m[j] - from);
        l[j] = l[j] * alpha + warp_sum(w);
        m[j] = to;
        sp[r * kSimtKeys + lane] = w;
        if (lane == 0) sa[r] = alpha;
      }
      __syncthreads();
#pragma unroll
      for (int c = 0; c < SIMT_COLS; ++c) {
        const int col = threadIdx.x + c * SIMT_THREADS;
        if (col >= d_c) break;
#pragma unroll
        for (int r = 0; r < kSimtRows; ++r) acc[r][c] *= sa[r];
#pragma unroll 2
        for (int k = 0; k < kSimtKeys; k += 4) {
          const float* v = sk + k * stride + col;
          const float v0 = v[0], v1 = v[stride], v2 = v[2 * stride], v3 = v[3 * stride];
#pragma unroll
          for (int r = 0; r < kSimtRows; ++r) {
            const float4 w = *reinterpret_cast<const float4*>(sp + r * kSimtKeys + k);
            acc[r][c] = fmaf(w.w, v3, fmaf(w.z, v2, fmaf(w.y, v1, fmaf(w.x, v0, acc[r][c]))));
          }
        }
      }
    }
    const bool whole = begins && ends;
    if (lane == 0)
      for (int j = 0; j < 2; ++j) sl[warp * 2 + j] = whole ? row_sum(l[j], bounds[warp * 2 + j]) : l[j];
    __syncthreads();
    const ll slot = static_cast<ll>(2 * part + (begins ? 1 : 0)) * kSimtRows;
    if (lane == 0)
      for (int j = 0; j < 2; ++j) {
        const int r = warp * 2 + j;
        if (r >= rows) continue;
        if (whole) {
          const int i = (r0 + r) / a.n_h, h = (r0 + r) - i * a.n_h;
          const float sum = sl[r];
          a.lse[(static_cast<ll>(b) * a.n_h + h) * a.Sq + i] = sum == 0.f ? -INFINITY : m[j] + logf(sum);
        } else {
          a.part_ml[slot + r] = make_float2(m[j], l[j]);
        }
      }
#pragma unroll
    for (int c = 0; c < SIMT_COLS; ++c) {
      const int col = threadIdx.x + c * SIMT_THREADS;
      if (col >= d_c) break;
#pragma unroll
      for (int r = 0; r < kSimtRows; ++r) {
        if (r >= rows) break;
        const float s = sl[r];
        if (whole)
          ctx[(static_cast<ll>(b) * a.rows + r0 + r) * d_c + col] = s != s ? s : s == 0.f ? 0.f : acc[r][c] / s;
        else
          a.part_o[(slot + r) * d_c + col] = acc[r][c];
      }
    }
  }
}

// Rows of a warp, so that the SMs hold all CTAs at once (as far as 32 rows go), and the CTAs.
struct RowDeal {
  int per;
  unsigned grid;
};
RowDeal deal_rows(const CacheRows& at) {
  const ll rows = static_cast<ll>(at.pages.B) * at.rows, warps = static_cast<ll>(ROW_CTAS) * sm_count() * ROW_WARPS;
  const ll per = std::min<ll>(std::max<ll>((rows + warps - 1) / warps, 1), 32);
  return {static_cast<int>(per), static_cast<unsigned>((rows + per * ROW_WARPS - 1) / (per * ROW_WARPS))};
}
template <typename T>
LaunchResult append(const CacheAppend& a, const RopeTable& t, cudaStream_t st) {
  const RowDeal d = deal_rows(a.at);
  const bool vec = a.cache.d_c % 16 == 0 && aligned_to_16(a.c_kv);
  LaunchResult r;
  r.err = launch_next(vec ? append_kernel<T, true> : append_kernel<T, false>, d.grid, ROW_WARPS * 32, 0, st, a, t, d.per);
  if (r.err != cudaSuccess) r.what = "cache4_append";
  return r;
}
template <typename T>
LaunchResult read(const CacheRead& a, cudaStream_t st) {
  const RowDeal d = deal_rows(a.at);
  const bool vec = a.cache.d_c % 16 == 0 && aligned_to_16(a.c_kv);
  LaunchResult r;
  r.err = launch_next(vec ? read_kernel<T, true> : read_kernel<T, false>, d.grid, ROW_WARPS * 32, 0, st, a, d.per);
  if (r.err != cudaSuccess) r.what = "cache4_read";
  return r;
}

unsigned token_tiles(const CacheAttn& a) {
  return static_cast<unsigned>(std::min((static_cast<ll>(a.pages.B) * a.Sq + 31) / 32, ll{65535}));
}

}  // namespace

LaunchResult cache4_append(const CacheAppend& a, const RopeTable& t, cudaStream_t st) {
  return a.cache.is_bf16 ? append<bf16>(a, t, st) : append<float>(a, t, st);
}
LaunchResult cache4_read(const CacheRead& a, cudaStream_t st) {
  return a.cache.is_bf16 ? read<bf16>(a, st) : read<float>(a, st);
}

LaunchResult cache4_join(const CacheAttn& a, float* ctx, cudaStream_t st) {
  LaunchResult r;
  const ll rows = static_cast<ll>(a.items()) * std::min(a.tile, a.rows);
  const dim3 grid(static_cast<unsigned>(a.items()), static_cast<unsigned>(rows > 65536 ? 8 : std::min(a.tile, a.rows)));
  r.err = launch_next(join_kernel, grid, JOIN_THREADS, 0, st, a, ctx);
  if (r.err != cudaSuccess) r.what = "cache4_join";
  return r;
}

LaunchResult cache4_simt_prepare(const CacheAttn& a, bool is_bf16, int d_nope, const void* q, const void* W_UK, float* q_lat,
                                 cudaStream_t st) {
  LaunchResult r;
  const dim3 grid((a.cache.d_c + 31) / 32 + 1, a.n_h, token_tiles(a));
  r.err = is_bf16 ? launch_next(simt_prepare_kernel<bf16>, grid, 256, 0, st, a, d_nope, static_cast<const bf16*>(q),
                                static_cast<const bf16*>(W_UK), q_lat)
                  : launch_next(simt_prepare_kernel<float>, grid, 256, 0, st, a, d_nope, static_cast<const float*>(q),
                                static_cast<const float*>(W_UK), q_lat);
  if (r.err != cudaSuccess) r.what = "cache4_simt_prepare";
  return r;
}

LaunchResult cache4_simt_out(const CacheAttn& a, bool is_bf16, int d_v, const float* ctx, const void* W_UV, void* out,
                             cudaStream_t st) {
  LaunchResult r;
  const int tokens = a.pages.B * a.Sq, d_c = a.cache.d_c;
  const dim3 grid((d_v + 31) / 32, a.n_h, token_tiles(a));
  r.err = is_bf16 ? launch_next(simt_out_kernel<bf16>, grid, 256, 0, st, tokens, a.n_h, d_c, d_v, ctx,
                                static_cast<const bf16*>(W_UV), static_cast<bf16*>(out))
                  : launch_next(simt_out_kernel<float>, grid, 256, 0, st, tokens, a.n_h, d_c, d_v, ctx,
                                static_cast<const float*>(W_UV), static_cast<float*>(out));
  if (r.err != cudaSuccess) r.what = "cache4_simt_out";
  return r;
}

LaunchResult cache4_simt_attn(const CacheAttn& a, bool is_bf16, int d_nope, const void* q, const float* q_lat, float* ctx,
                              cudaStream_t st) {
  LaunchResult r;
  const int D = a.cache.d_c + a.cache.d_rope;
  const size_t floats = static_cast<size_t>(kSimtRows) * D + kSimtKeys * (D | 1) + kSimtRows * kSimtKeys + 2 * kSimtRows;
  const size_t smem = floats * 4 + kSimtRows * 8 + kSimtKeys * 4;
  const void* kern = is_bf16 ? reinterpret_cast<const void*>(simt_attn_kernel<bf16>)
                             : reinterpret_cast<const void*>(simt_attn_kernel<float>);
  r.err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (r.err == cudaSuccess)
    r.err = is_bf16 ? launch_next(simt_attn_kernel<bf16>, a.parts, SIMT_THREADS, smem, st, a, d_nope,
                                  static_cast<const bf16*>(q), q_lat, ctx)
                    : launch_next(simt_attn_kernel<float>, a.parts, SIMT_THREADS, smem, st, a, d_nope,
                                  static_cast<const float*>(q), q_lat, ctx);
  if (r.err != cudaSuccess) r.what = "cache4_simt_attn";
  return r;
}

}  // namespace laga
