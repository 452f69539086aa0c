// The paged 4-bit latent cache: rows written and read, the sharing out of an attention call's key
// tiles and the joining of its pieces, and the attention on the CUDA cores for any widths.
//
// Writing and reading are bound by memory (a prompt) or by a launch (a token): a warp takes a row, a
// lane a block of 16 latents (at d_c = 512 each lane exactly one) and a pair of the RoPE key, so that
// the only thing that lanes exchange is the key's sum of squares.
#include "cache4.h"
#include "rope_device.cuh"

#include <cuda_fp16.h>
#include <cuda_fp4.h>

#include <algorithm>

namespace laga {
namespace {

constexpr int ROW_WARPS = 8;

__device__ __forceinline__ float scale_of(int byte) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>(byte << 7)));
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

// The code of v: its nearest multiple of s, ties to the even code. The halves between neighbours are
// few-bit multiples of s, exact in fp32.
__device__ __forceinline__ uint32_t code_for(float v, float s) {
  const float a = fabsf(v);
  uint32_t c = (a > 0.25f * s) + (a >= 0.75f * s) + (a > 1.25f * s) + (a >= 1.75f * s) + (a > 2.5f * s) +
               (a >= 3.5f * s) + (a > 5.f * s);
  return s > 0.f ? c | (v < 0.f ? 8u : 0u) : (v < 0.f ? 8u : 0u);
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
  const float s = finite ? scale_of(e) : 1.f;
  uint2 w = make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w.x |= code_for(v[i], s) << (4 * i);
    w.y |= code_for(v[8 + i], s) << (4 * i);
  }
  *scale = e;
  return finite ? w : make_uint2(0, 0);
}

// The row of the padded batch that this warp takes: its sequence, its position, its slot in the pool
// (-1: none). False past the batch.
struct CacheRow {
  int b, i;
  ll row, p, slot;
  bool stored;  // i < counts[b]
};
__device__ __forceinline__ bool cache_row(const CacheView& c, const CacheRows& at, int* status, int where, CacheRow& r) {
  r.row = static_cast<ll>(blockIdx.x) * ROW_WARPS + (threadIdx.x >> 5);
  if (r.row >= static_cast<ll>(at.pages.B) * at.rows) return false;
  r.b = static_cast<int>(r.row / at.rows);
  r.i = static_cast<int>(r.row - static_cast<ll>(r.b) * at.rows);
  r.stored = !at.counts || r.i < __ldg(at.counts + r.b);
  r.p = static_cast<ll>(__ldg(at.starts + r.b)) + r.i;
  r.slot = r.stored ? cache_slot(c, at.pages, r.b, r.p) : -1;
  if (r.stored && r.slot < 0 && (threadIdx.x & 31) == 0) report_page(status, where);
  return true;
}

// VEC: d_c a multiple of 16 and the latents 16-byte aligned.
template <typename T, bool VEC>
__global__ void __launch_bounds__(ROW_WARPS * 32) append_kernel(const CacheAppend a, const RopeTable t) {
  after_previous();
  CacheRow r;
  if (!cache_row(a.cache, a.at, a.status, 301, r) || r.slot < 0) return;
  const int lane = threadIdx.x & 31, d_c = a.cache.d_c, bytes = a.cache.code_bytes();
  const T* c = static_cast<const T*>(a.c_kv) + r.row * d_c;
  uint8_t* codes = a.cache.codes + r.slot * bytes;
  uint8_t* scales = a.cache.scales + r.slot * a.cache.blocks();
  for (int k = lane; k < a.cache.blocks(); k += 32) {
    float v[16];
    if constexpr (VEC) {
      constexpr int N = Vec<T>::N;
#pragma unroll
      for (int j = 0; j < 16 / N; ++j) {
        float x[N];
        Vec<T>::get(__ldcs(reinterpret_cast<const uint4*>(c + k * 16) + j), x);
#pragma unroll
        for (int i = 0; i < N; ++i) v[j * N + i] = x[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = k * 16 + i < d_c ? to_f(c[k * 16 + i]) : 0.f;
    }
    int e;
    const uint2 w = encode_block(v, &e);
    scales[k] = static_cast<uint8_t>(e);
    if constexpr (VEC) {
      *reinterpret_cast<uint2*>(codes + k * 8) = w;
    } else {
      for (int j = 0; j < 8 && k * 8 + j < bytes; ++j)
        codes[k * 8 + j] = static_cast<uint8_t>((j < 4 ? w.x : w.y) >> (8 * (j & 3)));
    }
  }
  const int dr = a.cache.d_rope, n = dr / 2;
  if (dr == 0) return;
  const T* x = static_cast<const T*>(a.k_rope) + r.row * dr;
  T* out = static_cast<T*>(a.cache.keys) + r.slot * dr;
  const T* w = static_cast<const T*>(a.w_k);
  float down = 1.f, f = 1.f;
  if (w) {
    float sum = 0.f;
    for (int i = lane; i < dr; i += 32) sum = fmaf(to_f(x[i]), to_f(x[i]), sum);
    sum = warp_sum(sum);
    if (!(sum < 0x1p120f)) {  // squares that may have left fp32
      down = 0x1p-70f;
      sum = 0.f;
      for (int i = lane; i < dr; i += 32) sum = fmaf(to_f(x[i]) * down, to_f(x[i]) * down, sum);
      sum = warp_sum(sum);
    }
    f = rsqrtf(fmaf(sum, 1.f / dr, a.eps * down * down));
  }
  auto value = [&](int i) { return w ? to_f(x[i]) * down * f * to_f(w[i]) : to_f(x[i]); };
  if (!a.turn) {
    for (int i = lane; i < dr; i += 32) out[i] = static_cast<T>(value(i));
    return;
  }
  for (int u = lane; u < n; u += 32) {
    ll p = r.p;
    if (a.own_pos) {
      const ll at = t.axis[u] * a.rope.tokens + r.row;
      p = a.rope.pos64 ? static_cast<const ll*>(a.rope.pos)[at] : static_cast<ll>(static_cast<const int*>(a.rope.pos)[at]);
    }
    const float2 cs = cos_sin(p, t.turns[u]);
    const int i0 = a.rope.interleaved ? 2 * u : u, i1 = a.rope.interleaved ? 2 * u + 1 : n + u;
    const float y0 = value(i0), y1 = value(i1);
    out[i0] = static_cast<T>(y0 * cs.x - y1 * cs.y);
    out[i1] = static_cast<T>(y0 * cs.y + y1 * cs.x);
  }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(ROW_WARPS * 32) read_kernel(const CacheRead a) {
  after_previous();
  CacheRow r;
  if (!cache_row(a.cache, a.at, a.status, 302, r)) return;
  const int lane = threadIdx.x & 31, d_c = a.cache.d_c, dr = a.cache.d_rope;
  T* c = static_cast<T*>(a.c_kv) + r.row * d_c;
  T* key = static_cast<T*>(a.k_rope) + r.row * dr;
  const float fill = r.stored ? __int_as_float(0x7fc00000) : 0.f;  // a row that the table has no page for: NaN
  if (r.slot < 0) {
    for (int i = lane; i < d_c; i += 32) c[i] = static_cast<T>(fill);
    for (int i = lane; i < dr; i += 32) key[i] = static_cast<T>(fill);
    return;
  }
  const uint8_t* codes = a.cache.codes + r.slot * a.cache.code_bytes();
  const uint8_t* scales = a.cache.scales + r.slot * a.cache.blocks();
  const T* from = static_cast<const T*>(a.cache.keys) + r.slot * dr;
  for (int i = lane; i < dr; i += 32) key[i] = from[i];
  if constexpr (VEC) {
    constexpr int N = Vec<T>::N;
    for (int k = lane; k < a.cache.blocks(); k += 32) {
      const uint2 w = *reinterpret_cast<const uint2*>(codes + k * 8);
      const float s = scale_of(scales[k]);
      float v[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 f = codes_to_float2(((j < 4 ? w.x : w.y) >> (8 * (j & 3))) & 0xffu);
        v[2 * j] = f.x * s;
        v[2 * j + 1] = f.y * s;
      }
#pragma unroll
      for (int j = 0; j < 16 / N; ++j) {
        float x[N];
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = v[j * N + i];
        reinterpret_cast<uint4*>(c + k * 16)[j] = Vec<T>::put(x);
      }
    }
  } else {
    for (int i = lane; i < d_c; i += 32) {
      const float2 f = codes_to_float2(codes[i >> 1]);
      c[i] = static_cast<T>((i & 1 ? f.y : f.x) * scale_of(scales[i / kCacheBlock]));
    }
  }
}

// ---------------------------------------------------------------- sharing out and joining

__global__ void __launch_bounds__(1024) plan_kernel(const CacheAttn a) {
  after_previous();
  cache4_plan_items<1024>(a);
}

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
  const int2 hull = __ldcg(a.hull + item);
  const int rows = min(a.tile, a.rows - r0), d_c = a.cache.d_c, pieces = p1 - p0 + 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int r = blockIdx.y; r < rows; r += gridDim.y) {
    const ll row = static_cast<ll>(b) * a.rows + r0 + r;
    const int i = (r0 + r) / a.n_h, h = (r0 + r) - i * a.n_h;
    float* out = ctx + row * d_c;
    float* lse = a.lse + (static_cast<ll>(b) * a.n_h + h) * a.Sq + i;
    if (end == begin) {  // no keys: zero, or NaN where the table had no room
      const float v = hull.x < 0 ? __int_as_float(0x7fc00000) : 0.f;
      for (int c = threadIdx.x; c < d_c; c += JOIN_THREADS) out[c] = v;
      if (threadIdx.x == 0) *lse = hull.x < 0 ? v : -INFINITY;
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
template <typename T>
__global__ void __launch_bounds__(256) simt_qlat_kernel(int tokens, int n_h, int d_c, int d_nope, int d_qk, const T* q,
                                                        const T* W, float* q_lat) {
  __shared__ float sq[32][33], sw[32][33];
  after_previous();
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
      if (threadIdx.x < kSimtKeys) bad[threadIdx.x] = 0;
      __syncthreads();
      for (int k = warp; k < kSimtKeys; k += SIMT_THREADS / 32) {
        float* to = sk + k * stride;
        const int p = key0 + k;
        const ll slot = p >= hull.x && p < hull.y ? cache_slot(a.cache, a.pages, b, p) : -1;
        if (slot < 0) {
          for (int i = lane; i < D; i += 32) to[i] = 0.f;
          if (lane == 0 && p >= hull.x && p < hull.y) {
            bad[k] = 1;
            report_page(a.status, 304);
          }
          continue;
        }
        const uint8_t* codes = a.cache.codes + slot * a.cache.code_bytes();
        const uint8_t* scales = a.cache.scales + slot * a.cache.blocks();
        const T* key = static_cast<const T*>(a.cache.keys) + slot * dr;
        bool fine = true;
        for (int i = lane; i < (d_c + 1) / 2; i += 32) {
          const int e = scales[i / (kCacheBlock / 2)];
          const float2 f = codes_to_float2(codes[i]);
          const float s = scale_of(e);
          fine = fine && e <= kCacheTopScale;
          to[2 * i] = f.x * s;
          if (2 * i + 1 < d_c) to[2 * i + 1] = f.y * s;
        }
        for (int i = lane; i < dr; i += 32) {
          const float v = to_f(key[i]);
          fine = fine && fabsf(v) <= 3.402823466e38f;
          to[d_c + i] = v;
        }
        if (!__all_sync(0xffffffffu, fine)) {
          for (int i = lane; i < D; i += 32) to[i] = 0.f;
          if (lane == 0) bad[k] = 1;
        }
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = warp * 2 + j, p = key0 + lane;
        const int2 seen = bounds[r];
        float s = 0.f;
        const float* x = sq + r * D;
        const float* y = sk + lane * stride;
        for (int k = 0; k < D; ++k) s = fmaf(x[k], y[k], s);
        s *= a.scale;
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
        for (int k = 0; k < kSimtKeys; ++k) {
          const float v = sk[k * stride + col];
#pragma unroll
          for (int r = 0; r < kSimtRows; ++r) acc[r][c] = fmaf(sp[r * kSimtKeys + k], v, acc[r][c]);
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

template <typename T>
LaunchResult append(const CacheAppend& a, const RopeTable& t, cudaStream_t st) {
  const ll rows = static_cast<ll>(a.at.pages.B) * a.at.rows;
  const unsigned grid = static_cast<unsigned>((rows + ROW_WARPS - 1) / ROW_WARPS);
  const bool vec = a.cache.d_c % 16 == 0 && aligned_to_16(a.c_kv);
  LaunchResult r;
  r.err = launch_next(vec ? append_kernel<T, true> : append_kernel<T, false>, grid, ROW_WARPS * 32, 0, st, a, t);
  if (r.err != cudaSuccess) r.what = "cache4_append";
  return r;
}
template <typename T>
LaunchResult read(const CacheRead& a, cudaStream_t st) {
  const ll rows = static_cast<ll>(a.at.pages.B) * a.at.rows;
  const unsigned grid = static_cast<unsigned>((rows + ROW_WARPS - 1) / ROW_WARPS);
  const bool vec = a.cache.d_c % 16 == 0 && aligned_to_16(a.c_kv);
  LaunchResult r;
  r.err = launch_next(vec ? read_kernel<T, true> : read_kernel<T, false>, grid, ROW_WARPS * 32, 0, st, a);
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

LaunchResult cache4_plan(const CacheAttn& a, cudaStream_t st) {
  LaunchResult r;
  r.err = launch_next(plan_kernel, 1, 1024, 0, st, a);
  if (r.err != cudaSuccess) r.what = "cache4_plan";
  return r;
}

LaunchResult cache4_join(const CacheAttn& a, float* ctx, cudaStream_t st) {
  LaunchResult r;
  const ll rows = static_cast<ll>(a.items()) * std::min(a.tile, a.rows);
  const dim3 grid(static_cast<unsigned>(a.items()), static_cast<unsigned>(rows > 65536 ? 8 : std::min(a.tile, a.rows)));
  r.err = launch_next(join_kernel, grid, JOIN_THREADS, 0, st, a, ctx);
  if (r.err != cudaSuccess) r.what = "cache4_join";
  return r;
}

LaunchResult cache4_simt_qlat(const CacheAttn& a, bool is_bf16, int d_nope, const void* q, const void* W_UK, float* q_lat,
                              cudaStream_t st) {
  LaunchResult r;
  const int tokens = a.pages.B * a.Sq, d_c = a.cache.d_c, d_qk = d_nope + a.cache.d_rope;
  const dim3 grid((d_c + 31) / 32, a.n_h, token_tiles(a));
  r.err = is_bf16 ? launch_next(simt_qlat_kernel<bf16>, grid, 256, 0, st, tokens, a.n_h, d_c, d_nope, d_qk,
                                static_cast<const bf16*>(q), static_cast<const bf16*>(W_UK), q_lat)
                  : launch_next(simt_qlat_kernel<float>, grid, 256, 0, st, tokens, a.n_h, d_c, d_nope, d_qk,
                                static_cast<const float*>(q), static_cast<const float*>(W_UK), q_lat);
  if (r.err != cudaSuccess) r.what = "cache4_simt_qlat";
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
