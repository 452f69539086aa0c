// What the masked attention runs before its kernels: the visible interval of every
// query row, the tiles that follow from it, and copies of the inputs in which rows
// holding a non-finite value (in the latent: one that its rebuild may make non-finite) are zero.
//
// Why the copies: the attention kernels give a masked score the weight 0 and then
// multiply it by the key's V row (forward), or by the query's q and dO rows (dK, dV).
// 0 times a NaN is a NaN, so one uninitialised padding row would reach every row of
// its tile. With such rows zeroed a masked weight contributes exactly nothing; the
// query rows that do see such a key, and the keys that are seen by such a query, get
// NaN through the row statistics instead (rows' bit 31 in the forward, lse in the
// backward). The latent is small (d_c + d_rope values per key, shared by all heads),
// so its copy is always made: 2 x 19 MB at 16384 keys. q and dout are copied only when
// a row of theirs is non-finite, which the pass that computes D sees.
//
// All of it is launches and latency, not work: the two launches take 11 us for 519 keys and 15
// for 2 x 4096 (rows, keys and tiles in a launch each took 18 and 23).
#include "internal.h"
#include "mask.h"

#include <type_traits>

namespace laga {
namespace {

using ll = long long;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ bool finite(float v) { return (__float_as_uint(v) & 0x7f800000u) != 0x7f800000u; }
// The largest size of a latent or RoPE value that counts as finite: beyond it the rebuilt K and V may
// not be (below it they are while no column of the weights adds up to 2^16), and 0 times an infinite V
// is a NaN. Uninitialised padding holds 3e38 as readily as a NaN, and some masks fill with the type's lowest value.
constexpr float kLatentMax = 0x1p112f;
__device__ __forceinline__ bool latent_ok(float v) { return fabsf(v) <= kLatentMax; }  // false for a NaN
// whether any of eight packed bf16 of a latent row is not
__device__ __forceinline__ bool bad_latent_x2(uint32_t w) {
  constexpr uint32_t top = (112u + 127u) << 7;  // kLatentMax as bf16
  return (w & 0x7fffu) > top || (w & 0x7fff0000u) > top << 16;
}
__device__ __forceinline__ bool bad_latent_x8(uint4 v) {
  return bad_latent_x2(v.x) || bad_latent_x2(v.y) || bad_latent_x2(v.z) || bad_latent_x2(v.w);
}
// whether any of eight packed bf16 is infinite or NaN
__device__ __forceinline__ bool bad_bf16x2(uint32_t w) {
  return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ bool bad_bf16x8(uint4 v) {
  return bad_bf16x2(v.x) || bad_bf16x2(v.y) || bad_bf16x2(v.z) || bad_bf16x2(v.w);
}

// Latent rows -> clean copies; one CTA (unit) per 32 keys of a batch element, a warp for four of
// them. bad[b][word] bit r: key 32 * word + r holds a value that does not count as finite.
// The tensor-core dims: the four rows' 72 16-byte chunks each are loaded before the first is
// looked at (row by row the kernel took 11 us however few keys there were).
constexpr int KEY_ROWS = 4;

__device__ __forceinline__ void clean_keys_tc(int S, int unit, int units, const bf16* __restrict__ c,
                                              const bf16* __restrict__ r, bf16* __restrict__ c_out,
                                              bf16* __restrict__ r_out, uint32_t* __restrict__ bad) {
  constexpr int NC = 64, NR = 8;  // chunks of a latent row (512 values), of a RoPE key (64)
  __shared__ uint32_t warp_bad[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.y;
  const int j0 = unit * 32 + warp * KEY_ROWS;
  const uint4* cs = reinterpret_cast<const uint4*>(c) + (static_cast<ll>(b) * S + j0) * NC;
  const uint4* rs = reinterpret_cast<const uint4*>(r) + (static_cast<ll>(b) * S + j0) * NR;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  uint4 v[KEY_ROWS][2], w;
#pragma unroll
  for (int k = 0; k < KEY_ROWS; ++k)
#pragma unroll
    for (int i = 0; i < 2; ++i) v[k][i] = j0 + k < S ? cs[k * NC + 32 * i + lane] : zero;
  w = j0 + (lane >> 3) < S ? rs[lane] : zero;  // the four RoPE keys, eight lanes each
  const unsigned rope_bad = __ballot_sync(0xffffffffu, bad_latent_x8(w));
  uint32_t mask = 0u;
#pragma unroll
  for (int k = 0; k < KEY_ROWS; ++k)
    if (__any_sync(0xffffffffu, bad_latent_x8(v[k][0]) || bad_latent_x8(v[k][1])) || (rope_bad & (0xffu << (8 * k)))) mask |= 1u << k;
  uint4* cd = reinterpret_cast<uint4*>(c_out) + (static_cast<ll>(b) * S + j0) * NC;
  uint4* rd = reinterpret_cast<uint4*>(r_out) + (static_cast<ll>(b) * S + j0) * NR;
#pragma unroll
  for (int k = 0; k < KEY_ROWS; ++k)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (j0 + k < S) cd[k * NC + 32 * i + lane] = (mask >> k) & 1u ? zero : v[k][i];
  if (j0 + (lane >> 3) < S) rd[lane] = (mask >> (lane >> 3)) & 1u ? zero : w;
  if (lane == 0) warp_bad[warp] = mask << (KEY_ROWS * warp);
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t m = 0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) m |= warp_bad[k];
    bad[static_cast<ll>(b) * units + unit] = m;
  }
}

// Any widths: one value a lane.
template <typename T>
__device__ __forceinline__ void clean_keys(int S, int unit, int units, int d_c, int d_rope, const T* __restrict__ c,
                                           const T* __restrict__ r, T* __restrict__ c_out, T* __restrict__ r_out,
                                           uint32_t* __restrict__ bad) {
  __shared__ uint32_t warp_bad[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.y;
  const int j0 = unit * 32 + warp * KEY_ROWS;
  uint32_t mask = 0u;
  auto sweep = [&](int width, const T* src, T* dst, bool write) {
    const T* from = src + (static_cast<ll>(b) * S + j0) * width;
    T* to = dst + (static_cast<ll>(b) * S + j0) * width;
    for (int i = lane; i < ((width + 31) & ~31); i += 32) {
      T v[KEY_ROWS];
#pragma unroll
      for (int k = 0; k < KEY_ROWS; ++k)
        v[k] = i < width && j0 + k < S ? from[static_cast<ll>(k) * width + i] : static_cast<T>(0.f);
#pragma unroll
      for (int k = 0; k < KEY_ROWS; ++k) {
        if (!write) {
          if (__any_sync(0xffffffffu, !latent_ok(to_f(v[k])))) mask |= 1u << k;
        } else if (i < width && j0 + k < S) {
          to[static_cast<ll>(k) * width + i] = (mask >> k) & 1u ? static_cast<T>(0.f) : v[k];
        }
      }
    }
  };
  sweep(d_c, c, c_out, false);
  sweep(d_rope, r, r_out, false);
  sweep(d_c, c, c_out, true);  // the second reading hits the caches
  sweep(d_rope, r, r_out, true);
  if (lane == 0) warp_bad[warp] = mask << (KEY_ROWS * warp);
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t m = 0u;
#pragma unroll
    for (int k = 0; k < 8; ++k) m |= warp_bad[k];
    bad[static_cast<ll>(b) * units + unit] = m;
  }
}

__device__ __forceinline__ int position(const Dims& d, int i) {
  return (d.q_split > 0 && i >= d.q_split) ? d.q_offset2 + (i - d.q_split) : d.q_offset + i;
}

// The visible intervals of 256 query rows (two 128-row tiles) of a batch element: thread = row.
__device__ __forceinline__ void row_intervals(const Dims& d, int unit, const int* __restrict__ key_lo,
                                              const int* __restrict__ key_hi, int2* __restrict__ rows,
                                              int2* __restrict__ q_tiles, int2* __restrict__ q_hull) {
  __shared__ int s_lo[8], s_hi[8];
  const int b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = unit * 256 + threadIdx.x;
  int lo = 0, hi = 0;
  if (i < d.Sq) {
    const ll at = static_cast<ll>(b) * d.Sq + i;
    lo = key_lo ? max(0, key_lo[at]) : 0;
    hi = key_hi ? min(d.S, key_hi[at]) : d.S;
    if (d.causal) hi = min(hi, position(d, i) + 1);
    if (lo >= hi) lo = hi = 0;
  }
  if (i < d.sq_pad) rows[static_cast<ll>(b) * d.sq_pad + i] = make_int2(lo, hi);
  const bool some = lo < hi;
  const int wlo = __reduce_min_sync(0xffffffffu, some ? lo : 0x7fffffff);
  const int whi = __reduce_max_sync(0xffffffffu, some ? hi : 0);
  if (lane == 0) {
    s_lo[warp] = wlo;
    s_hi[warp] = whi;
  }
  __syncthreads();
  const int k = threadIdx.x, tile = unit * 2 + (k >> 1);
  if (k >= 4 || tile * 128 >= d.sq_pad) return;
  q_hull[static_cast<ll>(b) * (d.sq_pad / 64) + unit * 4 + k] =
      make_int2(min(s_lo[2 * k], s_lo[2 * k + 1]), max(s_hi[2 * k], s_hi[2 * k + 1]));
  if (k & 1) return;
  const int l = min(min(s_lo[2 * k], s_lo[2 * k + 1]), min(s_lo[2 * k + 2], s_lo[2 * k + 3]));
  const int h = max(max(s_hi[2 * k], s_hi[2 * k + 1]), max(s_hi[2 * k + 2], s_hi[2 * k + 3]));
  // a tile whose rows see nothing still walks one (wholly masked) key tile
  const int first = l < h ? l / 128 : 0, end = l < h ? (h + 127) / 128 : 1;
  q_tiles[static_cast<ll>(b) * (d.sq_pad / 128) + tile] = make_int2(first, end - first);
}

// Rows and keys of all batch elements in one launch: the first CTAs take the rows, 256 each, the
// others the keys, 32 each. TC: the tensor-core dims. One launch, because in small calls a launch
// is most of what any of this costs.
template <typename T, bool TC>
__global__ void __launch_bounds__(256)
    mask_inputs_kernel(const __grid_constant__ Dims d, const int* __restrict__ key_lo, const int* __restrict__ key_hi,
                       const T* __restrict__ c, const T* __restrict__ r, const __grid_constant__ MaskBuffers m) {
  after_previous();
  const int row_units = (d.sq_pad + 255) / 256, units = static_cast<int>(gridDim.x) - row_units;
  const int unit = static_cast<int>(blockIdx.x) - row_units;
  if (unit < 0) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *m.q_bad = m.counters[0] = m.counters[1] = m.counters[2] = 0;
    row_intervals(d, blockIdx.x, key_lo, key_hi, m.rows, m.q_tiles, m.q_hull);
  } else if constexpr (TC) {
    clean_keys_tc(d.S, unit, units, c, r, reinterpret_cast<bf16*>(m.c_kv), reinterpret_cast<bf16*>(m.k_rope), m.bad);
  } else {
    clean_keys(d.S, unit, units, d.d_c, d.d_rope, c, r, reinterpret_cast<T*>(m.c_kv), reinterpret_cast<T*>(m.k_rope), m.bad);
  }
}

// One CTA per batch element. First, only if one of its keys is bad: bit 31 of the rows that see
// such a key. Then, a warp per 128-key tile in turn: the 64-row query tiles whose hull meets it, in
// order. The CTA that finishes last lists the key tiles (of all batch
// elements, in order) that some query tile's walk touches: only those are rebuilt, and only
// their gradients summed.
__global__ void __launch_bounds__(1024) mask_tiles_kernel(int kt, int nq64, const uint32_t* __restrict__ bad,
                                                          int bad_words, int2* __restrict__ rows,
                                                          const int2* __restrict__ q_tiles,
                                                          const int2* __restrict__ q_hull, int* __restrict__ kt_count,
                                                          int* __restrict__ kt_list, int* __restrict__ seen,
                                                          int* __restrict__ seen_list, int* __restrict__ counters,
                                                          int4* __restrict__ work) {
  after_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.x;
  const uint32_t* words = bad + static_cast<ll>(b) * bad_words;
  bool any = false;
  for (int w = threadIdx.x; w < bad_words; w += 1024) any |= words[w] != 0u;
  if (__syncthreads_or(any))
    for (int i = threadIdx.x; i < nq64 * 64; i += 1024) {
      int2& row = rows[static_cast<ll>(b) * nq64 * 64 + i];
      if (sees_bad_key(words, row.x, row.y, 0, 1)) row.x |= static_cast<int>(0x80000000u);
    }
  const int2* hull = q_hull + static_cast<ll>(b) * nq64;
  const int2* walk = q_tiles + static_cast<ll>(b) * (nq64 / 2);
  for (int t = warp; t < kt; t += 32) {
    const ll at = static_cast<ll>(b) * kt + t;
    int* list = kt_list + at * nq64;
    int n = 0;
    bool touched = false;
    for (int q0 = 0; q0 < nq64; q0 += 32) {
      const int q = q0 + lane;
      bool meets = false;
      if (q < nq64) {
        const int2 v = hull[q], w = walk[q >> 1];
        meets = v.x < v.y && v.x < (t + 1) * 128 && v.y > t * 128;
        touched |= w.x <= t && t < w.x + w.y;
      }
      const unsigned m = __ballot_sync(0xffffffffu, meets);
      if (meets) list[n + __popc(m & ((1u << lane) - 1u))] = q;
      n += __popc(m);
    }
    touched = __any_sync(0xffffffffu, touched);
    if (lane == 0) {
      kt_count[at] = n;
      seen[at] = touched ? 1 : 0;
    }
  }
  // the query tiles by the length of their walk, longest first (ties by number)
  const int nq = nq64 / 2;
  for (int q = threadIdx.x; q < nq; q += 1024) {
    const int2 w = walk[q];
    int rank = 0;
    for (int o = 0; o < nq; ++o) {
      const int n = walk[o].y;
      rank += n > w.y || (n == w.y && o < q);
    }
    work[static_cast<ll>(b) * nq + rank] = make_int4(q, w.x, w.y, 0);
  }
  __shared__ bool last;
  __shared__ int warp_n[32];
  if (gridDim.x > 1) __threadfence();
  __syncthreads();
  if (gridDim.x > 1) {  // a batch of one needs no count of its CTAs
    if (threadIdx.x == 0) last = atomicAdd(&counters[1], 1) == static_cast<int>(gridDim.x) - 1;
    __syncthreads();
    if (!last) return;
    __threadfence();
  }
  const int total = kt * static_cast<int>(gridDim.x);
  int base = 0;
  for (int i0 = 0; i0 < total; i0 += 1024) {
    const int i = i0 + static_cast<int>(threadIdx.x);
    const bool in = i < total && __ldcg(seen + i) != 0;
    const unsigned m = __ballot_sync(0xffffffffu, in);
    if (lane == 0) warp_n[warp] = __popc(m);
    __syncthreads();
    const int n = warp_n[lane];
    const int before = base + __reduce_add_sync(0xffffffffu, lane < warp ? n : 0);
    const int all = __reduce_add_sync(0xffffffffu, n);
    if (in) seen_list[before + __popc(m & ((1u << lane) - 1u))] = i;
    base += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) counters[0] = base;
}

// key_lo, key_hi of packed documents: one thread per query row.
__global__ void key_bounds_kernel(Dims d, const int* __restrict__ starts, int n_docs, const int* __restrict__ prefix,
                                  int window, int* __restrict__ key_lo, int* __restrict__ key_hi) {
  after_previous();
  const int i = blockIdx.x * blockDim.x + threadIdx.x, b = blockIdx.y;
  if (i >= d.Sq) return;
  const int pos = position(d, i);
  const int* s = starts + static_cast<ll>(b) * (n_docs + 1);
  int a = 0, z = n_docs + 1;  // entries <= pos: the last of them starts the row's document
  while (a < z) {
    const int m = (a + z) >> 1;
    if (s[m] <= pos)
      a = m + 1;
    else
      z = m;
  }
  const int doc = a - 1;
  int lo = 0, hi = 0;
  if (doc >= 0 && doc < n_docs) {
    const int first = s[doc], last = min(s[doc + 1], d.S);
    lo = max(first, 0);
    if (window > 0 && pos - window + 1 > lo) lo = pos - window + 1;
    hi = pos + 1;
    if (prefix) {
      const ll end = static_cast<ll>(first) + prefix[static_cast<ll>(b) * n_docs + doc];
      if (end > hi) hi = end < last ? static_cast<int>(end) : last;
    }
    hi = min(hi, last);
  }
  const ll at = static_cast<ll>(b) * d.Sq + i;
  key_lo[at] = lo;
  key_hi[at] = hi;
}

// ---- the backward's row pass, tensor-core dims: 8 lanes per (b, h, i) of the padded rows.
// lse2 = lse log2(e) (+inf: the row sees nothing or does not exist; NaN: its q, dout or
// forward result is not finite), delta = rowsum(dout out), *q_bad if q or dout is not finite.
// PACKED: q and out come from their 8-bit checkpoints; q is written in bf16 to q_clean (zero
// if the row is bad), out is only summed. Otherwise q is read for its finiteness alone: with a
// cap (CHECK_Q) always, else only where lse is not finite, because every score of a row whose q
// is not finite is not finite, and so is its lse (a cap makes finite scores of infinite ones).
// That leaves 3 of 7 bytes unread (q has 192 values a row, dout and out 128 each). Bound by
// memory: 2 x 4096 rows of 16 heads, 67 MB, in 15 us with everything from DRAM (16 lanes a row: 18,
// bound by instructions).
template <bool PACKED, bool CHECK_Q>
__global__ void __launch_bounds__(256) mask_bwd_pre_kernel(Dims d, const bf16* __restrict__ q, const bf16* __restrict__ out,
                                                           const Packed q8, const Packed out8,
                                                           const bf16* __restrict__ dout,
                                                           const float* __restrict__ lse, float* __restrict__ lse2,
                                                           float* __restrict__ delta, bf16* __restrict__ q_clean,
                                                           int* __restrict__ q_bad, bool beside) {
  if (beside)
    beside_previous();
  else
    after_previous();
  const ll row = (static_cast<ll>(blockIdx.x) * blockDim.x + threadIdx.x) >> 3;
  const ll rows = static_cast<ll>(d.B) * d.sq_pad * d.n_h;
  const int l8 = threadIdx.x & 7;
  // heads fastest: neighbouring rows are neighbours in q, out and dout
  int h, i, b;
  if (rows < (ll(1) << 31)) {  // cheaper divisions
    const uint32_t r = static_cast<uint32_t>(row), bi = r / static_cast<uint32_t>(d.n_h);
    h = static_cast<int>(r - bi * d.n_h);
    b = static_cast<int>(bi / static_cast<uint32_t>(d.sq_pad));
    i = static_cast<int>(bi - b * static_cast<uint32_t>(d.sq_pad));
  } else {
    const ll bi = row / d.n_h;
    h = static_cast<int>(row - bi * d.n_h);
    b = static_cast<int>(bi / d.sq_pad);
    i = static_cast<int>(bi - static_cast<ll>(b) * d.sq_pad);
  }
  const bool in = row < rows && i < d.Sq;
  const ll src = (static_cast<ll>(b) * d.Sq + i) * d.n_h + h;
  float acc = 0.f;
  bool bad = false;
  uint4 qv[3] = {};  // 16-byte chunks l8, l8 + 8, ... of the row's q
  const float row_lse = in ? __ldcg(&lse[(static_cast<ll>(b) * d.n_h + h) * d.Sq + i]) : -INFINITY;
  if (in) {
    uint4 g[2], a[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) g[c] = __ldcg(reinterpret_cast<const uint4*>(dout + src * 128) + l8 + 8 * c);
    if constexpr (PACKED) {
#pragma unroll
      for (int c = 0; c < 2; ++c) a[c] = unpack8_bf16x8(out8, src, 128, l8 + 8 * c);
#pragma unroll
      for (int c = 0; c < 3; ++c) qv[c] = unpack8_bf16x8(q8, src, 192, l8 + 8 * c);
    } else {
#pragma unroll
      for (int c = 0; c < 2; ++c) a[c] = __ldcg(reinterpret_cast<const uint4*>(out + src * 128) + l8 + 8 * c);
      if (CHECK_Q || !finite(row_lse)) {
#pragma unroll
        for (int c = 0; c < 3; ++c) qv[c] = __ldcg(reinterpret_cast<const uint4*>(q + src * 192) + l8 + 8 * c);
      }
    }
    if (PACKED || CHECK_Q || !finite(row_lse)) bad = bad_bf16x8(qv[0]) || bad_bf16x8(qv[1]) || bad_bf16x8(qv[2]);
    float zero = 0.f;  // NaN once a value of dout is not finite: one multiply-add a value, where bit tests take two
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const __nv_bfloat162* a2 = reinterpret_cast<const __nv_bfloat162*>(&a[c]);
      const __nv_bfloat162* g2 = reinterpret_cast<const __nv_bfloat162*>(&g[c]);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 af = __bfloat1622float2(a2[k]);
        const float2 gf = __bfloat1622float2(g2[k]);
        acc = fmaf(af.x, gf.x, acc);
        acc = fmaf(af.y, gf.y, acc);
        zero = fmaf(gf.x, 0.f, fmaf(gf.y, 0.f, zero));
      }
    }
    bad = bad || zero != 0.f;
  }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  const unsigned votes = __ballot_sync(0xffffffffu, bad);
  bad = ((votes >> (threadIdx.x & 24)) & 0xffu) != 0u;
  if (PACKED && in) {
    uint4* dst = reinterpret_cast<uint4*>(q_clean + src * 192);
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int c = 0; c < 3; ++c) dst[l8 + 8 * c] = bad ? zero : qv[c];
  }
  if (row < rows && l8 == 0) {
    float L = INFINITY, D = 0.f;
    if (in) {
      const float v = row_lse;
      if (v == -INFINITY) {
        L = INFINITY;  // the row sees nothing: its weights are 0
      } else if (bad || !finite(v) || !finite(acc)) {
        L = NAN;
      } else {
        L = v * 1.4426950408889634f;
        D = acc;
      }
      if (bad) *q_bad = 1;
    }
    const ll at = (static_cast<ll>(b) * d.n_h + h) * d.sq_pad + i;
    lse2[at] = L;
    delta[at] = D;
  }
  if (beside) end_after_previous(blockIdx.x == gridDim.x - 1);
}

// Runs only when *q_bad is set: clean copies of q (unless it was unpacked already) and dout.
__global__ void __launch_bounds__(256) mask_clean_kernel(ll rows, const bf16* __restrict__ q,
                                                         const bf16* __restrict__ dout, bf16* __restrict__ q_clean,
                                                         bf16* __restrict__ dout_clean, const int* __restrict__ q_bad) {
  after_previous();
  if (*q_bad == 0) return;
  const int l16 = threadIdx.x & 15;
  const ll step = (static_cast<ll>(gridDim.x) * blockDim.x) >> 4;
  for (ll row0 = ((static_cast<ll>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5) << 1; row0 < rows; row0 += step) {
    const ll row = row0 + ((threadIdx.x >> 4) & 1);
    const bool in = row < rows;
    uint4 q0 = make_uint4(0u, 0u, 0u, 0u), q1 = q0, g = q0;
    bool bad = false;
    if (in) {
      g = reinterpret_cast<const uint4*>(dout + row * 128)[l16];
      bad = bad_bf16x8(g);
      if (q) {
        q0 = reinterpret_cast<const uint4*>(q + row * 192)[l16];
        if (l16 < 8) q1 = reinterpret_cast<const uint4*>(q + row * 192)[16 + l16];
        bad |= bad_bf16x8(q0) || bad_bf16x8(q1);
      }
    }
    const unsigned votes = __ballot_sync(0xffffffffu, bad);
    bad = (votes & (threadIdx.x & 16 ? 0xffff0000u : 0xffffu)) != 0u;
    if (in) {
      const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
      reinterpret_cast<uint4*>(dout_clean + row * 128)[l16] = bad ? zero : g;
      if (q) {
        reinterpret_cast<uint4*>(q_clean + row * 192)[l16] = bad ? zero : q0;
        if (l16 < 8) reinterpret_cast<uint4*>(q_clean + row * 192)[16 + l16] = bad ? zero : q1;
      }
    }
  }
}

// ---- the same for any widths, to fp32 copies: a warp per (b, i, h) row.
template <typename T>
__global__ void __launch_bounds__(256) mask_bwd_pre_any_kernel(Dims d, const T* __restrict__ q, const T* __restrict__ out,
                                                               const Packed q8, const Packed out8, bool packed,
                                                               const T* __restrict__ dout, const float* __restrict__ lse,
                                                               float* __restrict__ lse_row, float* __restrict__ delta,
                                                               float* __restrict__ q_clean, float* __restrict__ dout_clean,
                                                               bool beside) {
  if (beside)
    beside_previous();
  else
    after_previous();
  const ll row = (static_cast<ll>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const ll rows = static_cast<ll>(d.B) * d.Sq * d.n_h;
  if (row >= rows) return;
  const int lane = threadIdx.x & 31, dqk = d.d_qk();
  const int h = static_cast<int>(row % d.n_h);
  const ll bi = row / d.n_h;
  const int i = static_cast<int>(bi % d.Sq);
  const int b = static_cast<int>(bi / d.Sq);
  auto q_at = [&](int k) { return packed ? unpack8_value(q8, row, dqk, k) : to_f(__ldcg(q + row * dqk + k)); };
  float acc = 0.f;
  bool bad = false;
  for (int k = lane; k < dqk; k += 32) bad |= !finite(q_at(k));
  for (int k = lane; k < d.d_v; k += 32) {
    const float g = to_f(__ldcg(dout + row * d.d_v + k));
    bad |= !finite(g);
    acc = fmaf(packed ? unpack8_value(out8, row, d.d_v, k) : to_f(__ldcg(out + row * d.d_v + k)), g, acc);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  bad = __any_sync(0xffffffffu, bad);
  for (int k = lane; k < dqk; k += 32) q_clean[row * dqk + k] = bad ? 0.f : q_at(k);
  for (int k = lane; k < d.d_v; k += 32) dout_clean[row * d.d_v + k] = bad ? 0.f : to_f(__ldcg(dout + row * d.d_v + k));
  if (lane == 0) {
    const ll at = (static_cast<ll>(b) * d.n_h + h) * d.Sq + i;
    const float v = __ldcg(lse + at);
    float L = v, D = acc;
    if (v == -INFINITY) {
      L = INFINITY;
      D = 0.f;
    } else if (bad || !finite(v) || !finite(acc)) {
      L = NAN;
      D = 0.f;
    }
    lse_row[at] = L;
    delta[at] = D;
  }
  if (beside) end_after_previous(blockIdx.x == gridDim.x - 1);
}

}  // namespace

size_t mask_bytes(const Dims& d, int elem) {
  char* const base = reinterpret_cast<char*>(256);  // only measured, never read
  char* p = base;
  mask_carve(d, elem, p);
  return static_cast<size_t>(p - base);
}

MaskBuffers mask_carve(const Dims& d, int elem, char*& p) {
  auto take = [&](size_t n) {
    char* r = p;
    p += align_up(n, 256);
    return r;
  };
  const size_t B = d.B, kt = d.skv_pad / 128, nq64 = d.sq_pad / 64;
  MaskBuffers m{};
  m.rows = reinterpret_cast<int2*>(take(B * d.sq_pad * 8));
  m.q_tiles = reinterpret_cast<int2*>(take(B * (nq64 / 2) * 8));
  m.q_hull = reinterpret_cast<int2*>(take(B * nq64 * 8));
  m.kt_count = reinterpret_cast<int*>(take(B * kt * 4));
  m.kt_list = reinterpret_cast<int*>(take(B * kt * nq64 * 4));
  m.q_bad = reinterpret_cast<int*>(take(4));
  m.counters = reinterpret_cast<int*>(take(12));
  m.work = reinterpret_cast<int4*>(take(B * (nq64 / 2) * 16));
  m.seen = reinterpret_cast<int*>(take(B * kt * 4));
  m.seen_list = reinterpret_cast<int*>(take(B * kt * 4));
  m.bad = reinterpret_cast<uint32_t*>(take(B * ((d.S + 31) / 32) * 4));
  m.c_kv = take(B * d.S * d.d_c * elem);
  m.k_rope = take(B * d.S * d.d_rope * elem);
  return m;
}

LaunchResult mask_prepare(const Dims& d, bool is_bf16, const int* key_lo, const int* key_hi, const void* c_kv,
                          const void* k_rope, const MaskBuffers& m, bool key_tiles, cudaStream_t st) {
  LaunchResult r;
  const int words = (d.S + 31) / 32;
  const dim3 grid(words + (d.sq_pad + 255) / 256, d.B);
  auto aligned = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  auto run = [&](auto* kern, auto* type) {
    using T = std::remove_pointer_t<decltype(type)>;
    return launch_next(kern, grid, 256, 0, st, d, key_lo, key_hi, static_cast<const T*>(c_kv),
                       static_cast<const T*>(k_rope), m);
  };
  if (is_bf16 && d.d_c == 512 && d.d_rope == 64 && aligned(c_kv) && aligned(k_rope))
    r.err = run(mask_inputs_kernel<bf16, true>, static_cast<bf16*>(nullptr));
  else if (is_bf16)
    r.err = run(mask_inputs_kernel<bf16, false>, static_cast<bf16*>(nullptr));
  else
    r.err = run(mask_inputs_kernel<float, false>, static_cast<float*>(nullptr));
  if (r.err == cudaSuccess && key_tiles)
    r.err = launch_next(mask_tiles_kernel, d.B, 1024, 0, st, d.skv_pad / 128, d.sq_pad / 64, m.bad, words, m.rows,
                        m.q_tiles, m.q_hull, m.kt_count, m.kt_list, m.seen, m.seen_list, m.counters, m.work);
  if (r.err != cudaSuccess) r.what = "mask preparation";
  return r;
}

LaunchResult mask_key_bounds(const Dims& d, const int* starts, int n_docs, const int* prefix, int window, int* key_lo,
                             int* key_hi, cudaStream_t st) {
  LaunchResult r;
  r.err = launch_next(key_bounds_kernel, dim3((d.Sq + 127) / 128, d.B), 128, 0, st, d, starts, n_docs, prefix, window,
                      key_lo, key_hi);
  if (r.err != cudaSuccess) r.what = "key bounds";
  return r;
}

LaunchResult tc_mask_bwd_pre(const Dims& d, const bf16* q, const bf16* out, const Packed* q8, const Packed* out8,
                             const bf16* dout, const float* lse, const BwdWorkspace& w, bf16* q_clean,
                             bf16* dout_clean, int* q_bad, bool check_q, bool beside, cudaStream_t st) {
  LaunchResult r;
  const ll rows = static_cast<ll>(d.B) * d.sq_pad * d.n_h;
  const unsigned grid = static_cast<unsigned>((rows + 31) / 32);
  const auto kern = q8 ? mask_bwd_pre_kernel<true, true>
                       : check_q ? mask_bwd_pre_kernel<false, true> : mask_bwd_pre_kernel<false, false>;
  r.err = launch_next(kern, grid, 256, 0, st, d, q, out, q8 ? *q8 : Packed{}, out8 ? *out8 : Packed{}, dout, lse, w.lse2,
                      w.delta, q_clean, q_bad, beside);
  if (r.err == cudaSuccess)
    r.err = launch_next(mask_clean_kernel, 2 * sm_count(), 256, 0, st, static_cast<ll>(d.B) * d.Sq * d.n_h,
                        q8 ? nullptr : q, dout, q_clean, dout_clean, q_bad);
  if (r.err != cudaSuccess) r.what = "masked backward row pass";
  return r;
}

LaunchResult simt_mask_bwd_pre(const Dims& d, bool is_bf16, const void* q, const void* out, const Packed* q8,
                               const Packed* out8, const void* dout, const float* lse, float* lse_row, float* delta,
                               float* q_clean, float* dout_clean, bool beside, cudaStream_t st) {
  LaunchResult r;
  const ll rows = static_cast<ll>(d.B) * d.Sq * d.n_h;
  const unsigned grid = static_cast<unsigned>((rows + 7) / 8);
  const Packed a = q8 ? *q8 : Packed{}, o = out8 ? *out8 : Packed{};
  auto run = [&](auto* kern, auto* type) {
    using T = std::remove_pointer_t<decltype(type)>;
    return launch_next(kern, grid, 256, 0, st, d, static_cast<const T*>(q), static_cast<const T*>(out), a, o,
                       q8 != nullptr, static_cast<const T*>(dout), lse, lse_row, delta, q_clean, dout_clean, beside);
  };
  r.err = is_bf16 ? run(mask_bwd_pre_any_kernel<bf16>, static_cast<bf16*>(nullptr))
                  : run(mask_bwd_pre_any_kernel<float>, static_cast<float*>(nullptr));
  if (r.err != cudaSuccess) r.what = "masked backward row pass";
  return r;
}

}  // namespace laga
