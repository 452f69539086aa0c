// Masked attention on the CUDA cores in fp32, for any head widths up to 256: the
// forward, dq and dK/dV, and the small products of the K/V rebuild and its backward.
//
// Attention: tiles of 16 RI rows by 64 (forward) or 32 (backward) columns live in shared
// memory; one pass over the keys with the running maximum and sum of the softmax; O, dq,
// dK and dV stay in registers. Rows are stored with a pitch of an odd number of 16-byte
// units, so the 16 threads that read 16 consecutive rows as float4 touch different banks.
// Thread (tx, ty) of 16 x 16 owns tile rows RI ty .. RI ty + RI - 1 and, of the score tile,
// columns tx, tx + 16, ...; of a head-wide accumulator, columns 64 c + 4 tx .. + 3.
// N = ceil(widest head / 64) picks the accumulator's width, RI the rows. More rows a thread
// mean more multiply-adds per shared-memory load, fewer mean more CTAs. And a cluster of CTAs
// shares a tile's walk, each taking every second or fourth step, the results merged through
// distributed shared memory: walks differ in length (causal rows, documents), the longest sets
// the time, and a CTA alone on its SM waits for its own latencies. Measured forward / backward,
// us, rows a thread x CTAs a tile:
//   256 rows x 4 heads, d 48 / 32      1x1: 25 / 43      2x1: 29 / 44      2x4: 18 / 29
//   2 x 509 x 3, d 64 / 56             1x1: 46 / 88      2x1: 50 / 84      2x2: 38 / 70
//   1024 x 2, d 96 / 64                2x1: 162 / 310    2x4: 87 / 145     4x4: 59 / -
//   4096 x 8, d 64 / 56, 6 documents   2x1: 420 / 983    2x2: 399 / 967    4x2: 415 / -
//   4096 x 8, d 96 / 96                2x1: 3200 / 5576  2x2: 3025 / 5173  4x2: 1745 / -
//   600 x 4, d 192 / 128               2x1: 133 / 256    2x2: 83 / 169     4x2: 100 / -
//   2048 x 4, d 192 / 128              2x1: 635 / 1237   2x2: 531 / 1018   4x2: 453 / -
// A tile's global loads are issued eight rows deep per warp, lanes along the width, and where
// the registers allow it a step ahead; one value at a time cost 14 us per key step.
// What bounds it is still each CTA's walk: the schedulers wait for shared memory and for each
// other's arithmetic more than they issue.
#include "mask.h"

#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

namespace laga {
namespace {

using ll = long long;
constexpr int KFWD = 64;     // keys per step, forward
constexpr int KBWD = 32;     // keys (dq) or queries (dK/dV) per step
constexpr int THREADS = 256;

__host__ __device__ __forceinline__ int pitch4(int width) { return ((width + 3) / 4) | 1; }  // in float4

struct SimtParams {
  Dims d;
  int splits;            // CTAs (a cluster) that share a tile's walk, every splits-th step each
  const void* q;         // [B][Sq][n_h][d_qk]; the forward's in the inputs' type, else fp32
  bool q_bf16;
  const float* kn;       // [B][S][n_h][d_nope]
  const float* v;        // [B][S][n_h][d_v]
  const void* k_rope;    // [B][S][d_rope], the inputs' type
  bool rope_bf16;
  const int2* rows;      // [B][sq_pad]
  const int2* q_hull;    // [B][sq_pad / 64]
  const uint32_t* bad;   // [B][ceil(S / 32)] bit per key: not finite
  float cap, inv_cap;    // 0: none
  const float* slopes;
  const float* dout;     // [B][Sq][n_h][d_v], clean
  const float* lse_row;  // [B][n_h][Sq]
  const float* delta;
  void* out;             // out or dq
  bool out_bf16;
  float* lse;
  float *dkn, *dv, *dkr; // dkr [B][S][n_h][d_rope]
};

__device__ __forceinline__ int position(const Dims& d, int i) {
  return (d.q_split > 0 && i >= d.q_split) ? d.q_offset2 + (i - d.q_split) : d.q_offset + i;
}

__device__ __forceinline__ float load(const void* p, bool is_bf16, ll at) {
  return is_bf16 ? __bfloat162float(static_cast<const bf16*>(p)[at]) : static_cast<const float*>(p)[at];
}
__device__ __forceinline__ void store(void* p, bool is_bf16, ll at, float v) {
  if (is_bf16)
    static_cast<bf16*>(p)[at] = __float2bfloat16_rn(v);
  else
    static_cast<float*>(p)[at] = v;
}

// dst[r][k] = get(r, k) for r < ROWS (a multiple of 8), k < width, zero up to the next multiple of four.
template <int ROWS, class F>
__device__ __forceinline__ void fill(float4* dst, int pitch, int width, F&& get) {
  const int w = (width + 3) & ~3, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int DEEP = ROWS / 8 < 8 ? ROWS / 8 : 8;
  float* f = reinterpret_cast<float*>(dst);
  for (int k = lane; k < w; k += 32)
#pragma unroll
    for (int r0 = 0; r0 < ROWS; r0 += 8 * DEEP) {
      float v[DEEP];
#pragma unroll
      for (int i = 0; i < DEEP; ++i) v[i] = k < width ? get(r0 + 8 * i + warp, k) : 0.f;
#pragma unroll
      for (int i = 0; i < DEEP; ++i) f[(r0 + 8 * i + warp) * pitch * 4 + k] = v[i];
    }
}

// The same through registers: fetch() issues all of a tile's loads, put() stores them later, so
// that the next step's tile is on its way while this one is worked on. C: columns per lane.
template <int ROWS, int C>
struct Staged {
  float v[ROWS / 8][C];
  template <class F>
  __device__ __forceinline__ void fetch(int width, F&& get) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < ROWS / 8; ++i)
#pragma unroll
      for (int c = 0; c < C; ++c) v[i][c] = lane + 32 * c < width ? get(8 * i + warp, lane + 32 * c) : 0.f;
  }
  __device__ __forceinline__ void put(float4* dst, int pitch, int width) const {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = (width + 3) & ~3;
    float* f = reinterpret_cast<float*>(dst);
#pragma unroll
    for (int i = 0; i < ROWS / 8; ++i)
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (lane + 32 * c < w) f[(8 * i + warp) * pitch * 4 + lane + 32 * c] = v[i][c];
  }
};

__device__ __forceinline__ float dot4(float4 a, float4 b, float acc) {
  acc = fmaf(a.x, b.x, acc);
  acc = fmaf(a.y, b.y, acc);
  acc = fmaf(a.z, b.z, acc);
  return fmaf(a.w, b.w, acc);
}

// acc[i][j] = sum_k A[RI ty + i][k] B[tx + 16 j][k]
template <int RI, int NJ>
__device__ __forceinline__ void score_tile(const float4* A, const float4* B, int pitch, int n4, int tx, int ty,
                                           float (&acc)[RI][NJ]) {
#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = 0.f;
#pragma unroll 2
  for (int k = 0; k < n4; ++k) {
    float4 a[RI], b[NJ];
#pragma unroll
    for (int i = 0; i < RI; ++i) a[i] = A[(RI * ty + i) * pitch + k];
#pragma unroll
    for (int j = 0; j < NJ; ++j) b[j] = B[(tx + 16 * j) * pitch + k];
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = dot4(a[i], b[j], acc[i][j]);
  }
}

// A column of RI weights per (row of the shared dimension, ty): written by the score tile's
// owner, read by the accumulators'. Pitch 17 keeps the 16 threads of a write apart.
template <int RI>
__device__ __forceinline__ void put_weights(float* w, int n, int ty, const float (&v)[RI]) {
  float* d = w + (n * 17 + ty) * RI;
  if constexpr (RI == 4)
    *reinterpret_cast<float4*>(d) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<float2*>(d) = make_float2(v[0], v[1]);
}

// acc[i][c] += sum_n Wt[n][RI ty + i] B[n][64 c + 4 tx ..]
template <int RI, int N>
__device__ __forceinline__ void weighted_rows(const float* Wt, const float4* B, int pitch, int count, int width4, int tx,
                                              int ty, float4 (&acc)[RI][N]) {
#pragma unroll 4
  for (int n = 0; n < count; ++n) {
    float wi[RI];
    const float* w = Wt + (n * 17 + ty) * RI;
    if constexpr (RI == 4) {
      const float4 t = *reinterpret_cast<const float4*>(w);
      wi[0] = t.x;
      wi[1] = t.y;
      wi[2] = t.z;
      wi[3] = t.w;
    } else {
#pragma unroll
      for (int i = 0; i < RI; ++i) wi[i] = w[i];
    }
#pragma unroll
    for (int c = 0; c < N; ++c) {
      if (16 * c + tx >= width4) continue;
      const float4 b = B[n * pitch + 16 * c + tx];
#pragma unroll
      for (int i = 0; i < RI; ++i) {
        acc[i][c].x = fmaf(wi[i], b.x, acc[i][c].x);
        acc[i][c].y = fmaf(wi[i], b.y, acc[i][c].y);
        acc[i][c].z = fmaf(wi[i], b.z, acc[i][c].z);
        acc[i][c].w = fmaf(wi[i], b.w, acc[i][c].w);
      }
    }
  }
}

// A score from its raw product; *slope of the cap.
__device__ __forceinline__ float score_of(const SimtParams& p, float raw, float slope, int pos, int key, float* dcap) {
  float s = raw * p.d.scale;
  if (p.cap > 0.f) {
    const float t = tanhf(s * p.inv_cap);
    s = t * p.cap;
    *dcap = fmaf(-t, t, 1.f);
  }
  return s - slope * fabsf(static_cast<float>(pos - key));
}

// Element k of row r of a tile that starts at row `first` (0 past the end).
struct KRows {
  const SimtParams& p;
  int b, h, first;
  __device__ __forceinline__ float operator()(int r, int k) const {
    const Dims& d = p.d;
    const int j = first + r;
    if (j >= d.S) return 0.f;
    const ll row = static_cast<ll>(b) * d.S + j;
    return k < d.d_nope ? p.kn[(row * d.n_h + h) * d.d_nope + k]
                        : load(p.k_rope, p.rope_bf16, row * d.d_rope + (k - d.d_nope));
  }
};
struct VRows {
  const SimtParams& p;
  int b, h, first;
  __device__ __forceinline__ float operator()(int r, int k) const {
    const int j = first + r;
    return j < p.d.S ? p.v[((static_cast<ll>(b) * p.d.S + j) * p.d.n_h + h) * p.d.d_v + k] : 0.f;
  }
};
struct QRows {
  const SimtParams& p;
  int b, h, first;
  __device__ __forceinline__ float operator()(int r, int k) const {
    const int i = first + r;
    return i < p.d.Sq ? load(p.q, p.q_bf16, ((static_cast<ll>(b) * p.d.Sq + i) * p.d.n_h + h) * p.d.d_qk() + k) : 0.f;
  }
};
struct DoRows {
  const SimtParams& p;
  int b, h, first;
  __device__ __forceinline__ float operator()(int r, int k) const {
    const int i = first + r;
    return i < p.d.Sq ? p.dout[((static_cast<ll>(b) * p.d.Sq + i) * p.d.n_h + h) * p.d.d_v + k] : 0.f;
  }
};

// Two streamed tiles (K and V, or q and dO) of ROWS rows: staged a step ahead where the
// registers allow (widths up to 128), else loaded in place.
template <int ROWS, int N>
struct StreamedPair {
  static constexpr bool AHEAD = N <= 2;
  static constexpr int C = AHEAD ? 2 * N : 1;
  Staged<ROWS, C> x, y;
  template <class A, class B>
  __device__ __forceinline__ void ahead(int wx, int wy, A&& a, B&& b) {
    if constexpr (AHEAD) {
      x.fetch(wx, a);
      y.fetch(wy, b);
    }
  }
  template <class A, class B>
  __device__ __forceinline__ void store(float4* sx, int px, int wx, float4* sy, int py, int wy, A&& a, B&& b) {
    if constexpr (AHEAD) {
      x.put(sx, px, wx);
      y.put(sy, py, wy);
    } else {
      fill<ROWS>(sx, px, wx, a);
      fill<ROWS>(sy, py, wy, b);
    }
  }
};

__device__ __forceinline__ float half_warp_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float half_warp_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A cluster's CTAs put their threads' partial results into their shared memory (one that is free
// by then), the first one takes the others' in order, and nobody leaves before that.
template <int COUNT, class Take>
__device__ __forceinline__ bool merge_in_cluster(const SimtParams& p, float4* buf, const float4 (&mine)[COUNT], Take&& take) {
  if (p.splits == 1) return true;
  namespace cg = cooperative_groups;
  const cg::cluster_group cluster = cg::this_cluster();
  const unsigned rank = cluster.block_rank();
  __syncthreads();
  if (rank != 0)
#pragma unroll
    for (int i = 0; i < COUNT; ++i) buf[i * THREADS + threadIdx.x] = mine[i];
  cluster.sync();
  if (rank == 0)
    for (int r = 1; r < p.splits; ++r) {
      const float4* from = cluster.map_shared_rank(buf, r);
      float4 v[COUNT];
#pragma unroll
      for (int i = 0; i < COUNT; ++i) v[i] = from[i * THREADS + threadIdx.x];
      take(v);
    }
  cluster.sync();
  return rank == 0;
}
__device__ __forceinline__ float4 plus(float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }

// out and lse of 16 RI query rows of one head.
template <int N, int RI>
__global__ void __launch_bounds__(THREADS) masked_simt_fwd(const SimtParams p) {
  constexpr int ROWS = 16 * RI;
  extern __shared__ float4 sm[];
  const Dims& d = p.d;
  const int pk = pitch4(d.d_qk()), pv = pitch4(d.d_v);
  float4 *sq = sm, *sk = sq + ROWS * pk, *sv = sk + KFWD * pk, *weights = sv + KFWD * pv;
  float* sp = reinterpret_cast<float*>(weights);
  const int t = blockIdx.x / p.splits, rank = blockIdx.x - t * p.splits, step = p.splits * KFWD, h = blockIdx.y, b = blockIdx.z;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int i0 = t * ROWS + RI * ty;  // this thread's first row
  after_previous();
  fill<ROWS>(sq, pk, d.d_qk(), QRows{p, b, h, t * ROWS});
  int lo[RI], hi[RI];
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int2 v = p.rows[static_cast<ll>(b) * d.sq_pad + i0 + i];
    lo[i] = v.x;
    hi[i] = v.y;
  }
  const float slope = p.slopes ? p.slopes[h] : 0.f;
  float m[RI], l[RI];
  float4 o[RI][N];
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < N; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const int2 hull = p.q_hull[static_cast<ll>(b) * (d.sq_pad / 64) + t * ROWS / 64];  // of the 64 rows around
  const int j_first = (hull.x < hull.y ? hull.x / KFWD * KFWD : 0) + rank * KFWD;
  StreamedPair<KFWD, N> kv;
  if (j_first < hull.y) kv.ahead(d.d_qk(), d.d_v, KRows{p, b, h, j_first}, VRows{p, b, h, j_first});
  for (int j0 = j_first; j0 < hull.y; j0 += step) {
    __syncthreads();
    kv.store(sk, pk, d.d_qk(), sv, pv, d.d_v, KRows{p, b, h, j0}, VRows{p, b, h, j0});
    __syncthreads();
    if (j0 + step < hull.y) kv.ahead(d.d_qk(), d.d_v, KRows{p, b, h, j0 + step}, VRows{p, b, h, j0 + step});
    float s[RI][4];
    score_tile<RI>(sq, sk, pk, (d.d_qk() + 3) / 4, tx, ty, s);
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      const int pos = position(d, i0 + i);
      float unused, mt = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = j0 + tx + 16 * j;
        s[i][j] = key >= lo[i] && key < hi[i] ? score_of(p, s[i][j], slope, pos, key, &unused) : -INFINITY;
        mt = fmaxf(mt, s[i][j]);
      }
      const float mn = fmaxf(m[i], half_warp_max(mt));
      const float base = mn == -INFINITY ? 0.f : mn;
      const float alpha = expf(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = expf(s[i][j] - base);
        sum += s[i][j];
      }
      l[i] = l[i] * alpha + half_warp_sum(sum);
      m[i] = mn;
#pragma unroll
      for (int c = 0; c < N; ++c) {
        o[i][c].x *= alpha;
        o[i][c].y *= alpha;
        o[i][c].z *= alpha;
        o[i][c].w *= alpha;
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float w[RI];
#pragma unroll
      for (int i = 0; i < RI; ++i) w[i] = s[i][j];
      put_weights<RI>(sp, tx + 16 * j, ty, w);
    }
    __syncthreads();
    weighted_rows<RI, N>(sp, sv, pv, KFWD, (d.d_v + 3) / 4, tx, ty, o);
  }
  float4 part[RI * (N + 1)];
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    part[i * (N + 1)] = make_float4(m[i], l[i], 0.f, 0.f);
#pragma unroll
    for (int c = 0; c < N; ++c) part[i * (N + 1) + 1 + c] = o[i][c];
  }
  const bool writes = merge_in_cluster(p, sm, part, [&](const float4 (&v)[RI * (N + 1)]) {
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      const float4 w = v[i * (N + 1)];
      const float mn = fmaxf(m[i], w.x), base = mn == -INFINITY ? 0.f : mn;
      const float a = expf(m[i] - base), g = expf(w.x - base);
      l[i] = l[i] * a + w.y * g;
      m[i] = mn;
#pragma unroll
      for (int c = 0; c < N; ++c) {
        const float4 x = v[i * (N + 1) + 1 + c];
        o[i][c] = make_float4(o[i][c].x * a + x.x * g, o[i][c].y * a + x.y * g, o[i][c].z * a + x.z * g,
                              o[i][c].w * a + x.w * g);
      }
    }
  });
  if (!writes) return;
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    // the row's 16 threads share the words of the keys it sees
    const uint32_t* words = p.bad + static_cast<ll>(b) * ((d.S + 31) / 32);
    const unsigned votes = __ballot_sync(0xffffffffu, sees_bad_key(words, lo[i], hi[i], tx, 16));
    const bool poisoned = (votes & (threadIdx.x & 16 ? 0xffff0000u : 0xffffu)) != 0u;
    if (i0 + i >= d.Sq) continue;
    float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
    float L = l[i] == 0.f ? -INFINITY : m[i] + logf(l[i]);
    if (poisoned || (lo[i] < hi[i] && l[i] == 0.f)) inv = L = NAN;  // l = 0: an infinite q, all scores -inf
    const ll row = (static_cast<ll>(b) * d.Sq + i0 + i) * d.n_h + h;
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const float v[4] = {o[i][c].x, o[i][c].y, o[i][c].z, o[i][c].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int col = 64 * c + 4 * tx + k;
        if (col < d.d_v) store(p.out, p.out_bf16, row * d.d_v + col, v[k] * inv);
      }
    }
    if (tx == 0) p.lse[(static_cast<ll>(b) * d.n_h + h) * d.Sq + i0 + i] = L;
  }
}

// dq of 16 RI query rows of one head.
template <int N, int RI>
__device__ __forceinline__ void masked_simt_dq(const SimtParams& p, int t, int rank) {
  constexpr int ROWS = 16 * RI;
  extern __shared__ float4 sm[];
  const Dims& d = p.d;
  const int pk = pitch4(d.d_qk()), pv = pitch4(d.d_v);
  float4 *sq = sm, *sdo = sq + ROWS * pk, *sk = sdo + ROWS * pv, *sv = sk + KBWD * pk, *weights = sv + KBWD * pv;
  float* sds = reinterpret_cast<float*>(weights);
  const int h = blockIdx.y, b = blockIdx.z;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int i0 = t * ROWS + RI * ty;
  fill<ROWS>(sq, pk, d.d_qk(), QRows{p, b, h, t * ROWS});
  fill<ROWS>(sdo, pv, d.d_v, DoRows{p, b, h, t * ROWS});
  int lo[RI], hi[RI];
  float L[RI], D[RI];
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int2 v = p.rows[static_cast<ll>(b) * d.sq_pad + i0 + i];
    lo[i] = v.x;
    hi[i] = v.y;
    const bool in = i0 + i < d.Sq;
    const ll at = (static_cast<ll>(b) * d.n_h + h) * d.Sq + i0 + i;
    L[i] = in ? p.lse_row[at] : INFINITY;
    D[i] = in ? p.delta[at] : 0.f;
  }
  const float slope = p.slopes ? p.slopes[h] : 0.f;
  float4 acc[RI][N];
#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int c = 0; c < N; ++c) acc[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int2 hull = p.q_hull[static_cast<ll>(b) * (d.sq_pad / 64) + t * ROWS / 64];  // of the 64 rows around
  const int step = p.splits * KBWD, j_first = (hull.x < hull.y ? hull.x / KBWD * KBWD : 0) + rank * KBWD;
  StreamedPair<KBWD, N> kv;
  if (j_first < hull.y) kv.ahead(d.d_qk(), d.d_v, KRows{p, b, h, j_first}, VRows{p, b, h, j_first});
  for (int j0 = j_first; j0 < hull.y; j0 += step) {
    __syncthreads();
    kv.store(sk, pk, d.d_qk(), sv, pv, d.d_v, KRows{p, b, h, j0}, VRows{p, b, h, j0});
    __syncthreads();
    if (j0 + step < hull.y) kv.ahead(d.d_qk(), d.d_v, KRows{p, b, h, j0 + step}, VRows{p, b, h, j0 + step});
    float s[RI][2], dp[RI][2];
    score_tile<RI>(sq, sk, pk, (d.d_qk() + 3) / 4, tx, ty, s);
    score_tile<RI>(sdo, sv, pv, (d.d_v + 3) / 4, tx, ty, dp);
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      const int pos = position(d, i0 + i);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int key = j0 + tx + 16 * j;
        float dcap = 1.f;
        const float v = score_of(p, s[i][j], slope, pos, key, &dcap);
        s[i][j] = key >= lo[i] && key < hi[i] ? expf(v - L[i]) * (dp[i][j] - D[i]) * dcap : 0.f;
      }
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float w[RI];
#pragma unroll
      for (int i = 0; i < RI; ++i) w[i] = s[i][j];
      put_weights<RI>(sds, tx + 16 * j, ty, w);
    }
    __syncthreads();
    weighted_rows<RI, N>(sds, sk, pk, KBWD, (d.d_qk() + 3) / 4, tx, ty, acc);
  }
  float4 part[RI * N];
#pragma unroll
  for (int i = 0; i < RI * N; ++i) part[i] = acc[i / N][i % N];
  const bool writes = merge_in_cluster(p, sm, part, [&](const float4 (&v)[RI * N]) {
#pragma unroll
    for (int i = 0; i < RI * N; ++i) acc[i / N][i % N] = plus(acc[i / N][i % N], v[i]);
  });
  if (!writes) return;
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    if (i0 + i >= d.Sq) continue;
    const ll row = (static_cast<ll>(b) * d.Sq + i0 + i) * d.n_h + h;
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const float v[4] = {acc[i][c].x, acc[i][c].y, acc[i][c].z, acc[i][c].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int col = 64 * c + 4 * tx + k;
        if (col < d.d_qk()) store(p.out, p.out_bf16, row * d.d_qk() + col, v[k] * d.scale);
      }
    }
  }
}

// dK (both parts) and dV of 16 RI keys of one head.
template <int N, int RI>
__device__ __forceinline__ void masked_simt_dkv(const SimtParams& p, int t, int rank) {
  constexpr int ROWS = 16 * RI;
  extern __shared__ float4 sm[];
  const Dims& d = p.d;
  const int pk = pitch4(d.d_qk()), pv = pitch4(d.d_v);
  float4 *sk = sm, *sv = sk + ROWS * pk, *sq = sv + ROWS * pv, *sdo = sq + KBWD * pk, *weights = sdo + KBWD * pv;
  float *sp = reinterpret_cast<float*>(weights), *sds = sp + KBWD * 17 * RI;
  const int h = blockIdx.y, b = blockIdx.z;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int k0 = t * ROWS + RI * ty;  // this thread's first key
  fill<ROWS>(sk, pk, d.d_qk(), KRows{p, b, h, t * ROWS});
  fill<ROWS>(sv, pv, d.d_v, VRows{p, b, h, t * ROWS});
  const float slope = p.slopes ? p.slopes[h] : 0.f;
  float4 dk[RI][N], dv[RI][N];
#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int c = 0; c < N; ++c) dk[i][c] = dv[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int nq64 = d.sq_pad / 64;
  // the next query tile from q0 on that may see these keys (the same for every thread)
  auto next_tile = [&](int q0) {
    for (; q0 < d.Sq; q0 += KBWD) {
      const int2 hull = p.q_hull[static_cast<ll>(b) * nq64 + q0 / 64];
      if (hull.x < hull.y && hull.x < (t + 1) * ROWS && hull.y > t * ROWS) break;
    }
    return q0;
  };
  StreamedPair<KBWD, N> qd;
  auto after = [&](int q0) {  // this CTA's next one
    for (int k = 0; k < p.splits && q0 < d.Sq; ++k) q0 = next_tile(q0 + KBWD);
    return q0;
  };
  int q0 = next_tile(0);
  for (int k = 0; k < rank && q0 < d.Sq; ++k) q0 = next_tile(q0 + KBWD);
  if (q0 < d.Sq) qd.ahead(d.d_qk(), d.d_v, QRows{p, b, h, q0}, DoRows{p, b, h, q0});
  for (int q1; q0 < d.Sq; q0 = q1) {
    __syncthreads();
    qd.store(sq, pk, d.d_qk(), sdo, pv, d.d_v, QRows{p, b, h, q0}, DoRows{p, b, h, q0});
    __syncthreads();
    q1 = after(q0);
    if (q1 < d.Sq) qd.ahead(d.d_qk(), d.d_v, QRows{p, b, h, q1}, DoRows{p, b, h, q1});
    float s[RI][2], dp[RI][2];
    score_tile<RI>(sk, sq, pk, (d.d_qk() + 3) / 4, tx, ty, s);
    score_tile<RI>(sv, sdo, pv, (d.d_v + 3) / 4, tx, ty, dp);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = q0 + tx + 16 * j;
      const int2 r = p.rows[static_cast<ll>(b) * d.sq_pad + i];  // {0, 0} past Sq
      const bool in = i < d.Sq;
      const ll at = (static_cast<ll>(b) * d.n_h + h) * d.Sq + i;
      const float L = in ? p.lse_row[at] : INFINITY, D = in ? p.delta[at] : 0.f;
      const int pos = position(d, i);
#pragma unroll
      for (int k = 0; k < RI; ++k) {
        const int key = k0 + k;
        float dcap = 1.f;
        const float v = score_of(p, s[k][j], slope, pos, key, &dcap);
        const bool sees = key >= r.x && key < r.y;
        const float e = sees ? expf(v - L) : 0.f;
        s[k][j] = e;
        dp[k][j] = sees ? e * (dp[k][j] - D) * dcap : 0.f;  // a masked dP may have overflowed (padding's dO)
      }
      float w[RI], g[RI];
#pragma unroll
      for (int k = 0; k < RI; ++k) {
        w[k] = s[k][j];
        g[k] = dp[k][j];
      }
      put_weights<RI>(sp, tx + 16 * j, ty, w);
      put_weights<RI>(sds, tx + 16 * j, ty, g);
    }
    __syncthreads();
    weighted_rows<RI, N>(sp, sdo, pv, KBWD, (d.d_v + 3) / 4, tx, ty, dv);
    weighted_rows<RI, N>(sds, sq, pk, KBWD, (d.d_qk() + 3) / 4, tx, ty, dk);
  }
  float4 part[2 * RI * N];
#pragma unroll
  for (int i = 0; i < RI * N; ++i) {
    part[2 * i] = dk[i / N][i % N];
    part[2 * i + 1] = dv[i / N][i % N];
  }
  const bool writes = merge_in_cluster(p, sm, part, [&](const float4 (&v)[2 * RI * N]) {
#pragma unroll
    for (int i = 0; i < RI * N; ++i) {
      dk[i / N][i % N] = plus(dk[i / N][i % N], v[2 * i]);
      dv[i / N][i % N] = plus(dv[i / N][i % N], v[2 * i + 1]);
    }
  });
  if (!writes) return;
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int j = k0 + i;
    if (j >= d.S) continue;
    const ll row = (static_cast<ll>(b) * d.S + j) * d.n_h + h;
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const float a[4] = {dk[i][c].x, dk[i][c].y, dk[i][c].z, dk[i][c].w};
      const float g[4] = {dv[i][c].x, dv[i][c].y, dv[i][c].z, dv[i][c].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int col = 64 * c + 4 * tx + k;
        if (col < d.d_nope)
          p.dkn[row * d.d_nope + col] = a[k] * d.scale;
        else if (col < d.d_qk())
          p.dkr[row * d.d_rope + (col - d.d_nope)] = a[k] * d.scale;
        if (col < d.d_v) p.dv[row * d.d_v + col] = g[k];
      }
    }
  }
}

// Both sides of the backward in one launch: neither needs the other's result, and a small
// problem's CTAs of either alone leave most SMs idle (256 rows, 4 heads: 64 CTAs each).
template <int N, int RI>
__global__ void __launch_bounds__(THREADS) masked_simt_bwd(const SimtParams p) {
  after_previous();
  const int q_blocks = (p.d.Sq + 16 * RI - 1) / (16 * RI);
  const int t = blockIdx.x / p.splits, rank = blockIdx.x - t * p.splits;
  if (t < q_blocks)
    masked_simt_dq<N, RI>(p, t, rank);
  else
    masked_simt_dkv<N, RI>(p, t - q_blocks, rank);
}

struct Ws {
  float *kn, *v;
  MaskBuffers mask;
  float *q, *dout, *lse_row, *delta, *dkn, *dv, *dkr;  // backward
};

Ws carve(const Dims& d, int elem, bool bwd, char*& p) {
  auto take = [&](size_t n) {
    float* r = reinterpret_cast<float*>(p);
    p += align_up(n * sizeof(float), 256);
    return r;
  };
  const size_t keys = static_cast<size_t>(d.B) * d.S * d.n_h, qs = static_cast<size_t>(d.B) * d.Sq * d.n_h;
  Ws w{};
  w.kn = take(keys * d.d_nope);  // K, V and the mask's buffers first: what a backward with reuse reads
  w.v = take(keys * d.d_v);
  w.mask = mask_carve(d, elem, p);
  if (bwd) {
    w.q = take(qs * d.d_qk());
    w.dout = take(qs * d.d_v);
    w.lse_row = take(qs);
    w.delta = take(qs);
    w.dkn = take(keys * d.d_nope);
    w.dv = take(keys * d.d_v);
    w.dkr = take(keys * d.d_rope);
  }
  return w;
}

size_t bytes(const Dims& d, int elem, bool bwd) {
  char* const base = reinterpret_cast<char*>(256);  // only measured, never read
  char* p = base;
  carve(d, elem, bwd, p);
  return static_cast<size_t>(p - base);
}

SimtParams params(const Dims& d, bool is_bf16, const ScoreMods& mods, const Ws& w) {
  SimtParams p{};
  p.d = d;
  p.kn = w.kn;
  p.v = w.v;
  p.k_rope = w.mask.k_rope;
  p.rope_bf16 = is_bf16;
  p.rows = w.mask.rows;
  p.q_hull = w.mask.q_hull;
  p.bad = w.mask.bad;
  p.cap = mods.cap;
  p.inv_cap = mods.cap > 0.f ? 1.f / mods.cap : 0.f;
  p.slopes = mods.slopes;
  p.out_bf16 = is_bf16;
  return p;
}

// Rows per thread and CTAs per tile, by the table at the top: four rows a thread (forward only;
// the backward's accumulators leave no registers for them) where the accumulators are wide enough
// to gain from it and, for the widest, the tiles many; four CTAs a tile as long as that does not
// overfill the SMs, else two; never more than a walk can have steps.
struct Tiling {
  int rows, splits;
};
Tiling tiling(const Dims& d, int n, bool bwd) {
  const ll of64 = (static_cast<ll>(bwd ? d.Sq + d.S : d.Sq) + 63) / 64 * d.n_h * d.B;  // tiles of 64 rows
  const int rows = !bwd && (n == 2 || (n == 4 && of64 >= 64)) ? 4 : 2;
  const int steps = bwd ? (std::max(d.Sq, d.S) + KBWD - 1) / KBWD : (d.S + KFWD - 1) / KFWD;
  const int most = 4 * (of64 * 4 / rows) <= (bwd ? 512 : 256) ? 4 : 2;
  return Tiling{rows, steps >= most ? most : steps >= 2 ? 2 : 1};
}

template <bool BWD, int N, int RI>
constexpr auto kernel_of() {
  if constexpr (BWD)
    return masked_simt_bwd<N, RI>;
  else
    return masked_simt_fwd<N, RI>;
}

template <bool BWD, int N, int RI>
cudaError_t launch_rows(const Dims& d, SimtParams p, int splits, cudaStream_t st) {
  const int pk = pitch4(d.d_qk()), pv = pitch4(d.d_v);
  constexpr int R = 16 * RI;
  size_t smem = BWD ? sizeof(float4) * (R + KBWD) * (pk + pv) + sizeof(float) * 2 * KBWD * 17 * RI
                    : sizeof(float4) * ((R + KFWD) * pk + KFWD * pv) + sizeof(float) * KFWD * 17 * RI;
  if (splits > 1) smem = std::max(smem, sizeof(float4) * THREADS * RI * (BWD ? 2 * N : N + 1));  // partial results
  p.splits = splits;
  const int blocks = (d.Sq + R - 1) / R + (BWD ? (d.S + R - 1) / R : 0);
  void (*kern)(SimtParams) = kernel_of<BWD, N, RI>();
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_next_in_clusters(splits, kern, dim3(blocks * splits, d.n_h, d.B), THREADS, smem, st, p);
}

template <bool BWD>
cudaError_t launch(const Dims& d, const SimtParams& p, cudaStream_t st) {
  const int w = std::max(d.d_qk(), d.d_v), n = w <= 64 ? 1 : w <= 128 ? 2 : 4;
  const Tiling t = tiling(d, n, BWD);
  if constexpr (BWD) {
    return n == 1   ? launch_rows<true, 1, 2>(d, p, t.splits, st)
           : n == 2 ? launch_rows<true, 2, 2>(d, p, t.splits, st)
                    : launch_rows<true, 4, 2>(d, p, t.splits, st);
  } else {
    return n == 1        ? launch_rows<false, 1, 2>(d, p, t.splits, st)
           : n == 2      ? launch_rows<false, 2, 4>(d, p, t.splits, st)
           : t.rows == 2 ? launch_rows<false, 4, 2>(d, p, t.splits, st)
                         : launch_rows<false, 4, 4>(d, p, t.splits, st);
  }
}

// ---- the rebuild's products: C[m][n] = sum over one or two pairs of A(m, k) B(k, n), any
// strides, several such products in one launch. A CTA makes one 32 x 32 tile; its four groups
// of 64 threads each take every fourth block of 16 k, and their sums are added in a fixed
// order through shared memory. These products are small (a weight gradient is d_c x n_h d
// with k = all keys): a few dozen tiles, so the k loop's latency is the time, and both the
// small tile and the split shorten it (2 x 509 keys of width 72, 3 heads: the three gradients in
// 31 us, where 64 x 64 tiles without the split took 182 for each dW). Where k is long and the tiles
// few, a cluster of two or four CTAs shares a tile's k too: the whole backward of that problem takes
// 92 us with one CTA a tile, 73 with two, 70 with four (of 256 keys, 4 heads: 33 / 29 / 30); the
// rebuild's short k loses by it (18 / 20 / 23).
struct GemmPair {
  const void *a, *b;
  bool a_bf16, b_bf16;
  int K;
  ll am, ak, bk, bn;
};
struct GemmJob {
  int M, N, pairs, tiles_n, first_tile;
  GemmPair p[2];
  void* c;
  bool c_bf16;
  ll cm, cn;
};
// dk_rope[b, j, :] = the heads' RoPE-key gradients summed, in order: the CTAs from first_block on, a
// thread per value.
struct RopeSum {
  int first_block;
  ll total;
  int n_h, d_rope;
  const float* dkr;  // [B][S][n_h][d_rope]
  void* dk_rope;
  bool bf16_out;
};
struct GemmJobs {
  int n;
  int slices;  // CTAs (a cluster) that share a tile's k, every slices-th step each
  GemmJob job[3];
  RopeSum rope;
};

__global__ void __launch_bounds__(THREADS) small_gemm_kernel(const __grid_constant__ GemmJobs jobs) {
  constexpr int T = 32, KB = 16, GROUPS = 4;
  __shared__ float As[GROUPS][KB][T + 4], Bs[GROUPS][KB][T + 4];
  after_previous();
  if (static_cast<int>(blockIdx.x) >= jobs.rope.first_block) {
    const RopeSum& s = jobs.rope;
    const ll idx = static_cast<ll>(blockIdx.x - s.first_block) * THREADS + threadIdx.x;
    if (idx >= s.total) return;
    const ll bj = idx / s.d_rope;
    const int k = static_cast<int>(idx - bj * s.d_rope);
    float acc = 0.f;
    for (int h = 0; h < s.n_h; ++h) acc += s.dkr[(bj * s.n_h + h) * s.d_rope + k];
    store(s.dk_rope, s.bf16_out, idx, acc);
    return;
  }
  const int tile_id = static_cast<int>(blockIdx.x) / jobs.slices, rank = static_cast<int>(blockIdx.x) - tile_id * jobs.slices;
  int which = 0;
  while (which + 1 < jobs.n && tile_id >= jobs.job[which + 1].first_tile) ++which;
  const GemmJob& j = jobs.job[which];
  const int tile = tile_id - j.first_tile;
  const int m0 = tile / j.tiles_n * T, n0 = tile % j.tiles_n * T;
  const int g = threadIdx.x >> 6, l = threadIdx.x & 63, tx = l & 7, ty = l >> 3;
  float acc[4][4] = {};
  for (int q = 0; q < j.pairs; ++q) {
    const GemmPair& p = j.p[q];
    const int steps = (p.K + GROUPS * KB - 1) / (GROUPS * KB);
    // lanes along whichever index is contiguous
    const bool a_k = p.ak == 1, b_n = p.bn == 1;
    float ra[8], rb[8];
    auto fetch = [&](int step) {
      const int k0 = (step * GROUPS + g) * KB;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = l + 64 * e;  // 512 = 16 k x 32
        const int am = a_k ? i >> 4 : i & 31, ak = a_k ? i & 15 : i >> 5;
        const int bk = b_n ? i >> 5 : i & 15, bn = b_n ? i & 31 : i >> 4;
        ra[e] = m0 + am < j.M && k0 + ak < p.K ? load(p.a, p.a_bf16, (m0 + am) * p.am + (k0 + ak) * p.ak) : 0.f;
        rb[e] = n0 + bn < j.N && k0 + bk < p.K ? load(p.b, p.b_bf16, (k0 + bk) * p.bk + (n0 + bn) * p.bn) : 0.f;
      }
    };
    if (rank < steps) fetch(rank);
    for (int step = rank; step < steps; step += jobs.slices) {
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = l + 64 * e;
        As[g][a_k ? i & 15 : i >> 5][a_k ? i >> 4 : i & 31] = ra[e];
        Bs[g][b_n ? i >> 5 : i & 15][b_n ? i & 31 : i >> 4] = rb[e];
      }
      __syncthreads();
      if (step + jobs.slices < steps) fetch(step + jobs.slices);
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        const float4 a = *reinterpret_cast<const float4*>(&As[g][k][4 * ty]);
        const float4 b = *reinterpret_cast<const float4*>(&Bs[g][k][4 * tx]);
        const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) acc[x][y] = fmaf(av[x], bv[y], acc[x][y]);
      }
    }
  }
  // the groups' sums, over the operand tiles: [group][32][36]
  __syncthreads();
  float* sums = &As[0][0][0] + g * (T * (T + 4) / 2);  // 16 rows' space per group in As, 16 in Bs
  float* more = &Bs[0][0][0] + g * (T * (T + 4) / 2);
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int r = 4 * ty + x;
    float* d = r < 16 ? sums + r * (T + 4) : more + (r - 16) * (T + 4);
    *reinterpret_cast<float4*>(d + 4 * tx) = make_float4(acc[x][0], acc[x][1], acc[x][2], acc[x][3]);
  }
  __syncthreads();
  float v[4];  // of the tile's 1024 elements
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int i = threadIdx.x + THREADS * e;
    const int r = j.cn == 1 ? i >> 5 : i & 31, c = j.cn == 1 ? i & 31 : i >> 5;
    v[e] = 0.f;
#pragma unroll
    for (int k = 0; k < GROUPS; ++k)
      v[e] += (r < 16 ? &As[0][0][0] : &Bs[0][0][0])[k * (T * (T + 4) / 2) + (r & 15) * (T + 4) + c];
  }
  if (jobs.slices > 1) {  // the slices' sums, in order, by the first CTA
    namespace cg = cooperative_groups;
    const cg::cluster_group cluster = cg::this_cluster();
    float* part = &As[0][0][0];
    __syncthreads();
    if (rank != 0)
#pragma unroll
      for (int e = 0; e < 4; ++e) part[threadIdx.x + THREADS * e] = v[e];
    cluster.sync();
    if (rank == 0)
      for (int r = 1; r < jobs.slices; ++r) {
        const float* from = cluster.map_shared_rank(part, r);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += from[threadIdx.x + THREADS * e];
      }
    cluster.sync();
    if (rank != 0) return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int i = threadIdx.x + THREADS * e;
    const int r = j.cn == 1 ? i >> 5 : i & 31, c = j.cn == 1 ? i & 31 : i >> 5;
    if (m0 + r < j.M && n0 + c < j.N) store(j.c, j.c_bf16, (m0 + r) * j.cm + (n0 + c) * j.cn, v[e]);
  }
}

struct Gemms {
  GemmJobs jobs{};
  ll tiles = 0;
  void add(int M, int N, const GemmPair& p, void* c, bool c_bf16, ll cm, ll cn, const GemmPair* p2 = nullptr) {
    if (M == 0 || N == 0) return;
    GemmJob& j = jobs.job[jobs.n++];
    j = GemmJob{M, N, p2 ? 2 : 1, (N + 31) / 32, static_cast<int>(tiles), {p, p2 ? *p2 : GemmPair{}}, c, c_bf16, cm, cn};
    tiles += static_cast<ll>((M + 31) / 32) * j.tiles_n;
  }
  cudaError_t run(cudaStream_t st, const RopeSum& rope = RopeSum{}) {
    int steps = 0;
    for (int i = 0; i < jobs.n; ++i)
      for (int q = 0; q < jobs.job[i].pairs; ++q) steps = std::max(steps, (jobs.job[i].p[q].K + 63) / 64);
    int slices = 1;
    while (steps >= 4 && slices < 4 && 2 * slices <= steps && 4 * slices * tiles <= 9 * sm_count()) slices *= 2;
    const ll ropes = (rope.total + THREADS - 1) / THREADS;
    const ll blocks = (tiles + (ropes + slices - 1) / slices) * slices;
    if (blocks == 0) return cudaSuccess;
    if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
    jobs.slices = slices;
    jobs.rope = rope;
    jobs.rope.first_block = static_cast<int>(tiles * slices);
    return launch_next_in_clusters(slices, small_gemm_kernel, static_cast<unsigned>(blocks), THREADS, 0, st, jobs);
  }
};

// K_nope = c W_UK, V = c W_UV
cudaError_t rebuild(const Dims& d, bool bf, const void* c, const void* W_UK, const void* W_UV, float* kn, float* v,
                    cudaStream_t st) {
  const int M = d.B * d.S;
  const ll nk = static_cast<ll>(d.n_h) * d.d_nope, nv = static_cast<ll>(d.n_h) * d.d_v;
  Gemms g;
  g.add(M, static_cast<int>(nk), GemmPair{c, W_UK, bf, bf, d.d_c, d.d_c, 1, nk, 1}, kn, false, nk, 1);
  g.add(M, static_cast<int>(nv), GemmPair{c, W_UV, bf, bf, d.d_c, d.d_c, 1, nv, 1}, v, false, nv, 1);
  return g.run(st);
}

// dc = dK W_UK^T + dV W_UV^T, dW_UK = c^T dK, dW_UV = c^T dV (k runs over the batch's rows too), dk_rope
cudaError_t rebuild_bwd(const Dims& d, bool bf, const void* c, const void* W_UK, const void* W_UV, const float* dk,
                        const float* dv, const float* dkr, const BwdGrads& o, cudaStream_t st) {
  const int M = d.B * d.S;
  const ll nk = static_cast<ll>(d.n_h) * d.d_nope, nv = static_cast<ll>(d.n_h) * d.d_v;
  Gemms g;
  g.add(d.d_c, static_cast<int>(nk), GemmPair{c, dk, bf, false, M, 1, d.d_c, nk, 1}, o.dW_UK, bf, nk, 1);
  g.add(d.d_c, static_cast<int>(nv), GemmPair{c, dv, bf, false, M, 1, d.d_c, nv, 1}, o.dW_UV, bf, nv, 1);
  const GemmPair second{dv, W_UV, false, bf, static_cast<int>(nv), nv, 1, 1, nv};
  g.add(M, d.d_c, GemmPair{dk, W_UK, false, bf, static_cast<int>(nk), nk, 1, 1, nk}, o.dc_kv, bf, d.d_c, 1, &second);
  return g.run(st, RopeSum{0, static_cast<ll>(M) * d.d_rope, d.n_h, d.d_rope, dkr, o.dk_rope, bf});
}

}  // namespace

size_t simt_masked_fwd_workspace(const Dims& d, int elem) { return bytes(d, elem, false); }
size_t simt_masked_bwd_workspace(const Dims& d, int elem) { return bytes(d, elem, true); }

LaunchResult simt_masked_fwd(const Dims& d, bool is_bf16, const ScoreMods& mods, const int* key_lo, const int* key_hi,
                             const void* q, const void* c_kv, const void* k_rope, const void* W_UK, const void* W_UV,
                             void* out, float* lse, void* ws, cudaStream_t st) {
  char* at = static_cast<char*>(ws);
  const Ws w = carve(d, is_bf16 ? 2 : 4, false, at);
  LaunchResult r = mask_prepare(d, is_bf16, key_lo, key_hi, c_kv, k_rope, w.mask, false, st);
  if (!r.ok()) return r;
  r.err = rebuild(d, is_bf16, w.mask.c_kv, W_UK, W_UV, w.kn, w.v, st);
  if (r.err != cudaSuccess) {
    r.what = "K/V rebuild (CUDA cores)";
    return r;
  }
  SimtParams p = params(d, is_bf16, mods, w);
  p.q = q;
  p.q_bf16 = is_bf16;
  p.out = out;
  p.lse = lse;
  r.err = launch<false>(d, p, st);
  if (r.err != cudaSuccess) r.what = "masked attention forward (CUDA cores)";
  return r;
}

LaunchResult simt_masked_bwd(const Dims& d, bool is_bf16, const ScoreMods& mods, const int* key_lo, const int* key_hi,
                             const void* q, const void* c_kv, const void* k_rope, const void* W_UK, const void* W_UV,
                             const void* out, const Packed* q8, const Packed* out8, const float* lse,
                             const void* dout, const BwdGrads& g, void* ws, bool reuse_kv, cudaStream_t st) {
  char* at = static_cast<char*>(ws);
  const Ws w = carve(d, is_bf16 ? 2 : 4, true, at);
  LaunchResult r;
  if (!reuse_kv) r = mask_prepare(d, is_bf16, key_lo, key_hi, c_kv, k_rope, w.mask, false, st);
  if (r.ok() && !reuse_kv) {
    r.err = rebuild(d, is_bf16, w.mask.c_kv, W_UK, W_UV, w.kn, w.v, st);
    if (r.err != cudaSuccess) r.what = "K/V rebuild (CUDA cores)";
  }
  if (r.ok()) r = simt_mask_bwd_pre(d, is_bf16, q, out, q8, out8, dout, lse, w.lse_row, w.delta, w.q, w.dout, !reuse_kv, st);
  if (!r.ok()) return r;
  SimtParams p = params(d, is_bf16, mods, w);
  p.q = w.q;
  p.q_bf16 = false;
  p.dout = w.dout;
  p.lse_row = w.lse_row;
  p.delta = w.delta;
  p.out = g.dq;
  p.dkn = w.dkn;
  p.dv = w.dv;
  p.dkr = w.dkr;
  r.err = launch<true>(d, p, st);
  if (r.err != cudaSuccess) {
    r.what = "masked attention backward (CUDA cores)";
    return r;
  }
  r.err = rebuild_bwd(d, is_bf16, w.mask.c_kv, W_UK, W_UV, w.dkn, w.dv, w.dkr, g, st);
  if (r.err != cudaSuccess) r.what = "rebuild backward (CUDA cores)";
  return r;
}

}  // namespace laga
