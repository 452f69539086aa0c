// Masked attention on the CUDA cores in fp32, for any head widths up to 256: the
// forward, dq and dK/dV. Tiles of 64 rows by 64 (forward) or 32 (backward) columns
// live in shared memory; one pass over the keys with the running maximum and sum of
// the softmax; O, dq, dK and dV stay in registers. Rows are stored with a pitch of an
// odd number of 16-byte units, so the 16 threads that read 16 consecutive rows as
// float4 touch different banks.
//
// Thread (tx, ty) of 16 x 16 owns tile rows 4 ty .. 4 ty + 3 and, of the score tile,
// columns tx, tx + 16, ...; of a head-wide accumulator, columns 64 c + 4 tx .. + 3.
// Every element of the shared dimension costs a thread 8 (4 + 4) 16-byte loads per 64
// multiply-adds in the 64 x 64 score product. N = ceil(widest head / 64) picks the
// accumulator's width.
#include "mask.h"

#include <algorithm>
#include <type_traits>

namespace laga {
namespace {

using ll = long long;
constexpr int ROWS = 64;     // tile rows: queries (forward, dq) or keys (dK/dV)
constexpr int KFWD = 64;     // keys per step, forward
constexpr int KBWD = 32;     // keys (dq) or queries (dK/dV) per step
constexpr int THREADS = 256;

__host__ __device__ __forceinline__ int pitch4(int width) { return ((width + 3) / 4) | 1; }  // in float4

struct SimtParams {
  Dims d;
  const void* q;         // [B][Sq][n_h][d_qk]; the forward's in the inputs' type, else fp32
  bool q_bf16;
  const float* kn;       // [B][S][n_h][d_nope]
  const float* v;        // [B][S][n_h][d_v]
  const void* k_rope;    // [B][S][d_rope], the inputs' type
  bool rope_bf16;
  const int2* rows;      // [B][sq_pad]
  const int2* q_hull;    // [B][sq_pad / 64]
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

// dst[r][k] = get(r, k) for r < rows, k < width, zero up to the next multiple of four.
template <class F>
__device__ __forceinline__ void fill(float4* dst, int pitch, int rows, int width, F&& get) {
  const int w = (width + 3) & ~3;
  float* f = reinterpret_cast<float*>(dst);
  for (int e = threadIdx.x; e < rows * w; e += THREADS) {
    const int r = e / w, k = e - r * w;
    f[r * pitch * 4 + k] = k < width ? get(r, k) : 0.f;
  }
}

__device__ __forceinline__ float dot4(float4 a, float4 b, float acc) {
  acc = fmaf(a.x, b.x, acc);
  acc = fmaf(a.y, b.y, acc);
  acc = fmaf(a.z, b.z, acc);
  return fmaf(a.w, b.w, acc);
}

// acc[i][j] += sum_k A[4 ty + i][k] B[tx + 16 j][k]
template <int NJ>
__device__ __forceinline__ void score_tile(const float4* A, const float4* B, int pitch, int n4, int tx, int ty,
                                           float (&acc)[4][NJ]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = 0.f;
  for (int k = 0; k < n4; ++k) {
    float4 a[4], b[NJ];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = A[(4 * ty + i) * pitch + k];
#pragma unroll
    for (int j = 0; j < NJ; ++j) b[j] = B[(tx + 16 * j) * pitch + k];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = dot4(a[i], b[j], acc[i][j]);
  }
}

// acc[i][c] += sum_n Wt[n][4 ty + i] B[n][64 c + 4 tx ..]; Wt has a pitch of 17 float4
template <int N>
__device__ __forceinline__ void weighted_rows(const float4* Wt, const float4* B, int pitch, int count, int width4, int tx,
                                              int ty, float4 (&acc)[4][N]) {
  for (int n = 0; n < count; ++n) {
    const float4 w = Wt[n * 17 + ty];
    const float wi[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int c = 0; c < N; ++c) {
      if (16 * c + tx >= width4) continue;
      const float4 b = B[n * pitch + 16 * c + tx];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
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

__device__ __forceinline__ void load_k(const SimtParams& p, float4* dst, int pitch, int b, int h, int first, int rows) {
  const Dims& d = p.d;
  fill(dst, pitch, rows, d.d_qk(), [&](int r, int k) {
    const int j = first + r;
    if (j >= d.S) return 0.f;
    const ll row = static_cast<ll>(b) * d.S + j;
    return k < d.d_nope ? p.kn[(row * d.n_h + h) * d.d_nope + k]
                        : load(p.k_rope, p.rope_bf16, row * d.d_rope + (k - d.d_nope));
  });
}
__device__ __forceinline__ void load_v(const SimtParams& p, float4* dst, int pitch, int b, int h, int first, int rows) {
  const Dims& d = p.d;
  fill(dst, pitch, rows, d.d_v, [&](int r, int k) {
    const int j = first + r;
    return j < d.S ? p.v[((static_cast<ll>(b) * d.S + j) * d.n_h + h) * d.d_v + k] : 0.f;
  });
}
__device__ __forceinline__ void load_q(const SimtParams& p, float4* dst, int pitch, int b, int h, int first, int rows) {
  const Dims& d = p.d;
  fill(dst, pitch, rows, d.d_qk(), [&](int r, int k) {
    const int i = first + r;
    return i < d.Sq ? load(p.q, p.q_bf16, ((static_cast<ll>(b) * d.Sq + i) * d.n_h + h) * d.d_qk() + k) : 0.f;
  });
}
__device__ __forceinline__ void load_do(const SimtParams& p, float4* dst, int pitch, int b, int h, int first, int rows) {
  const Dims& d = p.d;
  fill(dst, pitch, rows, d.d_v, [&](int r, int k) {
    const int i = first + r;
    return i < d.Sq ? p.dout[((static_cast<ll>(b) * d.Sq + i) * d.n_h + h) * d.d_v + k] : 0.f;
  });
}

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

// out and lse of 64 query rows of one head.
template <int N>
__global__ void __launch_bounds__(THREADS) masked_simt_fwd(const SimtParams p) {
  extern __shared__ float4 sm[];
  const Dims& d = p.d;
  const int pk = pitch4(d.d_qk()), pv = pitch4(d.d_v);
  float4 *sq = sm, *sk = sq + ROWS * pk, *sv = sk + KFWD * pk, *sp = sv + KFWD * pv;
  const int t = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int i0 = t * ROWS + 4 * ty;  // this thread's first row
  load_q(p, sq, pk, b, h, t * ROWS, ROWS);
  int lo[4], hi[4];
  bool poisoned[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int2 v = p.rows[static_cast<ll>(b) * d.sq_pad + i0 + i];
    poisoned[i] = v.x < 0;
    lo[i] = v.x & 0x7fffffff;
    hi[i] = v.y;
  }
  const float slope = p.slopes ? p.slopes[h] : 0.f;
  float m[4], l[4];
  float4 o[4][N];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < N; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const int2 hull = p.q_hull[static_cast<ll>(b) * (d.sq_pad / ROWS) + t];
  for (int j0 = hull.x < hull.y ? hull.x / KFWD * KFWD : 0; j0 < hull.y; j0 += KFWD) {
    __syncthreads();
    load_k(p, sk, pk, b, h, j0, KFWD);
    load_v(p, sv, pv, b, h, j0, KFWD);
    __syncthreads();
    float s[4][4];
    score_tile(sq, sk, pk, (d.d_qk() + 3) / 4, tx, ty, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
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
    for (int j = 0; j < 4; ++j) sp[(tx + 16 * j) * 17 + ty] = make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
    __syncthreads();
    weighted_rows<N>(sp, sv, pv, KFWD, (d.d_v + 3) / 4, tx, ty, o);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i0 + i >= d.Sq) continue;
    float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
    float L = l[i] == 0.f ? -INFINITY : m[i] + logf(l[i]);
    if (poisoned[i]) inv = L = NAN;
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

// dq of 64 query rows of one head.
template <int N>
__global__ void __launch_bounds__(THREADS) masked_simt_dq(const SimtParams p) {
  extern __shared__ float4 sm[];
  const Dims& d = p.d;
  const int pk = pitch4(d.d_qk()), pv = pitch4(d.d_v);
  float4 *sq = sm, *sdo = sq + ROWS * pk, *sk = sdo + ROWS * pv, *sv = sk + KBWD * pk, *sds = sv + KBWD * pv;
  const int t = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int i0 = t * ROWS + 4 * ty;
  load_q(p, sq, pk, b, h, t * ROWS, ROWS);
  load_do(p, sdo, pv, b, h, t * ROWS, ROWS);
  int lo[4], hi[4];
  float L[4], D[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int2 v = p.rows[static_cast<ll>(b) * d.sq_pad + i0 + i];
    lo[i] = v.x & 0x7fffffff;
    hi[i] = v.y;
    const bool in = i0 + i < d.Sq;
    const ll at = (static_cast<ll>(b) * d.n_h + h) * d.Sq + i0 + i;
    L[i] = in ? p.lse_row[at] : INFINITY;
    D[i] = in ? p.delta[at] : 0.f;
  }
  const float slope = p.slopes ? p.slopes[h] : 0.f;
  float4 acc[4][N];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < N; ++c) acc[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int2 hull = p.q_hull[static_cast<ll>(b) * (d.sq_pad / ROWS) + t];
  for (int j0 = hull.x < hull.y ? hull.x / KBWD * KBWD : 0; j0 < hull.y; j0 += KBWD) {
    __syncthreads();
    load_k(p, sk, pk, b, h, j0, KBWD);
    load_v(p, sv, pv, b, h, j0, KBWD);
    __syncthreads();
    float s[4][2], dp[4][2];
    score_tile(sq, sk, pk, (d.d_qk() + 3) / 4, tx, ty, s);
    score_tile(sdo, sv, pv, (d.d_v + 3) / 4, tx, ty, dp);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
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
    for (int j = 0; j < 2; ++j) sds[(tx + 16 * j) * 17 + ty] = make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
    __syncthreads();
    weighted_rows<N>(sds, sk, pk, KBWD, (d.d_qk() + 3) / 4, tx, ty, acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
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

// dK (both parts) and dV of 64 keys of one head.
template <int N>
__global__ void __launch_bounds__(THREADS) masked_simt_dkv(const SimtParams p) {
  extern __shared__ float4 sm[];
  const Dims& d = p.d;
  const int pk = pitch4(d.d_qk()), pv = pitch4(d.d_v);
  float4 *sk = sm, *sv = sk + ROWS * pk, *sq = sv + ROWS * pv, *sdo = sq + KBWD * pk, *sp = sdo + KBWD * pv;
  float4* sds = sp + KBWD * 17;
  const int t = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int k0 = t * ROWS + 4 * ty;  // this thread's first key
  load_k(p, sk, pk, b, h, t * ROWS, ROWS);
  load_v(p, sv, pv, b, h, t * ROWS, ROWS);
  const float slope = p.slopes ? p.slopes[h] : 0.f;
  float4 dk[4][N], dv[4][N];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < N; ++c) dk[i][c] = dv[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int nq64 = d.sq_pad / 64;
  for (int q0 = 0; q0 < d.Sq; q0 += KBWD) {
    const int2 hull = p.q_hull[static_cast<ll>(b) * nq64 + q0 / 64];
    if (hull.x >= hull.y || hull.x >= (t + 1) * ROWS || hull.y <= t * ROWS) continue;  // the same for every thread
    __syncthreads();
    load_q(p, sq, pk, b, h, q0, KBWD);
    load_do(p, sdo, pv, b, h, q0, KBWD);
    __syncthreads();
    float s[4][2], dp[4][2];
    score_tile(sk, sq, pk, (d.d_qk() + 3) / 4, tx, ty, s);
    score_tile(sv, sdo, pv, (d.d_v + 3) / 4, tx, ty, dp);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int i = q0 + tx + 16 * j;
      const int2 r = p.rows[static_cast<ll>(b) * d.sq_pad + i];  // {0, 0} past Sq
      const bool in = i < d.Sq;
      const ll at = (static_cast<ll>(b) * d.n_h + h) * d.Sq + i;
      const float L = in ? p.lse_row[at] : INFINITY, D = in ? p.delta[at] : 0.f;
      const int pos = position(d, i);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int key = k0 + k;
        float dcap = 1.f;
        const float v = score_of(p, s[k][j], slope, pos, key, &dcap);
        const float e = key >= (r.x & 0x7fffffff) && key < r.y ? expf(v - L) : 0.f;
        s[k][j] = e;
        dp[k][j] = e * (dp[k][j] - D) * dcap;
      }
      sp[(tx + 16 * j) * 17 + ty] = make_float4(s[0][j], s[1][j], s[2][j], s[3][j]);
      sds[(tx + 16 * j) * 17 + ty] = make_float4(dp[0][j], dp[1][j], dp[2][j], dp[3][j]);
    }
    __syncthreads();
    weighted_rows<N>(sp, sdo, pv, KBWD, (d.d_v + 3) / 4, tx, ty, dv);
    weighted_rows<N>(sds, sq, pk, KBWD, (d.d_qk() + 3) / 4, tx, ty, dk);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
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

// dk_rope[b, j, :] = the heads' RoPE-key gradients summed, in order.
template <typename T>
__global__ void masked_simt_rope_sum(ll total, int n_h, int d_rope, const float* __restrict__ dkr, T* __restrict__ dk_rope) {
  const ll idx = static_cast<ll>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (idx >= total) return;
  const ll bj = idx / d_rope;
  const int k = static_cast<int>(idx - bj * d_rope);
  float acc = 0.f;
  for (int h = 0; h < n_h; ++h) acc += dkr[(bj * n_h + h) * d_rope + k];
  dk_rope[idx] = static_cast<T>(acc);
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
  w.kn = take(keys * d.d_nope);  // first: what a backward that reuses the forward's rebuild reads
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
  p.cap = mods.cap;
  p.inv_cap = mods.cap > 0.f ? 1.f / mods.cap : 0.f;
  p.slopes = mods.slopes;
  p.out_bf16 = is_bf16;
  return p;
}

// Launches kern<1>, <2> or <4> by the widest head.
template <class F1, class F2, class F4>
cudaError_t launch(const Dims& d, F1 k1, F2 k2, F4 k4, dim3 grid, size_t smem, const SimtParams& p, cudaStream_t st) {
  const int w = std::max(d.d_qk(), d.d_v);
  void (*kern)(SimtParams) = w <= 64 ? k1 : w <= 128 ? k2 : k4;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  kern<<<grid, THREADS, smem, st>>>(p);
  return cudaGetLastError();
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
  if (r.ok()) r = simt_reconstruct(d, is_bf16, w.mask.c_kv, W_UK, W_UV, w.kn, w.v, true, st);
  if (!r.ok()) return r;
  SimtParams p = params(d, is_bf16, mods, w);
  p.q = q;
  p.q_bf16 = is_bf16;
  p.out = out;
  p.lse = lse;
  const int pk = pitch4(d.d_qk()), pv = pitch4(d.d_v);
  const size_t smem = sizeof(float4) * ((ROWS + KFWD) * pk + KFWD * pv + KFWD * 17);
  r.err = launch(d, masked_simt_fwd<1>, masked_simt_fwd<2>, masked_simt_fwd<4>,
                 dim3((d.Sq + ROWS - 1) / ROWS, d.n_h, d.B), smem, p, st);
  if (r.err != cudaSuccess) r.what = "masked attention forward (CUDA cores)";
  return r;
}

LaunchResult simt_masked_bwd(const Dims& d, bool is_bf16, const ScoreMods& mods, const int* key_lo, const int* key_hi,
                             const void* q, const void* c_kv, const void* k_rope, const void* W_UK, const void* W_UV,
                             const void* out, const Packed* q8, const Packed* out8, const float* lse,
                             const void* dout, const BwdGrads& g, void* ws, bool reuse_kv, cudaStream_t st) {
  char* at = static_cast<char*>(ws);
  const Ws w = carve(d, is_bf16 ? 2 : 4, true, at);
  LaunchResult r = mask_prepare(d, is_bf16, key_lo, key_hi, c_kv, k_rope, w.mask, false, st);
  if (r.ok() && !reuse_kv) r = simt_reconstruct(d, is_bf16, w.mask.c_kv, W_UK, W_UV, w.kn, w.v, true, st);
  if (r.ok()) r = simt_mask_bwd_pre(d, is_bf16, q, out, q8, out8, dout, lse, w.lse_row, w.delta, w.q, w.dout, st);
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
  const int pk = pitch4(d.d_qk()), pv = pitch4(d.d_v);
  const size_t both = sizeof(float4) * (ROWS + KBWD) * (pk + pv);
  r.err = launch(d, masked_simt_dq<1>, masked_simt_dq<2>, masked_simt_dq<4>, dim3((d.Sq + ROWS - 1) / ROWS, d.n_h, d.B),
                 both + sizeof(float4) * KBWD * 17, p, st);
  if (r.err == cudaSuccess)
    r.err = launch(d, masked_simt_dkv<1>, masked_simt_dkv<2>, masked_simt_dkv<4>,
                   dim3((d.S + ROWS - 1) / ROWS, d.n_h, d.B), both + sizeof(float4) * 2 * KBWD * 17, p, st);
  const ll nr = static_cast<ll>(d.B) * d.S * d.d_rope;
  if (r.err == cudaSuccess && nr > 0) {
    const unsigned grid = static_cast<unsigned>((nr + 255) / 256);
    if (is_bf16)
      masked_simt_rope_sum<bf16><<<grid, 256, 0, st>>>(nr, d.n_h, d.d_rope, w.dkr, static_cast<bf16*>(g.dk_rope));
    else
      masked_simt_rope_sum<float><<<grid, 256, 0, st>>>(nr, d.n_h, d.d_rope, w.dkr, static_cast<float*>(g.dk_rope));
    r.err = cudaGetLastError();
  }
  if (r.err != cudaSuccess) {
    r.what = "masked attention backward (CUDA cores)";
    return r;
  }
  return simt_rebuild_bwd(d, is_bf16, w.mask.c_kv, W_UK, W_UV, w.dkn, w.dv, g.dc_kv, g.dW_UK, g.dW_UV, st);
}

}  // namespace laga
