// RMS norms of the query heads and of the shared RoPE key, with the rotation in the same pass, and
// their gradients.
//
//   y = x r w,  r = 1 / sqrt(mean(x^2) + eps);   z = R y, R the rotation of the row's RoPE part
//   dy = R^T dz;  g = dy w;  xh = x r;  dx = r (g - xh mean(g xh));  dw = sum over rows of dy xh
//
// The backward makes r again from x, which it has to read for xh anyhow: nothing is kept between the
// two. Sums are fp32; each result is rounded once. dw: every thread sums its columns over its rows,
// the CTA's threads are added up in a fixed order into one row of `partials`, and a second launch adds
// those rows up: no atomics, the same bits every time.
//
// Memory bound: a row is held in registers between its sum and its result, so each value is read once
// and written once. Eight lanes share a row (24 chunks of 16 bytes for a bf16 head of 192: three a
// lane), so that a sum takes three shuffles and a warp has four rows in flight; rows wider than 24
// chunks take a whole warp.
#include "rope_device.cuh"

#include <algorithm>

namespace laga {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int BWD_CTAS_PER_SM = 4;

// x^2 of a value above 2^60 leaves fp32 in a sum of 1024: such rows are scaled down first.
constexpr float kBigSum = 0x1p120f;
constexpr float kDown = 0x1p-70f;

template <int LANES>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int m = LANES / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// What turns a row: `down` and then `r` bring it to root mean square 1.
struct Scale {
  float down, r;
};
template <int LANES, class F>
__device__ __forceinline__ Scale row_scale(float sum, float inv_d, float eps, F&& sum_scaled) {
  Scale s{1.f, 0.f};
  if (__any_sync(0xffffffffu, !(sum < kBigSum))) {
    const float again = sum_lanes<LANES>(sum_scaled(kDown));
    if (!(sum < kBigSum)) {
      s.down = kDown;
      sum = again;
    }
  }
  s.r = rsqrtf(fmaf(sum, inv_d, eps * s.down * s.down));
  return s;
}

// The geometry of one kind of rows (the query heads, or the keys), in chunks of N values.
struct RowShape {
  int chunks, nope, half;  // all of the row; before the RoPE part; half of the RoPE part
  float inv_d;
};

template <typename T, bool INTERLEAVED, int LANES, int K>
struct RowOps {
  using V = Vec<T>;
  static constexpr int N = V::N;

  // What a lane keeps of a row: its chunks, and for the layout in halves their partners.
  struct Held {
    uint4 own[K], other[INTERLEAVED ? 1 : K];
  };
  static __device__ __forceinline__ int partner(const RowShape& s, int c) {
    return c - s.nope < s.half ? c + s.half : c - s.half;
  }
  static __device__ __forceinline__ void load(const T* row, const RowShape& s, int l, bool active, bool partners,
                                              Held& h) {
    const uint4* p = reinterpret_cast<const uint4*>(row);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = l + LANES * k;
      const bool there = active && c < s.chunks;
      h.own[k] = there ? __ldcs(p + c) : make_uint4(0, 0, 0, 0);
      if constexpr (!INTERLEAVED)
        h.other[k] = partners && there && c >= s.nope ? __ldcs(p + partner(s, c)) : make_uint4(0, 0, 0, 0);
    }
  }
  // The turned values of chunk c: v and, in halves, o (already weighted) are its own and its partner's.
  // sign -1 turns back.
  static __device__ __forceinline__ void turn(const RowShape& s, int c, const float2* cs, float sign, float (&v)[N],
                                              const float (&o)[N]) {
    if (c < s.nope) return;
    if constexpr (INTERLEAVED) {
      const float2* w = cs + (c - s.nope) * (N / 2);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const float a = v[2 * i], b = v[2 * i + 1], sn = sign * w[i].y;
        v[2 * i] = a * w[i].x - b * sn;
        v[2 * i + 1] = a * sn + b * w[i].x;
      }
    } else {
      const int u = c - s.nope;
      const bool first = u < s.half;
      const float2* w = cs + (first ? u : u - s.half) * N;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float sn = sign * w[i].y;
        v[i] = first ? v[i] * w[i].x - o[i] * sn : o[i] * sn + v[i] * w[i].x;
      }
    }
  }
  static __device__ __forceinline__ float squares(const Held& h, float by) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float v[N];
      V::get(h.own[k], v);
#pragma unroll
      for (int i = 0; i < N; ++i) sum = fmaf(v[i] * by, v[i] * by, sum);
    }
    return sum;
  }

  static __device__ __forceinline__ void forward(const T* src, T* dst, const RowShape& s, const float* w,
                                                 const float2* cs, float eps, int l, bool active) {
    Held h;
    load(src, s, l, active, true, h);
    const float sum = sum_lanes<LANES>(squares(h, 1.f));
    const Scale sc = row_scale<LANES>(sum, s.inv_d, eps, [&](float by) { return squares(h, by); });
    __syncwarp();  // in place: every lane of the row has loaded
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = l + LANES * k;
      if (!active || c >= s.chunks) continue;
      float v[N], o[N];
      V::get(h.own[k], v);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = v[i] * sc.down * sc.r * w[c * N + i];
      if constexpr (!INTERLEAVED) {
        if (c >= s.nope) {
          const float* wo = w + partner(s, c) * N;
          V::get(h.other[k], o);
#pragma unroll
          for (int i = 0; i < N; ++i) o[i] = o[i] * sc.down * sc.r * wo[i];
        }
      }
      turn(s, c, cs, 1.f, v, o);
      reinterpret_cast<uint4*>(dst)[c] = V::put(v);
    }
  }

  static __device__ __forceinline__ void backward(const T* src, const T* grad, T* dst, const RowShape& s,
                                                  const float* w, const float2* cs, float eps, int l, bool active,
                                                  float (&acc)[K][N]) {
    Held x, z;
    load(src, s, l, active, false, x);
    load(grad, s, l, active, true, z);
    const float sum = sum_lanes<LANES>(squares(x, 1.f));
    const Scale sc = row_scale<LANES>(sum, s.inv_d, eps, [&](float by) { return squares(x, by); });
    float dot = 0.f, dy[K][N];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = l + LANES * k;
      float v[N], o[N];
      V::get(z.own[k], dy[k]);
      if (!active || c >= s.chunks) continue;
      if constexpr (!INTERLEAVED) V::get(z.other[k], o);
      turn(s, c, cs, -1.f, dy[k], o);
      V::get(x.own[k], v);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float xh = v[i] * sc.down * sc.r, p = dy[k][i] * xh;
        acc[k][i] += p;
        dot = fmaf(p, w[c * N + i], dot);
      }
    }
    const float mean = sum_lanes<LANES>(dot) * s.inv_d;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = l + LANES * k;
      if (!active || c >= s.chunks) continue;
      float v[N];
      V::get(x.own[k], v);
#pragma unroll
      for (int i = 0; i < N; ++i)
        v[i] = sc.down * sc.r * (dy[k][i] * w[c * N + i] - v[i] * sc.down * sc.r * mean);
      reinterpret_cast<uint4*>(dst)[c] = V::put(v);
    }
  }
};

// CTA partial sums of one weight: acc of all its threads, columns [c N, c N + N) at a lane's chunk c.
template <typename T, int LANES, int K>
__device__ __forceinline__ void reduce_columns(float (&acc)[K][Vec<T>::N], const RowShape& s, float* red, float* out) {
  constexpr int N = Vec<T>::N;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = s.chunks * N;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int m = LANES; m < 32; m <<= 1) acc[k][i] += __shfl_xor_sync(0xffffffffu, acc[k][i], m);
  if (lane < LANES)
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (const int c = lane + LANES * k; c < s.chunks)
#pragma unroll
        for (int i = 0; i < N; ++i) red[warp * d + c * N + i] = acc[k][i];
  __syncthreads();
  for (int c = threadIdx.x; c < d; c += THREADS) {
    float sum = 0.f;
    for (int j = 0; j < WARPS; ++j) sum += red[j * d + c];
    out[c] = sum;
  }
  __syncthreads();
}

// Rows of 16-byte chunks. A CTA takes `per` tokens at a time (their cosines and sines once, for all
// heads), the forward's one such group, the backward's every gridDim-th.
template <typename T, bool INTERLEAVED, int LANES, int K, bool BWD>
__global__ void __launch_bounds__(THREADS) norm_vec_kernel(const NormArgs a, const RopeTable t, int per) {
  using R = RowOps<T, INTERLEAVED, LANES, K>;
  constexpr int N = R::N, ROWS = 32 / LANES;  // rows of a warp
  extern __shared__ float smem[];
  const RopeArgs& p = a.rope;
  const int d = p.d_nope + p.d_rope, n = p.d_rope / 2;
  float* w = smem;                                         // [d], then the keys' [d_rope]
  float2* cs = reinterpret_cast<float2*>(smem + ((d + p.d_rope + 3) & ~3));  // [per][n]
  float* red = reinterpret_cast<float*>(cs + per * n);     // backward: [WARPS][d]
  after_previous();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LANES;
  if (p.q)
    for (int i = threadIdx.x; i < d; i += THREADS) w[i] = to_f(static_cast<const T*>(a.w_q)[i]);
  if (p.k)
    for (int i = threadIdx.x; i < p.d_rope; i += THREADS) w[d + i] = to_f(static_cast<const T*>(a.w_k)[i]);
  const ll groups = (p.tokens + per - 1) / per;
  for (int kind = 0; kind < 2; ++kind) {
    const void* src = kind ? p.k : p.q;
    if (!src) continue;
    const int heads = kind ? 1 : p.n_h, nope = kind ? 0 : p.d_nope, width = nope + p.d_rope;
    const RowShape s{width / N, nope / N, n / N, 1.f / width};
    const T* in = static_cast<const T*>(src);
    const T* grad = static_cast<const T*>(kind ? a.z_k : a.z_q);
    T* out = static_cast<T*>(kind ? p.k_out : p.q_out);
    const float* wk = w + (kind ? d : 0);
    float acc[K][N];
    if constexpr (BWD)
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) acc[k][i] = 0.f;
    for (ll g = blockIdx.x; g < groups; g += gridDim.x) {
      const ll first = g * per;
      const int tokens = static_cast<int>(min(static_cast<ll>(per), p.tokens - first));
      if (BWD || kind == 0 || !p.q) {  // else the first pass' angles stand
        __syncthreads();
        fill_angles<THREADS>(p, t, first, tokens, cs);
        __syncthreads();
      }
      const int rows = tokens * heads;
      const ll base = first * heads * width;
      for (int r0 = warp * ROWS; r0 < rows; r0 += WARPS * ROWS) {
        const int row = r0 + lane / LANES;
        const bool active = row < rows;
        const ll at = base + static_cast<ll>(active ? row : 0) * width;
        const float2* angles = cs + (active ? row / heads : 0) * n;
        if constexpr (BWD)
          R::backward(in + at, grad + at, out + at, s, wk, angles, a.eps, l, active, acc);
        else
          R::forward(in + at, out + at, s, wk, angles, a.eps, l, active);
      }
    }
    if constexpr (BWD) {
      __syncthreads();
      // rows of partials: all CTAs' queries, then all CTAs' keys
      float* to = a.partials + (kind ? static_cast<ll>(gridDim.x) * d : 0) + static_cast<ll>(blockIdx.x) * width;
      reduce_columns<T, LANES, K>(acc, s, red, to);
    }
  }
}

// One value at a time: any widths up to kNormWidth and any alignment. A warp takes a row; a lane owns
// pairs of the RoPE part and single values of the rest, the same columns in every row.
template <typename T, bool BWD>
__global__ void __launch_bounds__(THREADS) norm_any_kernel(const NormArgs a, const RopeTable t, int per) {
  extern __shared__ float smem[];
  const RopeArgs& p = a.rope;
  const int n = p.d_rope / 2, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = p.d_nope + p.d_rope;
  float2* cs = reinterpret_cast<float2*>(smem);
  float* red = reinterpret_cast<float*>(cs + per * n);  // backward: [WARPS][d]
  after_previous();
  const ll groups = (p.tokens + per - 1) / per;
  for (int kind = 0; kind < 2; ++kind) {
    const void* src = kind ? p.k : p.q;
    if (!src) continue;
    const int heads = kind ? 1 : p.n_h, nope = kind ? 0 : p.d_nope, width = nope + p.d_rope;
    const float inv_d = 1.f / width;
    const T* w = static_cast<const T*>(kind ? a.w_k : a.w_q);
    float* mine = red + warp * width;
    if constexpr (BWD) {
      __syncthreads();
      for (int i = lane; i < width; i += 32) mine[i] = 0.f;
      __syncwarp();  // the columns' owners are other lanes than those that clear them
    }
    // the two columns of pair u
    auto pair = [&](int u, int& i0, int& i1) {
      i0 = nope + (p.interleaved ? 2 * u : u);
      i1 = nope + (p.interleaved ? 2 * u + 1 : n + u);
    };
    for (ll g = blockIdx.x; g < groups; g += gridDim.x) {
      const ll first = g * per;
      const int tokens = static_cast<int>(min(static_cast<ll>(per), p.tokens - first));
      __syncthreads();
      fill_angles<THREADS>(p, t, first, tokens, cs);
      __syncthreads();
      for (int row = warp; row < tokens * heads; row += WARPS) {
        const ll at = (first * heads + row) * width;
        const T* x = static_cast<const T*>(src) + at;
        T* out = static_cast<T*>(kind ? p.k_out : p.q_out) + at;
        const float2* c = cs + (row / heads) * n;
        auto squares = [&](float by) {
          float sum = 0.f;
          for (int i = lane; i < width; i += 32) sum = fmaf(to_f(x[i]) * by, to_f(x[i]) * by, sum);
          return sum;
        };
        const float sum = sum_lanes<32>(squares(1.f));
        const Scale s = row_scale<32>(sum, inv_d, a.eps, squares);
        if constexpr (!BWD) {
          __syncwarp();  // in place: every lane has read the row
          for (int i = lane; i < nope; i += 32) out[i] = static_cast<T>(to_f(x[i]) * s.down * s.r * to_f(w[i]));
          for (int u = lane; u < n; u += 32) {
            int i0, i1;
            pair(u, i0, i1);
            const float y0 = to_f(x[i0]) * s.down * s.r * to_f(w[i0]), y1 = to_f(x[i1]) * s.down * s.r * to_f(w[i1]);
            out[i0] = static_cast<T>(y0 * c[u].x - y1 * c[u].y);
            out[i1] = static_cast<T>(y0 * c[u].y + y1 * c[u].x);
          }
        } else {
          const T* z = static_cast<const T*>(kind ? a.z_k : a.z_q) + at;
          float dot = 0.f;
          for (int i = lane; i < nope; i += 32) {
            const float v = to_f(z[i]) * (to_f(x[i]) * s.down * s.r);
            mine[i] += v;
            dot = fmaf(v, to_f(w[i]), dot);
          }
          for (int u = lane; u < n; u += 32) {
            int i0, i1;
            pair(u, i0, i1);
            const float z0 = to_f(z[i0]), z1 = to_f(z[i1]);
            const float v0 = (z0 * c[u].x + z1 * c[u].y) * (to_f(x[i0]) * s.down * s.r);
            const float v1 = (z1 * c[u].x - z0 * c[u].y) * (to_f(x[i1]) * s.down * s.r);
            mine[i0] += v0;
            mine[i1] += v1;
            dot = fmaf(v0, to_f(w[i0]), fmaf(v1, to_f(w[i1]), dot));
          }
          const float mean = sum_lanes<32>(dot) * inv_d, r = s.down * s.r;
          __syncwarp();
          for (int i = lane; i < nope; i += 32)
            out[i] = static_cast<T>(r * (to_f(z[i]) * to_f(w[i]) - to_f(x[i]) * s.down * s.r * mean));
          for (int u = lane; u < n; u += 32) {
            int i0, i1;
            pair(u, i0, i1);
            const float z0 = to_f(z[i0]), z1 = to_f(z[i1]), x0 = to_f(x[i0]), x1 = to_f(x[i1]);
            out[i0] = static_cast<T>(r * ((z0 * c[u].x + z1 * c[u].y) * to_f(w[i0]) - x0 * s.down * s.r * mean));
            out[i1] = static_cast<T>(r * ((z1 * c[u].x - z0 * c[u].y) * to_f(w[i1]) - x1 * s.down * s.r * mean));
          }
        }
      }
    }
    if constexpr (BWD) {
      __syncthreads();
      float* to = a.partials + (kind ? static_cast<ll>(gridDim.x) * d : 0) + static_cast<ll>(blockIdx.x) * width;
      for (int i = threadIdx.x; i < width; i += THREADS) {
        float sum = 0.f;
        for (int j = 0; j < WARPS; ++j) sum += red[j * width + i];
        to[i] = sum;
      }
      __syncthreads();
    }
  }
}

// dw of the queries' (blockIdx.y 0) or the keys' weight: the CTAs' partials, 32 columns a CTA.
template <typename T>
__global__ void __launch_bounds__(THREADS) norm_dw_kernel(const float* partials, int ctas, int d, int d_rope, T* dw_q,
                                                          T* dw_k) {
  __shared__ float red[WARPS][32];
  after_previous();
  T* out = blockIdx.y ? dw_k : dw_q;
  const int width = blockIdx.y ? d_rope : d, col = blockIdx.x * 32 + (threadIdx.x & 31), j = threadIdx.x >> 5;
  if (!out || static_cast<int>(blockIdx.x * 32) >= width) return;
  const float* p = partials + (blockIdx.y ? static_cast<ll>(ctas) * d : 0) + col;
  float sum = 0.f;
  if (col < width)
    for (int k = j; k < ctas; k += WARPS) sum += __ldcg(p + static_cast<ll>(k) * width);
  red[j][threadIdx.x & 31] = sum;
  __syncthreads();
  if (j == 0 && col < width) {
    for (int k = 1; k < WARPS; ++k) sum += red[k][threadIdx.x];
    out[col] = static_cast<T>(sum);
  }
}

template <typename T, int LANES, int K, bool BWD>
cudaError_t launch_vec(const NormArgs& a, const RopeTable& t, int per, unsigned grid, size_t smem, cudaStream_t st) {
  return launch_next(a.rope.interleaved ? norm_vec_kernel<T, true, LANES, K, BWD> : norm_vec_kernel<T, false, LANES, K, BWD>,
                     grid, THREADS, smem, st, a, t, per);
}

int bwd_ctas() { return BWD_CTAS_PER_SM * sm_count(); }

template <typename T, bool BWD>
cudaError_t launch(const NormArgs& a, const RopeTable& t, cudaStream_t st) {
  constexpr int N = Vec<T>::N;
  const RopeArgs& p = a.rope;
  const int d = p.d_nope + p.d_rope, n = p.d_rope / 2, widest = p.q ? d : p.d_rope;
  const bool vec = p.d_nope % N == 0 && p.d_rope % N == 0 && (p.interleaved || n % N == 0) && aligned_to_16(p.q) &&
                   aligned_to_16(p.q_out) && aligned_to_16(p.k) && aligned_to_16(p.k_out) && aligned_to_16(a.z_q) &&
                   aligned_to_16(a.z_k) && widest / N <= 128;
  // a few tokens per CTA when a token is little work, but no fewer CTAs than two per SM
  const ll work = static_cast<ll>(p.q ? p.n_h : 0) * d + (p.k ? p.d_rope : 0);
  ll per = std::min<ll>({work > 0 ? 4096 / work : 1, p.tokens / (2 * static_cast<ll>(sm_count())), 16});
  if (per < 1) per = 1;
  const ll groups = (p.tokens + per - 1) / per;
  const unsigned grid = static_cast<unsigned>(BWD ? std::min<ll>(groups, bwd_ctas()) : groups);
  const size_t angles = static_cast<size_t>(per) * n * sizeof(float2);
  const size_t red = BWD ? static_cast<size_t>(WARPS) * widest * sizeof(float) : 0;
  cudaError_t e;
  if (!vec) {
    e = launch_next(norm_any_kernel<T, BWD>, grid, THREADS, angles + red, st, a, t, static_cast<int>(per));
  } else {
    const size_t smem = ((d + p.d_rope + 3) & ~3) * sizeof(float) + angles + red;
    const int chunks = widest / N, k = static_cast<int>(per);
    e = chunks <= 24   ? launch_vec<T, 8, 3, BWD>(a, t, k, grid, smem, st)
        : chunks <= 32 ? launch_vec<T, 32, 1, BWD>(a, t, k, grid, smem, st)
        : chunks <= 64 ? launch_vec<T, 32, 2, BWD>(a, t, k, grid, smem, st)
                       : launch_vec<T, 32, 4, BWD>(a, t, k, grid, smem, st);
  }
  if constexpr (BWD) {
    if (e == cudaSuccess)
      e = launch_next(norm_dw_kernel<T>, dim3((widest + 31) / 32, p.k ? 2 : 1), THREADS, 0, st,
                      static_cast<const float*>(a.partials), static_cast<int>(grid), d, p.d_rope,
                      p.q ? static_cast<T*>(a.dw_q) : nullptr, p.k ? static_cast<T*>(a.dw_k) : nullptr);
  }
  return e;
}

}  // namespace

LaunchResult norm_rope(const NormArgs& a, const RopeTable& t, cudaStream_t st) {
  LaunchResult r;
  r.err = a.rope.is_bf16 ? launch<bf16, false>(a, t, st) : launch<float, false>(a, t, st);
  if (r.err != cudaSuccess) r.what = "norm_rope";
  return r;
}

LaunchResult norm_rope_bwd(const NormArgs& a, const RopeTable& t, cudaStream_t st) {
  LaunchResult r;
  r.err = a.rope.is_bf16 ? launch<bf16, true>(a, t, st) : launch<float, true>(a, t, st);
  if (r.err != cudaSuccess) r.what = "norm_rope_bwd";
  return r;
}

size_t norm_rope_bwd_partials(const RopeArgs& a) {
  return static_cast<size_t>(bwd_ctas()) * (a.d_nope + 2 * a.d_rope);
}

}  // namespace laga
