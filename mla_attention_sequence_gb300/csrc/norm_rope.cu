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
// lane), so that a sum takes three shuffles and a warp has four rows at a time; rows wider than 24
// chunks take a whole warp. As many CTAs as the SMs hold deal the rows out evenly, each warp takes
// consecutive rows, has the next ones loaded while it works on those at hand, and makes a token's angles
// once for all heads that it has of it.
//
// 2048 tokens of 128 heads of 192 in bf16, 201 MB moved forward, 302 MB backward (replayed from a graph):
// 35.5 us forward (halves 36.5), 53 us backward with the sum of the partials. A CTA a token, without loads
// ahead: 43 and 87. Forward through shared memory 37.4, in halves through registers 52 (spills; with two CTAs
// an SM 40); backward through registers 58, with two steps of rows ahead 55. Forward with 4 CTAs an SM 2 us
// more, with warps of 32 rows 8 (angles again for each); backward with 3 CTAs 22 more.
#include "ptx.cuh"
#include "rope_device.cuh"

#include <algorithm>

namespace laga {
namespace {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int BWD_CTAS_PER_SM = 4;  // at most: rows of partials

// x^2 of a value above 2^60 leaves fp32 in a sum of 1024: such rows are scaled down first.
constexpr float kBigSum = 0x1p120f;
constexpr float kDown = 0x1p-70f;

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
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

  // A warp's rows of one step, as they come: chunk c of its row j at place j chunks + c.
  static __device__ __forceinline__ int partner(const RowShape& s, int c) {
    return c - s.nope < s.half ? c + s.half : c - s.half;
  }
  static __device__ __forceinline__ void fetch(uint32_t to, const T* row, const RowShape& s, int l, bool active) {
    const uint4* p = reinterpret_cast<const uint4*>(row);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = l + LANES * k;
      if (active && c < s.chunks) copy16(to + 16 * c, p + c);
    }
  }
  struct Held {
    uint4 own[K];
  };
  static __device__ __forceinline__ void load(const T* row, const RowShape& s, int l, bool active, Held& h) {
    const uint4* p = reinterpret_cast<const uint4*>(row);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = l + LANES * k;
      h.own[k] = active && c < s.chunks ? __ldcs(p + c) : make_uint4(0, 0, 0, 0);
    }
  }
  static __device__ __forceinline__ void load(const uint4* row, const RowShape& s, int l, bool active, Held& h) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = l + LANES * k;
      h.own[k] = active && c < s.chunks ? row[c] : make_uint4(0, 0, 0, 0);
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

  // The weights of chunk c, laid out for the row's lanes: N / 4 quarters, chunks of 16 bytes beside each other.
  static __device__ __forceinline__ int weight_at(int pitch, int c, int quarter) { return quarter * pitch + 4 * c; }
  static __device__ __forceinline__ void weights(const float* w, int pitch, int c, float (&v)[N]) {
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
      const float4 f = *reinterpret_cast<const float4*>(w + weight_at(pitch, c, q));
      v[4 * q] = f.x, v[4 * q + 1] = f.y, v[4 * q + 2] = f.z, v[4 * q + 3] = f.w;
    }
  }

  static __device__ __forceinline__ void forward(const Held& h, const uint4* row, T* dst, const RowShape& s, const float* w, int pitch,
                                                 const float2* cs, float eps, int l, bool active) {
    const float sum = sum_lanes<LANES>(squares(h, 1.f));
    const Scale sc = row_scale<LANES>(sum, s.inv_d, eps, [&](float by) { return squares(h, by); });
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = l + LANES * k;
      if (!active || c >= s.chunks) continue;
      float v[N], o[N], wv[N];
      V::get(h.own[k], v);
      weights(w, pitch, c, wv);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = v[i] * sc.down * sc.r * wv[i];
      if constexpr (!INTERLEAVED) {
        if (c >= s.nope) {
          weights(w, pitch, partner(s, c), wv);
          V::get(row[partner(s, c)], o);
#pragma unroll
          for (int i = 0; i < N; ++i) o[i] = o[i] * sc.down * sc.r * wv[i];
        }
      }
      turn(s, c, cs, 1.f, v, o);
      __stcs(reinterpret_cast<uint4*>(dst) + c, V::put(v));
    }
  }

  static __device__ __forceinline__ void backward(const Held& x, const Held& z, const uint4* z_row, T* dst, const RowShape& s,
                                                  const float* w, int pitch, const float2* cs, float eps, int l,
                                                  bool active, float (&acc)[K][N]) {
    const float sum = sum_lanes<LANES>(squares(x, 1.f));
    const Scale sc = row_scale<LANES>(sum, s.inv_d, eps, [&](float by) { return squares(x, by); });
    float dot = 0.f, dy[K][N];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = l + LANES * k;
      float v[N], o[N], wv[N];
      V::get(z.own[k], dy[k]);
      if (!active || c >= s.chunks) continue;
      if constexpr (!INTERLEAVED)
        if (c >= s.nope) V::get(z_row[partner(s, c)], o);
      turn(s, c, cs, -1.f, dy[k], o);
      V::get(x.own[k], v);
      weights(w, pitch, c, wv);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float xh = v[i] * sc.down * sc.r, p = dy[k][i] * xh;
        acc[k][i] += p;
        dot = fmaf(p, wv[i], dot);
        dy[k][i] *= wv[i];
      }
    }
    const float mean = sum_lanes<LANES>(dot) * s.inv_d;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = l + LANES * k;
      if (!active || c >= s.chunks) continue;
      float v[N];
      V::get(x.own[k], v);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = sc.down * sc.r * (dy[k][i] - v[i] * sc.down * sc.r * mean);
      __stcs(reinterpret_cast<uint4*>(dst) + c, V::put(v));
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

// How the rows are dealt out: the first `ctas_q` CTAs take the queries' rows and the others the keys',
// `share` consecutive rows a warp.
struct NormDeal {
  int ctas_q, ctas_k;
  ll share_q, share_k;
  int held;   // tokens whose cosines and sines a warp holds at a time
  int pitch;  // of the weights' quarters in shared memory, in floats
  int rows;   // with a ring: bytes of a warp's rows of one step, of x (backward: as many of z behind them)
};

// Whether the next rows come to shared memory (two steps a warp) or to registers, of which the backward has
// none left; a layout in halves reads its rows' partners there.
template <bool INTERLEAVED, bool BWD>
constexpr bool kNormRing = BWD || !INTERLEAVED;
// CTAs of a variant that an SM holds: rows in flight against registers (the figures above).
template <int LANES, int K, bool BWD>
constexpr int kNormCtas = LANES * K > 64 ? (BWD ? 1 : 2) : (BWD ? 2 : 3);

// Rows of 16-byte chunks. A warp keeps the cosines and sines of the tokens that it is at, and the next
// rows' loads are under way while it works on its rows.
template <typename T, bool INTERLEAVED, int LANES, int K, bool BWD>
__global__ void __launch_bounds__(THREADS, (kNormCtas<LANES, K, BWD>))
    norm_vec_kernel(const NormArgs a, const RopeTable t, const NormDeal deal) {
  using R = RowOps<T, INTERLEAVED, LANES, K>;
  using Held = typename R::Held;
  constexpr int N = R::N, ROWS = 32 / LANES;  // rows of a warp
  constexpr bool RING = kNormRing<INTERLEAVED, BWD>;
  constexpr int KINDS = BWD ? 2 : 1;
  extern __shared__ __align__(16) float smem[];
  const RopeArgs& p = a.rope;
  const int n = p.d_rope / 2, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LANES;
  const bool keys = static_cast<int>(blockIdx.x) >= deal.ctas_q;
  const int heads = keys ? 1 : p.n_h, nope = keys ? 0 : p.d_nope, width = nope + p.d_rope, pitch = deal.pitch;
  const RowShape s{width / N, nope / N, n / N, 1.f / width};
  float* w = smem;  // [N / 4][pitch]
  // then a warp's two steps of rows, then its angles [held][n]
  uint8_t* ring = reinterpret_cast<uint8_t*>(smem + N / 4 * pitch) + warp * (2 * KINDS * deal.rows);
  float2* cs = reinterpret_cast<float2*>(reinterpret_cast<uint8_t*>(smem + N / 4 * pitch) + WARPS * (2 * KINDS * deal.rows)) +
               warp * deal.held * n;
  const T* in = static_cast<const T*>(keys ? p.k : p.q);
  const T* grad = static_cast<const T*>(keys ? a.z_k : a.z_q);
  T* out = static_cast<T*>(keys ? p.k_out : p.q_out);
  const ll share = keys ? deal.share_k : deal.share_q;
  const ll begin = (static_cast<ll>(blockIdx.x - (keys ? deal.ctas_q : 0)) * WARPS + warp) * share;
  const int rows = static_cast<int>(max(min(share, p.tokens * heads - begin), 0ll));  // of this warp
  const ll first_token = begin / heads;
  const int first_head = static_cast<int>(begin - first_token * heads);
  const int tokens = rows ? (first_head + rows - 1) / heads + 1 : 0;
  after_previous();

  int row = lane / LANES, head = first_head + row, token = head / heads;  // this lane's, from the warp's first
  head -= token * heads;
  const ll at0 = begin * width;
  const uint32_t ring_at = smem_u32(ring) + (lane / LANES) * width * sizeof(T);
  Held nx;  // without a ring: the next rows
  // asks for the rows of the step at r0, of an even or odd one
  auto ask = [&](int r0, int which) {
    const int r = r0 + lane / LANES;
    const bool there = r < rows;
    const ll at = at0 + static_cast<ll>(there ? r : 0) * width;
    if constexpr (RING) {
      R::fetch(ring_at + which * (KINDS * deal.rows), in + at, s, l, there);
      if constexpr (BWD) R::fetch(ring_at + which * (KINDS * deal.rows) + deal.rows, grad + at, s, l, there);
      asm volatile("cp.async.commit_group;" ::: "memory");
    } else {
      R::load(in + at, s, l, there, nx);
    }
  };
  ask(0, 0);
  const T* weight = static_cast<const T*>(keys ? a.w_k : a.w_q);
  for (int i = threadIdx.x; i < width; i += THREADS)
    w[R::weight_at(pitch, i / N, i % N / 4) + i % 4] = to_f(weight[i]);
  __syncthreads();

  float acc[K][N];
  if constexpr (BWD)
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < N; ++i) acc[k][i] = 0.f;
  int held0 = 0, held1 = 0;  // the tokens whose angles are there
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += ROWS) {
    const bool active = row < rows;
    const int which = (r0 / ROWS) & 1;
    const uint8_t* from = ring + which * (KINDS * deal.rows) + (lane / LANES) * width * sizeof(T);
    const uint4 *x_row = reinterpret_cast<const uint4*>(from), *z_row = reinterpret_cast<const uint4*>(from + deal.rows);
    Held x, z;
    if constexpr (RING) {
      __syncwarp();  // all lanes have read the rows of the step before, whose place is taken now
      ask(r0 + ROWS, which ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncwarp();
      R::load(x_row, s, l, active, x);
      if constexpr (BWD) R::load(z_row, s, l, active, z);
    } else {
      x = nx;
      ask(r0 + ROWS, 0);
    }
    const int last = min(__shfl_sync(0xffffffffu, token, 31), tokens - 1);
    if (last >= held1) {
      held0 = __shfl_sync(0xffffffffu, token, 0);
      held1 = min(held0 + deal.held, tokens);
      __syncwarp();
      const ll from = first_token + held0;
#pragma unroll 4
      for (int e = lane; e < (held1 - held0) * n; e += 32) {
        const int k = e / n, i = e - k * n;
        const ll at = t.axis[i] * p.tokens + from + k;
        const ll pos = p.pos64 ? static_cast<const ll*>(p.pos)[at] : static_cast<ll>(static_cast<const int*>(p.pos)[at]);
        cs[e] = cos_sin(pos, t.turns[i]);
      }
      __syncwarp();
    }
    const float2* angles = cs + (active ? token - held0 : 0) * n;
    T* to = out + at0 + static_cast<ll>(active ? row : 0) * width;
    if constexpr (BWD)
      R::backward(x, z, z_row, to, s, w, pitch, angles, a.eps, l, active, acc);
    else
      R::forward(x, x_row, to, s, w, pitch, angles, a.eps, l, active);
    row += ROWS;
    head += ROWS;
    if (head >= heads) {
      const int k = head / heads;
      token += k;
      head -= k * heads;
    }
  }
  if constexpr (BWD) {
    // rows of partials: the CTAs' of the queries, then those of the keys
    const int d = p.d_nope + p.d_rope;
    float* to = a.partials + (keys ? static_cast<ll>(deal.ctas_q) * d + static_cast<ll>(blockIdx.x - deal.ctas_q) * width
                                   : static_cast<ll>(blockIdx.x) * width);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the rows' and the angles' places are taken again
    reduce_columns<T, LANES, K>(acc, s, smem + N / 4 * pitch, to);
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

// dw of the queries' (blockIdx.y 0) or the keys' weight: the CTAs' partials, 32 columns a CTA, every
// 32nd row a warp.
constexpr int DW_WARPS = 32;
template <typename T>
__global__ void __launch_bounds__(32 * DW_WARPS) norm_dw_kernel(const float* partials, int ctas_q, int ctas_k, int d,
                                                                int d_rope, T* dw_q, T* dw_k) {
  __shared__ float red[DW_WARPS][33];
  after_previous();
  T* out = blockIdx.y ? dw_k : dw_q;
  const int width = blockIdx.y ? d_rope : d, ctas = blockIdx.y ? ctas_k : ctas_q;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  if (!out || static_cast<int>(blockIdx.x * 32) >= width) return;
  const float* p = partials + (blockIdx.y ? static_cast<ll>(ctas_q) * d : 0) + col;
  float sum = 0.f;
  if (col < width) {
#pragma unroll 8
    for (int k = warp; k < ctas; k += DW_WARPS) sum += __ldcg(p + static_cast<ll>(k) * width);
  }
  red[warp][lane] = sum;
  __syncthreads();
  // a warp joins the 32 sums of one column
  const float v = sum_lanes<32>(red[lane][warp]);
  const int mine = blockIdx.x * 32 + warp;
  if (lane == 0 && mine < width) out[mine] = static_cast<T>(v);
}

int bwd_ctas() { return BWD_CTAS_PER_SM * sm_count(); }

template <typename T, int LANES, int K, bool BWD>
cudaError_t launch_vec(const NormArgs& a, const RopeTable& t, NormDeal& deal, cudaStream_t st) {
  constexpr int N = Vec<T>::N, ROWS = 32 / LANES, CTAS = kNormCtas<LANES, K, BWD>;
  const RopeArgs& p = a.rope;
  const int d = p.d_nope + p.d_rope, n = p.d_rope / 2, widest = p.q ? d : p.d_rope;
  // Whole steps of ROWS rows a warp, as many for all; the keys' warps take a share of the same length in bytes.
  const ll q_rows = p.q ? p.tokens * p.n_h : 0, k_rows = p.k ? p.tokens : 0, warps = static_cast<ll>(CTAS) * sm_count() * WARPS;
  const auto up = [](ll x, ll y) { return (x + y - 1) / y; };
  // a token's angles cost about as much as the bytes of 16 RoPE rows
  const double angle_cost = 16. * p.d_rope * p.tokens;
  const double q_cost = q_rows ? static_cast<double>(q_rows) * d + angle_cost : 0.;
  const double k_cost = k_rows ? static_cast<double>(k_rows) * p.d_rope + angle_cost : 0.;
  const auto deal_out = [&](ll rows, double cost, ll& share) {
    const ll of_these = std::max<ll>(WARPS, static_cast<ll>(warps * (cost / (q_cost + k_cost))) / WARPS * WARPS);
    share = std::max<ll>(up(up(rows, of_these), ROWS), 1) * ROWS;
    return static_cast<int>(up(rows, share * WARPS));
  };
  deal.ctas_q = q_rows ? deal_out(q_rows, q_cost, deal.share_q) : 0;
  deal.ctas_k = k_rows ? deal_out(k_rows, k_cost, deal.share_k) : 0;
  // tokens that a step can touch; more where a token is few rows, as far as 4 KB a warp go
  const int step = ROWS == 1 ? 1 : (ROWS - 2) / (k_rows ? 1 : p.n_h) + 2;
  deal.held = std::max(step, std::min(32 / (k_rows ? 1 : std::min(p.n_h, 32)), 4096 / static_cast<int>(n * sizeof(float2))));
  deal.pitch = 4 * (widest / N);
  deal.rows = BWD || !p.interleaved ? static_cast<int>(ROWS * widest * sizeof(T)) : 0;
  const size_t angles = static_cast<size_t>(WARPS) * deal.held * n * sizeof(float2);
  const size_t ring = static_cast<size_t>(WARPS) * 2 * (BWD ? 2 : 1) * deal.rows;
  const size_t red = BWD ? static_cast<size_t>(WARPS) * widest * sizeof(float) : 0;
  const size_t smem = static_cast<size_t>(N / 4) * deal.pitch * sizeof(float) + std::max(ring + angles, red);
  const auto kern = p.interleaved ? norm_vec_kernel<T, true, LANES, K, BWD> : norm_vec_kernel<T, false, LANES, K, BWD>;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
  }
  return launch_next(kern, static_cast<unsigned>(deal.ctas_q + deal.ctas_k), THREADS, smem, st, a, t,
                     static_cast<const NormDeal&>(deal));
}

template <typename T, bool BWD>
cudaError_t launch(const NormArgs& a, const RopeTable& t, cudaStream_t st) {
  constexpr int N = Vec<T>::N;
  const RopeArgs& p = a.rope;
  const int d = p.d_nope + p.d_rope, n = p.d_rope / 2, widest = p.q ? d : p.d_rope;
  const bool vec = p.d_nope % N == 0 && p.d_rope % N == 0 && (p.interleaved || n % N == 0) && aligned_to_16(p.q) &&
                   aligned_to_16(p.q_out) && aligned_to_16(p.k) && aligned_to_16(p.k_out) && aligned_to_16(a.z_q) &&
                   aligned_to_16(a.z_k) && widest / N <= 128;
  NormDeal deal{};
  cudaError_t e;
  if (!vec) {
    // a few tokens per CTA when a token is little work, but no fewer CTAs than two per SM
    const ll work = static_cast<ll>(p.q ? p.n_h : 0) * d + (p.k ? p.d_rope : 0);
    ll per = std::min<ll>({work > 0 ? 4096 / work : 1, p.tokens / (2 * static_cast<ll>(sm_count())), 16});
    if (per < 1) per = 1;
    const ll groups = (p.tokens + per - 1) / per;
    const unsigned grid = static_cast<unsigned>(BWD ? std::min<ll>(groups, bwd_ctas()) : groups);
    const size_t angles = static_cast<size_t>(per) * n * sizeof(float2);
    const size_t red = BWD ? static_cast<size_t>(WARPS) * widest * sizeof(float) : 0;
    deal.ctas_q = deal.ctas_k = static_cast<int>(grid);
    e = launch_next(norm_any_kernel<T, BWD>, grid, THREADS, angles + red, st, a, t, static_cast<int>(per));
  } else {
    const int chunks = widest / N;
    e = chunks <= 24   ? launch_vec<T, 8, 3, BWD>(a, t, deal, st)
        : chunks <= 32 ? launch_vec<T, 32, 1, BWD>(a, t, deal, st)
        : chunks <= 64 ? launch_vec<T, 32, 2, BWD>(a, t, deal, st)
                       : launch_vec<T, 32, 4, BWD>(a, t, deal, st);
  }
  if constexpr (BWD) {
    if (e == cudaSuccess)
      e = launch_next(norm_dw_kernel<T>, dim3((widest + 31) / 32, p.k ? 2 : 1), 32 * DW_WARPS, 0, st,
                      static_cast<const float*>(a.partials), deal.ctas_q, deal.ctas_k, d, p.d_rope,
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
