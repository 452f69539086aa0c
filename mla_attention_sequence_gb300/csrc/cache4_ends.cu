// The two ends of the attention over the 4-bit cache on the tensor cores (bf16, d_c = 512, d_nope = d_v =
// 128, d_rope = 64), one launch each: before it the queries in the latent space, q_lat = q_nope W_UK^T, as
// operands, and the plan; after it the joining of split items' pieces and out = ctx W_UV.
//
// Per head a product of a few tokens with 128 KB of weights, so what counts is that the weights are read
// once, all of a CTA's loads at once, and how many launches wait for each other: as a plan, a product, a
// scaling, a join and a product they took 53 us around an attention of 12 (three tokens of 16 heads, event
// times), as two launches 21. A CTA takes a head and 16 tokens at a time (the rows of an mma.sync tile). 24
// tokens of 128 heads (events): 13 and 20 us, 17 MB of weights each (2.5 at memory's rate) and 20 MB of pieces;
// a CTA for each 16 tokens of a head, which reads the weights twice, 15 and 23. The sums of q_lat stay fp32
// until they are scaled to fp16; the context is split in two bf16 parts (its first 16 bits of fraction),
// both multiplied: neither costs the result a rounding that shows.
#include "cache4.h"
#include "cache4_tc.cuh"

#include <algorithm>

namespace laga {
namespace {

constexpr int TOKENS = 16, WARPS = 16, THREADS = 32 * WARPS;

// Where a token's row of head h lies among the items.
struct Row {
  int b, i, item, r;  // sequence, its query, item, row of the item
};
__device__ __forceinline__ Row row_of(const CacheAttn& a, int token, int h) {
  Row x;
  x.b = token / a.Sq;
  x.i = token - x.b * a.Sq;
  const int at = x.i * a.n_h + h, tile = at / a.tile;
  x.item = x.b * a.row_tiles + tile;
  x.r = at - tile * a.tile;
  return x;
}

// CTA h + n_h * k: head h's tiles k, k + tiles a head at once, ..; the last CTA makes the plan.
__global__ void __launch_bounds__(THREADS, 1) prepare_kernel(const CacheAttn a, int tokens, const bf16* q, const bf16* W,
                                                             const CacheOperands out) {
  __shared__ float tops[WARPS][TOKENS];
  __shared__ float downs[TOKENS];
  after_previous();
  if (blockIdx.x == gridDim.x - 1) {
    cache4_plan_items<THREADS>(a);
    return;
  }
  const int h = blockIdx.x % a.n_h, step = (gridDim.x - 1) / a.n_h * TOKENS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  // Warp w: latent columns [32 w, 32 w + 32). A lane's 16 bytes are 8 of a group of 32 k, the same ones
  // of the query's rows and of the weights', which serve two k steps.
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 wb[4][4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      wb[j][i] = __ldg(reinterpret_cast<const uint4*>(W + static_cast<ll>(32 * warp + 8 * j + g) * a.n_h * 128 + h * 128 + 32 * i + 8 * t4));
#pragma unroll 1
  for (int t0 = blockIdx.x / a.n_h * TOKENS; t0 < tokens; t0 += step) {
    uint4 qa[4], qb[4];
    const bool in0 = t0 + g < tokens, in1 = t0 + g + 8 < tokens;
    const bf16* q0 = q + (static_cast<ll>(t0 + g) * a.n_h + h) * 192;
    const bf16* q1 = q0 + static_cast<ll>(8) * a.n_h * 192;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      qa[i] = in0 ? ldg4(q0 + 32 * i + 8 * t4) : zero;
      qb[i] = in1 ? ldg4(q1 + 32 * i + 8 * t4) : zero;
    }
    // the RoPE part of token `warp`
    const bool mine = t0 + warp < tokens;
    const ll row = static_cast<ll>(t0 + warp) * a.n_h + h;
    const uint32_t rope = mine ? __ldcg(reinterpret_cast<const uint32_t*>(q + row * 192 + 128) + lane) : 0u;
    float s[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x0[4] = {qa[i].x, qb[i].x, qa[i].y, qb[i].y}, x1[4] = {qa[i].z, qb[i].z, qa[i].w, qb[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) mma_bf16(s[j], x0, wb[j][i].x, wb[j][i].y);
#pragma unroll
      for (int j = 0; j < 4; ++j) mma_bf16(s[j], x1, wb[j][i].z, wb[j][i].w);
    }
    // the rows' largest sizes; infinity where a value is not finite
    const float inf = __int_as_float(0x7f800000);
    auto size = [&](float v) { return fabsf(v) <= 3.402823466e38f ? fabsf(v) : inf; };
    float top0 = 0.f, top1 = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      top0 = max3f(top0, size(s[j][0]), size(s[j][1]));
      top1 = max3f(top1, size(s[j][2]), size(s[j][3]));
    }
#pragma unroll
    for (int k = 1; k < 4; k <<= 1) {
      top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, k));
      top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, k));
    }
    if (t4 == 0) {
      tops[warp][g] = top0;
      tops[warp][g + 8] = top1;
    }
    __syncthreads();
    float top = fmaxf(size(bf16_lo(rope)), size(bf16_hi(rope)));
    if (lane < WARPS) top = fmaxf(top, tops[lane][warp]);
    top = warp_max(top);
    const bool fine = top < inf;
    const int e = fine && top > 0.f ? row_exponent(top) : 0;
    const float down = fine ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : 0.f;
    if (mine) {
      reinterpret_cast<uint32_t*>(out.query + row * kQueryBytes + 1024)[lane] =
          fine ? pack_bf16x2(bf16_lo(rope) * down, bf16_hi(rope) * down) : 0u;
      if (lane == 0) out.up[row] = fine ? __uint_as_float(static_cast<uint32_t>(127 + e) << 23) : __int_as_float(0x7fc00000);
    }
    if (lane == 0) downs[warp] = down;
    __syncthreads();
    const float d0 = downs[g], d1 = downs[g + 8];
    uint8_t* to = out.query + (static_cast<ll>(t0 + g) * a.n_h + h) * kQueryBytes + 2 * (32 * warp + 2 * t4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (in0) *reinterpret_cast<uint32_t*>(to + 16 * j) = d0 != 0.f ? pack_f16x2(s[j][0] * d0, s[j][1] * d0) : 0u;
      if (in1)
        *reinterpret_cast<uint32_t*>(to + static_cast<ll>(8) * a.n_h * kQueryBytes + 16 * j) =
            d1 != 0.f ? pack_f16x2(s[j][2] * d1, s[j][3] * d1) : 0u;
    }
  }
}

// CTA h + n_h * k, as above: token `warp`'s context from its pieces, then 16 rows times the head's weights: warp w
// the output's columns [16 (w % 8), ..) over half w / 8 of the latent columns.
constexpr int A_STRIDE = 520;  // bf16 values: rows fall into different banks
constexpr int FINISH_SMEM = 2 * TOKENS * A_STRIDE * 2;
static_assert(FINISH_SMEM >= WARPS * 512 * 4, "the warps' sums fit");
__global__ void __launch_bounds__(THREADS, 1) finish_kernel(const CacheAttn a, int tokens, const CacheOperands x, const bf16* W,
                                                            bf16* out) {
  __shared__ __align__(16) uint8_t smem[FINISH_SMEM];
  bf16* hi = reinterpret_cast<bf16*>(smem);  // [16][520] the context's first part, then its second
  bf16* lo = hi + TOKENS * A_STRIDE;
  const int h = blockIdx.x % a.n_h, step = gridDim.x / a.n_h * TOKENS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  // The weights first: nothing before this call's first kernel writes them, and that has ended. A lane's
  // 8 bytes are 4 neighbouring columns of one latent row; movmatrix turns an 8 x 8 block of them.
  const int v0 = 16 * (warp & 7), c0 = 256 * (warp >> 3);
  uint2 w[16][2];
#pragma unroll
  for (int k = 0; k < 16; ++k)
#pragma unroll
    for (int i = 0; i < 2; ++i)
      w[k][i] = __ldg(reinterpret_cast<const uint2*>(W + static_cast<ll>(c0 + 16 * k + 8 * i + g) * a.n_h * 128 + h * 128 + v0 + 4 * t4));
  after_previous();
#pragma unroll 1
  for (int t0 = blockIdx.x / a.n_h * TOKENS; t0 < tokens; t0 += step) {
    // ---- the context of this warp's token: 4 columns at 4 lane + 128 j. Where the tokens are few, several
    // warps share a token's pieces (warp `sub` of `shared` takes every `shared`th).
    const int here = min(TOKENS, tokens - t0), shared = here > 8 ? 1 : here > 4 ? 2 : here > 2 ? 4 : here > 1 ? 8 : 16;
    const int token = t0 + warp / shared, sub = warp % shared;
    float4 c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (token < tokens) {
      const Row y = row_of(a, token, h);
      const int begin = __ldcg(a.first + y.item), end = __ldcg(a.first + y.item + 1);
      const CacheShare share = cache_share(a, 0);
      const int p0 = begin / share.quota, p1 = end > begin ? (end - 1) / share.quota : p0;
      float* lse = a.lse + (static_cast<ll>(y.b) * a.n_h + h) * a.Sq + y.i;
      if (end == begin) {
        const float v = lost_row(cache_row_bounds(a, y.b, y.i));
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = make_float4(v, v, v, v);
        if (lane == 0) *lse = v != v ? v : -INFINITY;
        if (sub > 0) c[0] = c[1] = c[2] = c[3] = make_float4(0.f, 0.f, 0.f, 0.f);
      } else if (p0 == p1) {  // one part had it all
        if (sub == 0) {
          const float4* from = reinterpret_cast<const float4*>(x.ctx + (static_cast<ll>(token) * a.n_h + h) * 512) + lane;
#pragma unroll
          for (int j = 0; j < 4; ++j) c[j] = __ldcg(from + 32 * j);
        }
      } else {
        // piece k is part p0 + k's; the first began the item
        const int pieces = p1 - p0 + 1;
        auto slot = [&](int k) { return static_cast<ll>(2 * (p0 + k) + (k == 0 ? 1 : 0)) * a.tile + y.r; };
        float m = -INFINITY, l = 0.f;
        auto add = [&](float2 v) {
          const float to = fmaxf(m, v.x), from = to == -INFINITY ? 0.f : to;
          l = l * exp2f(m - from) + v.y * exp2f(v.x - from);  // 2^-inf = 0; a NaN sum stays one
          m = to;
        };
        for (int k = lane; k < pieces; k += 32) add(__ldcg(a.part_ml + slot(k)));
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) add(make_float2(__shfl_xor_sync(0xffffffffu, m, k), __shfl_xor_sync(0xffffffffu, l, k)));
        l = row_sum(l, cache_row_bounds(a, y.b, y.i));
        const float from = m == -INFINITY ? 0.f : m, inv = l != l ? l : l == 0.f ? 0.f : 1.f / l;
        if (lane == 0) *lse = l == 0.f ? -INFINITY : fmaf(m, 0.6931471805599453f, logf(l));
        for (int k0 = sub; k0 < pieces; k0 += 32 * shared) {
          const int at = k0 + lane * shared;
          const float mine = at < pieces ? exp2f(__ldcg(a.part_ml + slot(at)).x - from) * inv : 0.f;
          const int n = min(32, (pieces - k0 + shared - 1) / shared);
#pragma unroll 4
          for (int k = 0; k < n; ++k) {
            const float by = __shfl_sync(0xffffffffu, mine, k);
            const float4* o = reinterpret_cast<const float4*>(a.part_o + slot(k0 + k * shared) * 512) + lane;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float4 v = __ldcg(o + 32 * j);
              c[j].x = fmaf(by, v.x, c[j].x);
              c[j].y = fmaf(by, v.y, c[j].y);
              c[j].z = fmaf(by, v.z, c[j].z);
              c[j].w = fmaf(by, v.w, c[j].w);
            }
          }
        }
      }
    }
    if (shared > 1) {  // the warps' sums, in their order
      float4* sums = reinterpret_cast<float4*>(smem);
#pragma unroll
      for (int j = 0; j < 4; ++j) sums[warp * 128 + 32 * j + lane] = c[j];
      __syncthreads();
      if (sub == 0)
        for (int k = 1; k < shared; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 v = sums[(warp + k) * 128 + 32 * j + lane];
            c[j].x += v.x;
            c[j].y += v.y;
            c[j].z += v.z;
            c[j].w += v.w;
          }
      __syncthreads();
    }
    if (sub == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint2 first = make_uint2(pack_bf16x2(c[j].x, c[j].y), pack_bf16x2(c[j].z, c[j].w));
        const uint2 second = make_uint2(pack_bf16x2(c[j].x - bf16_lo(first.x), c[j].y - bf16_hi(first.x)),
                                        pack_bf16x2(c[j].z - bf16_lo(first.y), c[j].w - bf16_hi(first.y)));
        *reinterpret_cast<uint2*>(hi + (warp / shared) * A_STRIDE + 128 * j + 4 * lane) = first;
        *reinterpret_cast<uint2*>(lo + (warp / shared) * A_STRIDE + 128 * j + 4 * lane) = second;
      }
    }
    __syncthreads();
    // ---- times the weights
    float s[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const uint32_t b0 = transposed(w[k][0].x), b1 = transposed(w[k][1].x), d0 = transposed(w[k][0].y), d1 = transposed(w[k][1].y);
#pragma unroll
      for (int part = 0; part < 2; ++part) {
        const bf16* from = (part ? lo : hi) + g * A_STRIDE + c0 + 16 * k + 2 * t4;
        const uint32_t aa[4] = {*reinterpret_cast<const uint32_t*>(from), *reinterpret_cast<const uint32_t*>(from + 8 * A_STRIDE),
                                *reinterpret_cast<const uint32_t*>(from + 8), *reinterpret_cast<const uint32_t*>(from + 8 * A_STRIDE + 8)};
        mma_bf16(s[0], aa, b0, b1);
        mma_bf16(s[1], aa, d0, d1);
      }
    }
    __syncthreads();
    float4* other = reinterpret_cast<float4*>(smem);  // the second half's sums
    if (warp >= 8) {
      other[(2 * (warp - 8)) * 32 + lane] = make_float4(s[0][0], s[0][1], s[1][0], s[1][1]);
      other[(2 * (warp - 8) + 1) * 32 + lane] = make_float4(s[0][2], s[0][3], s[1][2], s[1][3]);
    }
    __syncthreads();
    if (warp < 8) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int t = t0 + g + 8 * half;
        if (t >= tokens) continue;
        const float4 v = other[(2 * warp + half) * 32 + lane];
        *reinterpret_cast<uint2*>(out + (static_cast<ll>(t) * a.n_h + h) * 128 + v0 + 4 * t4) =
            make_uint2(pack_bf16x2(s[0][2 * half] + v.x, s[0][2 * half + 1] + v.y), pack_bf16x2(s[1][2 * half] + v.z, s[1][2 * half + 1] + v.w));
      }
    }
    __syncthreads();  // the sums have been read
  }
}

// As many CTAs a head as its tiles, as far as all fit on the SMs: more would read the weights again.
unsigned ctas(const CacheAttn& a) {
  const int tiles = (a.pages.B * a.Sq + TOKENS - 1) / TOKENS;
  return static_cast<unsigned>(std::min(tiles, std::max(1, (sm_count() - 1) / a.n_h)) * a.n_h);
}

}  // namespace

LaunchResult cache4_tc_prepare(const CacheAttn& a, const bf16* q, const bf16* W_UK, const CacheOperands& x, cudaStream_t st) {
  LaunchResult r;
  r.err = launch_next(prepare_kernel, ctas(a) + 1, THREADS, 0, st, a, a.pages.B * a.Sq, q, W_UK, x);
  if (r.err != cudaSuccess) r.what = "cache4_prepare";
  return r;
}

LaunchResult cache4_tc_finish(const CacheAttn& a, const CacheOperands& x, const bf16* W_UV, bf16* out, cudaStream_t st) {
  LaunchResult r;
  r.err = launch_next(finish_kernel, ctas(a), THREADS, 0, st, a, a.pages.B * a.Sq, x, W_UV, out);
  if (r.err != cudaSuccess) r.what = "cache4_finish";
  return r;
}

}  // namespace laga
