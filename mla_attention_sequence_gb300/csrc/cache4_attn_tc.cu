// Attention over the paged 4-bit latent cache on the tensor cores, in the latent space, for the
// DeepSeek-V3 widths (latent 512, RoPE key 64). For query row r (a head of a token)
//   s_rj = f_r (q_lat_r . c_j + q_rope_r . k_j),  P = softmax,  ctx_r = sum_j P_rj c_j.
//
// What a code and its scale stand for is exact in fp16 (cache4.h), so the latents' operand is fp16
// without a rounding, and so are the other two: the query, scaled by a power of two of its own row
// that keeps it within fp16's range, and the weights 2^(s - m), with m so far below the row's maximum
// that they use fp16's range (largest 2^14, down to 2^-24: a key is lost where its weight is below
// 2^-30 of the largest). The RoPE key's product is bf16 times bf16 into the same accumulator.
//
// One CTA per (part of the key tiles, half of the context's columns): TMEM cannot hold 128 x 512 fp32
// context columns beside the scores, so both halves of a part compute the scores. Of the query tile
// (nine [128 x 64] boxes, 144 KB) five boxes stay in TMEM as the A operand and four in shared memory,
// which leaves room there for two key tiles of 64 (nine [64 x 64] boxes, 72 KB each): one is being
// expanded while the other is read by the products. With the query all in shared memory only one
// would fit, and reading A from there would bound the products (6 KB for every 32 cycles of an
// N = 64 step, 128 bytes a cycle).
//
// Warp roles (416 threads): warps 0..3 load the queries and do the softmax, one row a thread (their
// TMEM lanes); warp 4 allocates TMEM and issues the MMAs; warps 5..12 expand the key tiles: a lane has
// a block of 16 values of one key (two keys' four blocks make eight lanes' stores hit eight different
// 16-byte columns of the swizzled rows), and loads the next tile's bytes before it works on this one's.
// The boxes that the context's product does not read are refilled as soon as the scores are done.
// TMEM columns: query [0,160), S [160,224), P [224,256), O [256,512).
#include "cache4.h"
#include "score_mod.cuh"

#include <cuda_fp16.h>

namespace laga {
namespace {

using ll = long long;
constexpr int BQ = 128, BKV = 64;
constexpr int NBOX = 9, QBOX = 16384, KBOX = 8192;
constexpr int Q_TMEM = 5;                    // query boxes in TMEM
constexpr int K_BYTES = NBOX * KBOX;
constexpr int Q_BYTES = (NBOX - Q_TMEM) * QBOX;
constexpr int SMEM_BYTES = 2 * K_BYTES + Q_BYTES + 1024 + 512;
constexpr int SOFTMAX_WARPS = 4, PRODUCER_WARPS = 8, MMA_WARP = 4;
constexpr int NTHREADS = 32 * (SOFTMAX_WARPS + 1 + PRODUCER_WARPS);
constexpr uint32_t TMEM_COLS = 512, COL_S = 160, COL_P = 224, COL_O = 256;
constexpr int HALF = 256;
// kind::f16 with fp16 operands is idesc_bf16 without the two type fields
constexpr uint32_t F16 = ~((1u << 7) | (1u << 10));
constexpr uint32_t IDESC_S = idesc_bf16(BQ, BKV, false, false) & F16;
constexpr uint32_t IDESC_ROPE = idesc_bf16(BQ, BKV, false, false);
constexpr uint32_t IDESC_PV = idesc_bf16(BQ, HALF, false, true) & F16;
constexpr float LIFT = 6.f, SLACK = 8.f;  // weights: the maximum's 2^6 when m is set, up to 2^14 before m is moved

struct Params {
  CacheAttn a;
  const bf16* q_lat;  // [B * rows][512]
  const bf16* q;      // [B * rows][192], the RoPE part at 128
  bf16* ctx;          // [B * rows][512]
  float sl2;          // scale * log2(e)
  ModParams mod;      // u_scale, cap_log2
};

// One part's piece of an item: its key tiles, in the order of the walk.
struct Piece {
  int item, b, r0, rows, tiles, key0;
  int2 hull;
  bool begins, ends;
};
struct Walk {
  const CacheAttn& a;
  CacheShare share;
  int t, item;
  __device__ __forceinline__ Walk(const CacheAttn& a_, int part) : a(a_), share(cache_share(a_, part)) {
    t = share.begin;
    item = t < share.end ? cache_item_of(a, t) - 1 : 0;
  }
  __device__ __forceinline__ bool next(Piece& p) {
    if (t >= share.end) return false;
    int begin, end;
    do {
      ++item;
      begin = __ldcg(a.first + item);
      end = __ldcg(a.first + item + 1);
    } while (end <= t);  // items without keys
    p.item = item;
    p.b = item / a.row_tiles;
    p.r0 = (item - p.b * a.row_tiles) * BQ;
    p.rows = min(BQ, a.rows - p.r0);
    p.hull = __ldcg(a.hull + item);
    p.key0 = (p.hull.x / BKV + (t - begin)) * BKV;
    p.begins = t == begin;
    p.ends = end <= share.end;
    p.tiles = min(end, share.end) - t;
    t += p.tiles;
    return true;
  }
};

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Eight codes times a scale (both halves of s), exactly: eight fp16 values in order.
__device__ __forceinline__ uint4 expand8(uint32_t codes, uint32_t s) {
  uint4 v;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
      : "r"(codes));
  v.x = mul_f16x2(v.x, s);
  v.y = mul_f16x2(v.y, s);
  v.z = mul_f16x2(v.z, s);
  v.w = mul_f16x2(v.w, s);
  return v;
}
__device__ __forceinline__ bool bf16x2_finite(uint32_t w) {
  return (w & 0x7f80u) != 0x7f80u && (w & 0x7f800000u) != 0x7f800000u;
}
__device__ __forceinline__ bool finite8(uint4 v) {
  return bf16x2_finite(v.x) && bf16x2_finite(v.y) && bf16x2_finite(v.z) && bf16x2_finite(v.w);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint4 ldg4(const void* p) { return __ldcg(static_cast<const uint4*>(p)); }

// What a producer lane holds of one key tile: its block of 16 values in each of the eight latent boxes,
// eight of the key's 32 scales (its neighbours have the others), two of its eight RoPE chunks.
struct Held {
  uint2 codes[8], scales;
  uint4 rope[2];
  bool bad;
};
__device__ __forceinline__ void hold(const CacheAttn& a, const Piece& p, int tile, int key, int lane4, Held& h) {
  const int at = p.key0 + tile * BKV + key;
  const bool wanted = at >= p.hull.x && at < p.hull.y;
  const ll slot = wanted ? cache_slot(a.cache, a.pages, p.b, at) : -1;
  h.bad = wanted && slot < 0;
  if (slot >= 0) {
    const uint2* c = reinterpret_cast<const uint2*>(a.cache.codes + slot * 256) + lane4;
#pragma unroll
    for (int k = 0; k < 8; ++k) h.codes[k] = __ldg(c + 4 * k);
    h.scales = __ldg(reinterpret_cast<const uint2*>(a.cache.scales + slot * 32) + lane4);
    const uint4* r = reinterpret_cast<const uint4*>(static_cast<const bf16*>(a.cache.keys) + slot * 64) + 2 * lane4;
    h.rope[0] = __ldg(r);
    h.rope[1] = __ldg(r + 1);
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) h.codes[k] = make_uint2(0, 0);
    h.scales = make_uint2(0, 0);
    h.rope[0] = h.rope[1] = make_uint4(0, 0, 0, 0);
  }
}

template <int MOD>
__global__ void __launch_bounds__(NTHREADS, 1) cache4_attn_kernel(const Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint8_t* sK = smem;
  uint8_t* sQ = smem + 2 * K_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sQ + Q_BYTES);
  uint64_t* k_full = bars;        // [2] a key tile is expanded
  uint64_t* ka_free = bars + 2;   // [2] its scores are done: the boxes outside this half's values
  uint64_t* kb_free = bars + 4;   // [2] its context product is done: the others
  uint64_t* s_full = bars + 6;
  uint64_t* s_empty = bars + 7;   // S is in registers
  uint64_t* p_full = bars + 8;
  uint64_t* pv_done = bars + 9;   // P read, O up to date
  uint64_t* q_full = bars + 10;
  uint64_t* drain = bars + 11;
  uint8_t* bad = reinterpret_cast<uint8_t*>(bars + 12);  // [2][8] a bit a key: it does not count as finite
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 14);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const CacheAttn& a = p.a;
  const int part = blockIdx.x >> 1, vh = blockIdx.x & 1;  // vh: this CTA's half of the context's columns

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], PRODUCER_WARPS);
      mbar_init(&ka_free[i], 1);
      mbar_init(&kb_free[i], 1);
    }
    mbar_init(s_full, 1);
    mbar_init(s_empty, SOFTMAX_WARPS);
    mbar_init(p_full, SOFTMAX_WARPS);
    mbar_init(pv_done, 1);
    mbar_init(q_full, SOFTMAX_WARPS);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == MMA_WARP) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  after_previous();

  Walk walk(a, part);
  Piece pc;
  if (warp > MMA_WARP) {
    // ---------------- expand key tiles
    const int pw = warp - MMA_WARP - 1, key = 8 * pw + (lane >> 2), b4 = lane & 3;
    const uint32_t row = static_cast<uint32_t>(key);
    const uint32_t off0 = sw128_offset(row, 2 * b4), off1 = sw128_offset(row, 2 * b4 + 1);
    int n = 0;
    bool ok = true, more = walk.next(pc);
    int j = 0;
    Held cur;
    if (more) hold(a, pc, 0, key, b4, cur);
    while (more && ok) {
      Held nxt;
      if (++j == pc.tiles) {
        j = 0;
        more = walk.next(pc);
      }
      if (more) hold(a, pc, j, key, b4, nxt);
      if (cur.bad && b4 == 0) report_page(a.status, 305);
      const int buf = n & 1;
      const uint32_t ph = static_cast<uint32_t>(((n >> 1) & 1) ^ 1);
      uint8_t* k = sK + buf * K_BYTES;
      bool fine = !cur.bad;
      auto box = [&](int c) {
        const uint32_t word = __shfl_sync(0xffffffffu, (c & 1) ? cur.scales.y : cur.scales.x, (lane & ~3) | (c >> 1));
        const uint32_t e = (word >> (8 * b4)) & 0xffu;
        uint2 w = cur.codes[c];
        uint32_t s = (e << 7) | (e << 23);
        if (e >= 248u) {  // a block that reads as NaN: zeros here, and every row that sees the key gets NaN
          s = 0;
          w = make_uint2(0, 0);
          fine = false;
        }
        *reinterpret_cast<uint4*>(k + c * KBOX + off0) = expand8(w.x, s);
        *reinterpret_cast<uint4*>(k + c * KBOX + off1) = expand8(w.y, s);
      };
      if (!warp_wait_or_abort(&ka_free[buf], ph, abort_flag, 401)) break;
      if (vh) {
#pragma unroll
        for (int c = 0; c < 4; ++c) box(c);
      } else {
#pragma unroll
        for (int c = 4; c < 8; ++c) box(c);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (!finite8(cur.rope[i])) {
          cur.rope[i] = make_uint4(0, 0, 0, 0);
          fine = false;
        }
      *reinterpret_cast<uint4*>(k + 8 * KBOX + off0) = cur.rope[0];
      *reinterpret_cast<uint4*>(k + 8 * KBOX + off1) = cur.rope[1];
      if (!warp_wait_or_abort(&kb_free[buf], ph, abort_flag, 402)) break;
      if (vh) {
#pragma unroll
        for (int c = 4; c < 8; ++c) box(c);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) box(c);
      }
      const uint32_t odd = ~__ballot_sync(0xffffffffu, fine);  // four lanes a key
      if (lane == 0) {
        uint32_t bits = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) bits |= ((odd >> (4 * i)) & 15u) ? 1u << i : 0u;
        bad[buf * 8 + pw] = static_cast<uint8_t>(bits);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&k_full[buf]);
      cur = nxt;
      ++n;
    }
  } else if (warp == MMA_WARP) {
    // ---------------- products
    bool ok = true, issued = false;
    const uint64_t q_desc = sdesc_sw128(smem_u32(sQ), 16, 1024);
    int n = 0, seg = 0;
    auto context = [&](int m, bool first) -> bool {  // O (+)= P(m) V(m)
      if (!warp_wait_or_abort(p_full, m & 1, abort_flag, 411)) return false;
      tc_fence_after();
      const uint64_t v = sdesc_sw128(smem_u32(sK + (m & 1) * K_BYTES + vh * 4 * KBOX), KBOX, 1024);
      const uint32_t pp = tmem + COL_P;
      mma4_ts_warp(tmem + COL_O, pp, pp + 8, pp + 16, pp + 24, v, v + (2048 >> 4), v + (4096 >> 4), v + (6144 >> 4), IDESC_PV,
                   first ? 0u : 1u);
      mma_commit_warp(&kb_free[m & 1]);
      mma_commit_warp(pv_done);
      return true;
    };
    while (ok && walk.next(pc)) {
      ok = warp_wait_or_abort(q_full, seg & 1, abort_flag, 412);
      ++seg;
      for (int j = 0; j < pc.tiles && ok; ++j, ++n) {
        ok = warp_wait_or_abort(&k_full[n & 1], (n >> 1) & 1, abort_flag, 413) &&
             (n == 0 || warp_wait_or_abort(s_empty, (n - 1) & 1, abort_flag, 414));
        if (!ok) break;
        tc_fence_after();
        const uint64_t kd = sdesc_sw128(smem_u32(sK + (n & 1) * K_BYTES), 16, 1024);
        const uint32_t s = tmem + COL_S;
#pragma unroll
        for (int c = 0; c < NBOX; ++c) {
          const uint64_t k = kd + ((c * KBOX) >> 4);
          if (c < Q_TMEM) {
            const uint32_t q = tmem + 32 * c;
            mma4_ts_warp(s, q, q + 8, q + 16, q + 24, k, k + 2, k + 4, k + 6, IDESC_S, c > 0 ? 1u : 0u);
          } else {
            const uint64_t q = q_desc + (((c - Q_TMEM) * QBOX) >> 4);
            mma4_ss_warp(s, q, q + 2, q + 4, q + 6, k, k + 2, k + 4, k + 6, c == 8 ? IDESC_ROPE : IDESC_S, 1u);
          }
        }
        issued = true;
        mma_commit_warp(&ka_free[n & 1]);
        mma_commit_warp(s_full);
        if (j > 0) ok = context(n - 1, j == 1);
      }
      if (ok) ok = context(n - 1, pc.tiles == 1);
    }
    if (!ok && issued) {
      mma_commit_warp(drain);
      if (lane == 0) mbar_drain(drain, 0);
      __syncwarp();
    }
  } else {
    // ---------------- queries and softmax: thread = row of the tile = TMEM lane
    const int r = threadIdx.x;
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    const float nan = __int_as_float(0x7fc00000);
    int n = 0;
    bool ok = true;
    while (ok && walk.next(pc)) {
      const bool there = r < pc.rows;
      const ll row = static_cast<ll>(pc.b) * a.rows + pc.r0 + (there ? r : 0);
      const int qi = (pc.r0 + r) / a.n_h, h = pc.r0 + r - qi * a.n_h;
      const int2 seen = there ? cache_row_bounds(a, pc.b, qi) : make_int2(0, 0);
      const uint4* ql = reinterpret_cast<const uint4*>(p.q_lat + row * 512);
      const uint4* qr = reinterpret_cast<const uint4*>(p.q + row * 192 + 128);
      float top = 0.f;
      bool odd = false;  // the row's result is NaN
      if (there) {
        auto look = [&](uint4 v) {
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) top = max3f(top, fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i])));
          odd = odd || !finite8(v);
        };
#pragma unroll 8
        for (int c = 0; c < 64; ++c) look(ldg4(ql + c));
#pragma unroll
        for (int c = 0; c < 8; ++c) look(ldg4(qr + c));
      }
      // the row's largest size becomes 2^8 to 2^9
      const int e = top > 0.f && !odd ? min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127 - 8, -118), 118) : 0;
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
      const bool load = there && !odd;
      auto f16_8 = [&](uint4 v) {
        return make_uint4(pack_f16x2(bf16_lo(v.x) * down, bf16_hi(v.x) * down), pack_f16x2(bf16_lo(v.y) * down, bf16_hi(v.y) * down),
                          pack_f16x2(bf16_lo(v.z) * down, bf16_hi(v.z) * down), pack_f16x2(bf16_lo(v.w) * down, bf16_hi(v.w) * down));
      };
#pragma unroll 1
      for (int c = 0; c < Q_TMEM; ++c) {
        uint32_t u[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 v = f16_8(load ? ldg4(ql + 8 * c + i) : make_uint4(0, 0, 0, 0));
          u[4 * i] = v.x;
          u[4 * i + 1] = v.y;
          u[4 * i + 2] = v.z;
          u[4 * i + 3] = v.w;
        }
        tmem_st32(tmem + 32 * c + lane_off, u);
      }
#pragma unroll 1
      for (int c = Q_TMEM; c < NBOX; ++c) {
        uint8_t* box = sQ + (c - Q_TMEM) * QBOX;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          uint4 v = load ? (c < 8 ? ldg4(ql + 8 * c + i) : ldg4(qr + i)) : make_uint4(0, 0, 0, 0);
          if (c < 8)
            v = f16_8(v);
          else
            v = make_uint4(pack_bf16x2(bf16_lo(v.x) * down, bf16_hi(v.x) * down), pack_bf16x2(bf16_lo(v.y) * down, bf16_hi(v.y) * down),
                           pack_bf16x2(bf16_lo(v.z) * down, bf16_hi(v.z) * down), pack_bf16x2(bf16_lo(v.w) * down, bf16_hi(v.w) * down));
          *reinterpret_cast<uint4*>(box + sw128_offset(static_cast<uint32_t>(r), static_cast<uint32_t>(i))) = v;
        }
      }
      tmem_wait_st();
      tc_fence_before();
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);

      const float f = MOD & kModCap ? p.mod.u_scale * up : p.sl2 * up;  // score -> log2 units, or -> tanh's argument
      float slope2 = 0.f, pos = 0.f;
      if constexpr ((MOD & kModBias) != 0) {
        if (there) slope2 = __ldg(p.mod.slopes + h) * 1.4426950408889634f;
        pos = static_cast<float>(__ldg(a.lengths + pc.b) - a.Sq + qi - pc.key0);
      }
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < pc.tiles && ok; ++j, ++n) {
        if (!warp_wait_or_abort(s_full, n & 1, abort_flag, 421)) { ok = false; break; }
        tc_fence_after();
        uint32_t x[64];
        tmem_ld32(tmem + COL_S + lane_off, *reinterpret_cast<uint32_t(*)[32]>(x));
        tmem_ld32(tmem + COL_S + 32 + lane_off, *reinterpret_cast<uint32_t(*)[32]>(x + 32));
        uint2 bits;
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(bits.x), "=r"(bits.y) : "r"(smem_u32(bad + (n & 1) * 8)));
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_empty);
        const int k0 = pc.key0 + j * BKV;
#pragma unroll
        for (int i = 0; i < 64; ++i) {
          float s = __uint_as_float(x[i]) * f;
          if constexpr ((MOD & kModCap) != 0) s = tanh_rel(s) * p.mod.cap_log2;
          if constexpr ((MOD & kModBias) != 0) s = fmaf(-slope2, fabsf(pos - static_cast<float>(j * BKV + i)), s);
          x[i] = __float_as_uint(s);
        }
        if (k0 < seen.x || k0 + BKV > seen.y) {
          const uint32_t v0 = visible_bits(seen.x - k0, seen.y - k0), v1 = visible_bits(seen.x - k0 - 32, seen.y - k0 - 32);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            if (!((v0 >> i) & 1u)) x[i] = 0xff800000u;
            if (!((v1 >> i) & 1u)) x[32 + i] = 0xff800000u;
          }
          odd = odd || ((bits.x & v0) | (bits.y & v1)) != 0;
        } else {
          odd = odd || (bits.x | bits.y) != 0;
        }
        float mx = __uint_as_float(x[0]);
#pragma unroll
        for (int i = 1; i < 63; i += 2) mx = max3f(mx, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
        mx = fmaxf(mx, __uint_as_float(x[63])) - LIFT;
        float alpha = 1.f;
        bool rescale = false;
        if (m == -INFINITY) {
          m = mx;
        } else if (mx > m + SLACK) {
          alpha = ex2_approx(m - mx);
          m = mx;
          rescale = true;
        }
        const float neg = m == -INFINITY ? 0.f : -m;
        float sum = 0.f;
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float w0 = ex2_approx(__uint_as_float(x[2 * i]) + neg), w1 = ex2_approx(__uint_as_float(x[2 * i + 1]) + neg);
          sum += w0 + w1;
          pk[i] = pack_f16x2(w0, w1);
        }
        l = fmaf(l, alpha, sum);
        // O and P are the products' until the tile before is done
        if (j > 0 && !warp_wait_or_abort(pv_done, (n - 1) & 1, abort_flag, 422)) { ok = false; break; }
        tc_fence_after();
        if (__any_sync(0xffffffffu, rescale)) {
          const uint32_t o = tmem + COL_O + lane_off;
#pragma unroll 1
          for (int c = 0; c < HALF / 32; ++c) {
            uint32_t u[32];
            tmem_ld32(o + c * 32, u);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(__uint_as_float(u[i]) * alpha);
            tmem_st32(o + c * 32, u);
          }
        }
        tmem_st32(tmem + COL_P + lane_off, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
      }
      if (!ok || !warp_wait_or_abort(pv_done, (n - 1) & 1, abort_flag, 423)) { ok = false; break; }
      tc_fence_after();
      if (odd) l = nan;
      const uint32_t o = tmem + COL_O + lane_off;
      if (pc.begins && pc.ends) {
        if (l == 0.f && seen.x < seen.y) l = nan;  // every score it sees is -inf
        const float inv = l == 0.f ? 0.f : 1.f / l;
        bf16* out = p.ctx + row * 512 + vh * HALF;
#pragma unroll 1
        for (int c = 0; c < HALF / 32; ++c) {
          uint32_t u[32];
          tmem_ld32(o + c * 32, u);
          tmem_wait_ld();
          if (there) {
            uint4* dst = reinterpret_cast<uint4*>(out + c * 32);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              float y[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) y[i] = l != l ? nan : __uint_as_float(u[8 * v + i]) * inv;
              dst[v] = make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7]));
            }
          }
        }
        if (there && vh == 0)
          a.lse[(static_cast<ll>(pc.b) * a.n_h + h) * a.Sq + qi] = l == 0.f ? -INFINITY : fmaf(m, 0.6931471805599453f, logf(l));
      } else {
        const ll slot = static_cast<ll>(2 * part + (pc.begins ? 1 : 0)) * BQ + r;
        if (there && vh == 0) a.part_ml[slot] = make_float2(m, l);
        float* out = a.part_o + slot * 512 + vh * HALF;
#pragma unroll 1
        for (int c = 0; c < HALF / 32; ++c) {
          uint32_t u[32];
          tmem_ld32(o + c * 32, u);
          tmem_wait_ld();
          if (there) {
            uint4* dst = reinterpret_cast<uint4*>(out + c * 32);
#pragma unroll
            for (int v = 0; v < 8; ++v) dst[v] = make_uint4(u[4 * v], u[4 * v + 1], u[4 * v + 2], u[4 * v + 3]);
          }
        }
      }
      tc_fence_before();  // O has been read before the next piece's products overwrite it (q_full, p_full)
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) publish_abort(abort_flag, a.status);
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

}  // namespace

LaunchResult cache4_tc_attn(const CacheAttn& a, const bf16* q, const bf16* q_lat, bf16* ctx, cudaStream_t st) {
  Params p{};
  p.a = a;
  p.q_lat = q_lat;
  p.q = q;
  p.ctx = ctx;
  p.sl2 = a.scale * 1.4426950408889634f;
  Dims d{};
  d.scale = a.scale;
  p.mod = mod_params(d, a.mods);
  LaunchResult r;
  const int mod = mod_of(a.mods);
  auto kern = mod == 0 ? cache4_attn_kernel<0> : mod == kModCap ? cache4_attn_kernel<kModCap>
            : mod == kModBias ? cache4_attn_kernel<kModBias> : cache4_attn_kernel<kModCap | kModBias>;
  r.err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (r.err == cudaSuccess) r.err = launch_next(kern, 2 * a.parts, NTHREADS, SMEM_BYTES, st, p);
  if (r.err != cudaSuccess) r.what = "cache4_attn";
  return r;
}

}  // namespace laga
