// Attention over the paged 4-bit latent cache for few query rows, with the key tiles expanded in
// registers. The mathematics and the operands' types are those of cache4_attn_tc.cu.
//
// Few rows make it a walk over memory: 416 bytes a token against 16 x 1088 multiply-adds, 18 cycles an
// SM at the copy's rate. Through shared memory (tcgen05 takes its key operand from nowhere else) each
// token's 1152 expanded bytes would be written once and read twice there, 27 cycles, beside what a tile
// of 128 mostly empty rows costs. mma.sync takes its operands from registers, at half of tcgen05's rate
// (1950 multiply-adds a cycle and SM, measured), which 16 rows of 8.5 cycles a token can afford.
//
// A CTA of four warps holds 16 rows. Warp w owns latent columns [128 w, 128 w + 128) and RoPE columns
// [16 w, 16 w + 16): it expands each token's codes of these columns once, into the B operand's layout
// of the scores (a lane has one key's block of 16 values, which serves four k steps), sums its part of
// the scores, and turns the same registers (movmatrix) into the B operand of the context's columns it
// owns. The parts of the scores are added up in shared memory, four rows a warp with a key a lane,
// where the softmax's weights come from; they return as the context's A operand.
//
// Tiles of 32 keys come in by cp.async (26 chunks of 16 bytes a token, zeros for tokens outside the
// item's interval), STAGES deep; two barriers a tile. The rows' stride of 416 bytes makes four tokens'
// 32 bytes fall into different banks.
//
// 64 sequences of 1000 .. 8192 tokens, 16 heads (events): 63 us, 116 MB read, 28% of memory's rate. Latency
// bounds it: neither memory (all sequences on one page: 2 us less) nor issue is full (42% of the cycles; 700
// instructions a warp and tile, 256 of which expand the codes and 68 are products), but 255 registers leave
// two warps a scheduler, which wait at two barriers a tile. Measured and dropped: bulk copies issued by the
// warps in turn 72, eight warps of 64 columns 111, tiles of 16 keys with three CTAs an SM 94, the values by way
// of shared memory and ldmatrix instead of movmatrix 65, and with three CTAs an SM 68, the loads' place among
// the pages worked out for every tile anew 68.
#include "cache4.h"
#include "cache4_tc.cuh"
#include "score_mod.cuh"

namespace laga {
namespace {

constexpr int ROWS = kMmaRows, KEYS = kMmaKeys, WARPS = 4, THREADS = 32 * WARPS;
constexpr int STAGES = 6;
constexpr int KEY_BYTES = 256 + 32 + 128;  // codes, scales, RoPE key
constexpr int STAGE_BYTES = KEYS * KEY_BYTES;
constexpr int SP_STRIDE = 40, PS_STRIDE = 40;  // floats, halves: rows of 32 keys
constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + WARPS * ROWS * SP_STRIDE * 4 + ROWS * PS_STRIDE * 2 + STAGES * 4 + WARPS * 4 +
                           ROWS * 4 + 16;

struct Params {
  CacheAttn a;
  CacheOperands x;
  float sl2;
  ModParams mod;
};

__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint2 lds8(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}

template <int MOD>
__global__ void __launch_bounds__(THREADS, 2) cache4_attn_mma_kernel(const Params p) {
  extern __shared__ __align__(16) uint8_t smem[];
  float* sp = reinterpret_cast<float*>(smem + STAGES * STAGE_BYTES);        // [4][16][40] parts of the scores
  __half* ps = reinterpret_cast<__half*>(sp + WARPS * ROWS * SP_STRIDE);    // [16][40] weights
  uint32_t* missing = reinterpret_cast<uint32_t*>(ps + ROWS * PS_STRIDE);   // [STAGES] a bit a key: it has no page
  uint32_t* bad = missing + STAGES;                                         // [4] .. : a warp saw it not finite
  float* scale_by = reinterpret_cast<float*>(bad + WARPS);                  // [16] what the context so far is scaled by
  uint32_t* rescale = reinterpret_cast<uint32_t*>(scale_by + ROWS);         // a bit a warp: some row's is not 1
  const CacheAttn& a = p.a;
  const int part = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const uint32_t stages = smem_u32(smem);
  after_previous();

  Walk<ROWS, KEYS> walk(a, part);
  Piece pc;
  // The loads run STAGES - 1 tiles ahead, across pieces: a walk of their own. Four lanes a key: chunks q,
  // q + 4, .. of its 26. The key's place among the pages is kept from tile to tile, and its entry of the
  // table is fetched a tile before it is used.
  Walk<ROWS, KEYS> ahead(a, part);
  Piece next;
  bool more = ahead.next(next);
  if (!more) return;
  const int my_key = threadIdx.x >> 2, q = threadIdx.x & 3, page = a.cache.page;
  int loaded = 0, left = next.tiles, at = 0, page_row = 0, id = -1;
  uint32_t page_of = 0;
  bool wanted = false, in = false;
  auto fetch = [&]() {  // id is not looked at before it is used: that would wait for it
    wanted = at >= next.hull.x && at < next.hull.y;
    in = page_of < static_cast<uint32_t>(a.pages.most);
    if (wanted && in) id = __ldg(a.pages.table + static_cast<ll>(next.b) * a.pages.most + page_of);
  };
  auto begin_piece = [&]() {
    left = next.tiles;
    at = next.key0 + my_key;
    page_of = static_cast<uint32_t>(at) / static_cast<uint32_t>(page);
    page_row = at - static_cast<int>(page_of) * page;
    fetch();
  };
  begin_piece();
  auto load = [&]() {
    const int s = loaded % STAGES;
    if (more) {
      const bool there = in && id >= 0 && id < a.cache.pages, live = wanted && there;
      const ll slot = live ? static_cast<ll>(id) * page + page_row : 0;
      const uint32_t gone = __ballot_sync(0xffffffffu, wanted && !there);
      if (lane == 0) reinterpret_cast<uint8_t*>(missing + s)[warp] = 0;
      if (gone) {
        if (lane == 0) {
          uint32_t bits = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) bits |= ((gone >> (4 * i)) & 1u) << i;
          reinterpret_cast<uint8_t*>(missing + s)[warp] = static_cast<uint8_t>(bits);
          report_page(a.status, 306);
        }
        __syncwarp();
      }
      const uint32_t to = stages + s * STAGE_BYTES + my_key * KEY_BYTES + 16 * q;
      const uint8_t* codes = a.cache.codes + slot * 256 + 16 * q;
      const uint8_t* keys = static_cast<const uint8_t*>(a.cache.keys) + slot * 128 + 16 * q;
#pragma unroll
      for (int i = 0; i < 4; ++i) copy16(to + 64 * i, codes + 64 * i, live);
#pragma unroll
      for (int i = 0; i < 2; ++i) copy16(to + 288 + 64 * i, keys + 64 * i, live);
      if (q < 2) copy16(to + 256, a.cache.scales + slot * 32 + 16 * q, live);
      if (--left == 0) {
        more = ahead.next(next);
        if (more) begin_piece();
      } else {
        at += KEYS;
        page_row += KEYS;
        while (page_row >= page) {
          page_row -= page;
          ++page_of;
        }
        fetch();
      }
    }
    ++loaded;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < STAGES - 1; ++i) load();
  asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
  __syncthreads();

  int n = 0;
  while (walk.next(pc)) {
    // this warp's part of the queries: the k steps' A operands, in the order of its lanes' codes
    const ll row0 = static_cast<ll>(pc.b) * a.rows + pc.r0;
    uint32_t qa[8][4], qr[4];
    {
      const uint2 zero = make_uint2(0, 0);
      const uint8_t* lo = p.x.query + (row0 + g) * 1152;
      const uint8_t* hi = lo + 8 * 1152;
      const bool in0 = g < pc.rows, in1 = g + 8 < pc.rows;
#pragma unroll
      for (int k = 0; k < 8; ++k) {  // group k / 4 of 64 columns, step k % 4
        const int at = 2 * (128 * warp + 64 * (k >> 2) + 16 * t4 + 4 * (k & 3));
        const uint2 x = in0 ? __ldcg(reinterpret_cast<const uint2*>(lo + at)) : zero;
        const uint2 y = in1 ? __ldcg(reinterpret_cast<const uint2*>(hi + at)) : zero;
        qa[k][0] = x.x;
        qa[k][1] = y.x;
        qa[k][2] = x.y;
        qa[k][3] = y.y;
      }
      const int at = 2 * (512 + 16 * warp + 4 * t4);
      const uint2 x = in0 ? __ldcg(reinterpret_cast<const uint2*>(lo + at)) : zero;
      const uint2 y = in1 ? __ldcg(reinterpret_cast<const uint2*>(hi + at)) : zero;
      qr[0] = x.x;
      qr[1] = y.x;
      qr[2] = x.y;
      qr[3] = y.y;
    }
    // the four rows whose softmax this warp does
    float f[4], m[4], l[4], slope2[4], pos[4];
    int2 seen[4];
    uint32_t odd = 0;  // a bit a row: its result is NaN, if it sees anything
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * warp + i;
      const bool there = r < pc.rows;
      const int qi = (pc.r0 + r) / a.n_h, h = pc.r0 + r - qi * a.n_h;
      seen[i] = there ? cache_row_bounds(a, pc.b, qi) : make_int2(0, 0);
      const float up = there ? __ldcg(p.x.up + row0 + r) : 1.f;
      if (up != up) odd |= 1u << i;
      f[i] = (MOD & kModCap ? p.mod.u_scale : p.sl2) * (up != up ? 1.f : up);
      slope2[i] = pos[i] = 0.f;
      if constexpr ((MOD & kModBias) != 0) {
        if (there) slope2[i] = __ldg(p.mod.slopes + h) * 1.4426950408889634f;
        pos[i] = static_cast<float>(__ldg(a.lengths + pc.b) - a.Sq + qi - pc.key0 - lane);
      }
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
    float o[2][8][4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[i][j][k] = 0.f;

    for (int j = 0; j < pc.tiles; ++j, ++n) {
      const int stage = n % STAGES;
      const uint32_t base = stages + stage * STAGE_BYTES + g * KEY_BYTES;
      // ---- expand, and this warp's part of the scores. (Straight code: the four key groups' chains of
      // products run beside each other.)
      uint32_t kv[4][2][8];
      uint2 rope[4];
      uint32_t strange = 0;  // a bit a key group: this lane's key is not finite
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) {  // 8 keys, one a lane group
        const uint32_t at = base + kt * 8 * KEY_BYTES;
        const uint2 sc = lds8(at + 256 + 8 * warp);
        rope[kt] = lds8(at + 288 + 32 * warp + 8 * t4);
        bool fine = true;
#pragma unroll
        for (int G = 0; G < 2; ++G) {
          const uint2 w = lds8(at + 64 * warp + 32 * G + 8 * t4);
          const uint32_t e = ((G ? sc.y : sc.x) >> (8 * t4)) & 0xffu;
          const bool number = e <= kCacheTopScale;
          fine = fine && number;
          const uint32_t s = number ? e * 0x800080u : 0u;
          const uint4 x = expand8(w.x, s), y = expand8(w.y, s);
          kv[kt][G][0] = x.x;
          kv[kt][G][1] = x.y;
          kv[kt][G][2] = x.z;
          kv[kt][G][3] = x.w;
          kv[kt][G][4] = y.x;
          kv[kt][G][5] = y.y;
          kv[kt][G][6] = y.z;
          kv[kt][G][7] = y.w;
        }
        const bool number = finite4(rope[kt]);
        fine = fine && number;
        rope[kt].x = number ? rope[kt].x : 0u;
        rope[kt].y = number ? rope[kt].y : 0u;
        strange |= fine ? 0u : 1u << kt;
      }
      float s[4][4];
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) {
        s[kt][0] = s[kt][1] = s[kt][2] = s[kt][3] = 0.f;
        mma_bf16(s[kt], qr, rope[kt].x, rope[kt].y);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) mma_f16(s[kt], qa[k], kv[kt][k >> 2][2 * (k & 3)], kv[kt][k >> 2][2 * (k & 3) + 1]);
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) {
        float* to = sp + (warp * ROWS + g) * SP_STRIDE + 8 * kt + 2 * t4;
        *reinterpret_cast<float2*>(to) = make_float2(s[kt][0], s[kt][1]);
        *reinterpret_cast<float2*>(to + 8 * SP_STRIDE) = make_float2(s[kt][2], s[kt][3]);
      }
      uint32_t strange_keys = 0;
      if (__any_sync(0xffffffffu, strange)) {
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
          const uint32_t votes = __ballot_sync(0xffffffffu, (strange >> kt) & 1u);
#pragma unroll
          for (int i = 0; i < 8; ++i) strange_keys |= ((votes >> (4 * i)) & 15u) ? 1u << (8 * kt + i) : 0u;
        }
      }
      if (lane == 0) bad[warp] = strange_keys;
      const uint32_t lost = missing[stage];
      __syncthreads();  // the scores' parts are there; the stage has been read, and the weights before
      load();
      // ---- weights: four rows, a key a lane. m stays while no weight passes 2^(LIFT + SLACK), so that a
      // tile needs no maximum but one vote.
      const int key0 = pc.key0 + j * KEYS, key = key0 + lane;
      const uint32_t not_finite = bad[0] | bad[1] | bad[2] | bad[3] | lost;
      float x[4], by[4];
      bool over = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* from = sp + (4 * warp + i) * SP_STRIDE + lane;
        float v = (from[0] + from[ROWS * SP_STRIDE]) + (from[2 * ROWS * SP_STRIDE] + from[3 * ROWS * SP_STRIDE]);
        v *= f[i];
        if constexpr ((MOD & kModCap) != 0) v = ((MOD & kModFar) != 0 ? tanh_rel(v) : tanh_abs(v)) * p.mod.cap_log2;
        if constexpr ((MOD & kModBias) != 0) v = fmaf(-slope2[i], fabsf(pos[i] - static_cast<float>(j * KEYS)), v);
        x[i] = key >= seen[i].x && key < seen[i].y ? v : -INFINITY;
        over = over || x[i] > m[i] + (LIFT + SLACK);
        by[i] = 1.f;
      }
      if (not_finite) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (__any_sync(0xffffffffu, key >= seen[i].x && key < seen[i].y && ((not_finite >> lane) & 1u))) odd |= 1u << i;
      }
      const bool changed = __any_sync(0xffffffffu, over);
      if (changed) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float top = warp_max(x[i]) - LIFT;
          if (top > m[i] + SLACK) {
            by[i] = m[i] == -INFINITY ? 1.f : ex2_approx(m[i] - top);
            m[i] = top;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * warp + i;
        const float w = ex2_approx(x[i] - (m[i] == -INFINITY ? 0.f : m[i]));
        l[i] = fmaf(l[i], by[i], w);
        ps[r * PS_STRIDE + lane] = __float2half_rn(w);
        if (lane == 0) scale_by[r] = by[i];
      }
      if (lane == 0) reinterpret_cast<uint8_t*>(rescale)[warp] = changed ? 1 : 0;
      asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");  // the next tile
      __syncthreads();
      // ---- context
      if (*rescale) {
        const float x = scale_by[g], y = scale_by[g + 8];
#pragma unroll
        for (int G = 0; G < 2; ++G)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            o[G][k][0] *= x;
            o[G][k][1] *= x;
            o[G][k][2] *= y;
            o[G][k][3] *= y;
          }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {  // 16 keys
        uint32_t pa[4];
        const __half* from = ps + g * PS_STRIDE + 16 * i + 2 * t4;
        pa[0] = *reinterpret_cast<const uint32_t*>(from);
        pa[1] = *reinterpret_cast<const uint32_t*>(from + 8 * PS_STRIDE);
        pa[2] = *reinterpret_cast<const uint32_t*>(from + 8);
        pa[3] = *reinterpret_cast<const uint32_t*>(from + 8 * PS_STRIDE + 8);
#pragma unroll
        for (int G = 0; G < 2; ++G)
#pragma unroll
          for (int k = 0; k < 8; ++k) mma_f16(o[G][k], pa, transposed(kv[2 * i][G][k]), transposed(kv[2 * i + 1][G][k]));
      }
    }

    // ---- the piece's end: sums of the rows to all warps
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * warp + i;
      float sum = l[i];
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
      if (((odd >> i) & 1u) && seen[i].x < seen[i].y) sum = __int_as_float(0x7fc00000);  // a row that sees nothing is 0 whatever it holds
      if (pc.begins && pc.ends && sum == 0.f && seen[i].x < seen[i].y) sum = __int_as_float(0x7fc00000);
      if (lane == 0) {
        scale_by[r] = sum;
        if (r < pc.rows) {
          if (pc.begins && pc.ends) {
            const int qi = (pc.r0 + r) / a.n_h, h = pc.r0 + r - qi * a.n_h;
            a.lse[(static_cast<ll>(pc.b) * a.n_h + h) * a.Sq + qi] =
                sum == 0.f ? -INFINITY : fmaf(m[i], 0.6931471805599453f, logf(sum));
          } else {
            a.part_ml[static_cast<ll>(2 * part + (pc.begins ? 1 : 0)) * ROWS + r] = make_float2(m[i], sum);
          }
        }
      }
    }
    __syncthreads();
    // a lane has 16 columns of each of its two groups, of rows g and g + 8
    const bool whole = pc.begins && pc.ends;
    float* out = whole ? p.x.ctx + row0 * 512 : a.part_o + static_cast<ll>(2 * part + (pc.begins ? 1 : 0)) * ROWS * 512;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = g + 8 * half;
      const float sum = scale_by[r], by = !whole ? 1.f : sum != sum ? sum : sum == 0.f ? 0.f : 1.f / sum;
      if (r < pc.rows)
#pragma unroll
        for (int G = 0; G < 2; ++G) {
          float4* to = reinterpret_cast<float4*>(out + r * 512 + 128 * warp + 64 * G + 16 * t4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            to[k] = make_float4(o[G][2 * k][2 * half] * by, o[G][2 * k][2 * half + 1] * by, o[G][2 * k + 1][2 * half] * by,
                                o[G][2 * k + 1][2 * half + 1] * by);
        }
    }
    __syncthreads();  // the sums have been read before the next piece's factors
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

}  // namespace

LaunchResult cache4_mma_attn(const CacheAttn& a, const CacheOperands& x, cudaStream_t st) {
  Params p{};
  p.a = a;
  p.x = x;
  p.sl2 = a.scale * 1.4426950408889634f;
  Dims d{};
  d.scale = a.scale;
  p.mod = mod_params(d, a.mods);
  LaunchResult r;
  auto kern = cache4_attn_mma_kernel<0>;
  switch (mod_of(a.mods) | (a.mods.cap > kFarCap ? kModFar : 0)) {
    case 0: break;
    case kModCap: kern = cache4_attn_mma_kernel<kModCap>; break;
    case kModBias: kern = cache4_attn_mma_kernel<kModBias>; break;
    case kModCap | kModBias: kern = cache4_attn_mma_kernel<kModCap | kModBias>; break;
    case kModCap | kModFar: kern = cache4_attn_mma_kernel<kModCap | kModFar>; break;
    default: kern = cache4_attn_mma_kernel<kModCap | kModBias | kModFar>; break;
  }
  r.err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (r.err == cudaSuccess) r.err = launch_next(kern, a.parts, THREADS, SMEM_BYTES, st, p);
  if (r.err != cudaSuccess) r.what = "cache4_attn_mma";
  return r;
}

}  // namespace laga
