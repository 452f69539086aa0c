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
// Tiles of 32 keys come in by bulk copies, three for each run of tokens that lie together in the pool,
// STAGES deep, issued by the four warps in turn; two barriers a tile. A key outside the item's
// interval, or without a page, is not copied: its lanes hold zeros. A key whose latent or RoPE key is not
// finite shows in every row's score (0 times it is a NaN), so that no tile pays for a look at its values:
// where a score is not finite the tile's scores are looked at key by key, the bad keys' lanes are zeroed,
// and the rows that see one are marked.
#include "cache4.h"
#include "cache4_tc.cuh"
#include "score_mod.cuh"

namespace laga {
namespace {

constexpr int ROWS = kMmaRows, KEYS = kMmaKeys, WARPS = 4, THREADS = 32 * WARPS;
constexpr int STAGES = 6;
constexpr int CODES = KEYS * 256, SCALES = KEYS * 32, ROPE = KEYS * 128, STAGE_BYTES = CODES + SCALES + ROPE;
constexpr int SP_STRIDE = 40, PS_STRIDE = 40;  // floats, halves: rows of 32 keys
constexpr int SP_BYTES = WARPS * ROWS * SP_STRIDE * 4, PS_BYTES = ROWS * PS_STRIDE * 2;
constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + SP_BYTES + PS_BYTES + 512;

struct Params {
  CacheAttn a;
  const uint8_t* query;  // [B * rows][576], 16-bit
  const float* up;
  bf16* ctx;
  float sl2;
  ModParams mod;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint2 lds8(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}

// The CTA's barrier; true if no warp has given up.
__device__ __forceinline__ bool together(bool ok) { return __syncthreads_and(ok) != 0; }

template <int MOD>
__global__ void __launch_bounds__(THREADS, 2) cache4_attn_mma_kernel(const Params p) {
  extern __shared__ __align__(128) uint8_t smem[];
  float* sp = reinterpret_cast<float*>(smem + STAGES * STAGE_BYTES);            // [4][16][40] parts of the scores
  __half* ps = reinterpret_cast<__half*>(smem + STAGES * STAGE_BYTES + SP_BYTES);  // [16][40] weights
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES + SP_BYTES + PS_BYTES);  // [STAGES]
  uint32_t* live = reinterpret_cast<uint32_t*>(full + STAGES);    // [STAGES] a bit a key: it was copied
  uint32_t* missing = live + STAGES;                              // [STAGES] a bit a key: it has no page
  uint32_t* bad = missing + STAGES;                               // [4] a bit a key: a warp's scores of it are not finite
  float* scale_by = reinterpret_cast<float*>(bad + WARPS);        // [16] what the context so far is scaled by
  uint32_t* flags = reinterpret_cast<uint32_t*>(scale_by + ROWS);  // a byte a warp: 1 some row is rescaled, 2 some key is bad
  volatile int* abort_flag = reinterpret_cast<volatile int*>(flags + 1);
  const CacheAttn& a = p.a;
  const int part = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) mbar_init(&full[i], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  after_previous();

  Walk<ROWS, KEYS> walk(a, part);
  Piece pc;
  // ---- copies: this warp's tiles are warp, warp + 4, .. of the part's, a lane a key. Where a key lies
  // is looked up when the warp's tile before is issued, so that the table's latency is nobody's.
  Walk<ROWS, KEYS> ahead(a, part);
  Piece next;
  bool more = ahead.next(next);
  int next_tile = warp, issued = warp;
  ll slot = 0;
  uint32_t keys = 0, gone = 0;  // a bit a key: to copy; without a page
  auto look = [&]() {
    while (more && next_tile >= next.tiles) {
      next_tile -= next.tiles;
      more = ahead.next(next);
    }
    if (!more) return;
    const int at = next.key0 + next_tile * KEYS + lane;
    const bool wanted = at >= next.hull.x && at < next.hull.y;
    bool there;
    slot = cache_slot_of(a.cache, a.pages, next.b, wanted ? at : next.hull.x, &there);
    keys = wanted && there;
    gone = wanted && !there;
  };
  auto issue = [&]() {
    if (!more) return;
    const int st = issued % STAGES;
    const bool mine = keys != 0;
    const uint32_t all = __ballot_sync(0xffffffffu, mine), lost = __ballot_sync(0xffffffffu, gone != 0);
    const ll before = __shfl_up_sync(0xffffffffu, slot, 1);
    const bool starts = mine && (lane == 0 || !((all >> (lane - 1)) & 1u) || before + 1 != slot);
    const uint32_t runs = __ballot_sync(0xffffffffu, starts);
    if (lane == 0) {
      live[st] = all;
      missing[st] = lost;
      if (lost) report_page(a.status, 306);
      mbar_arrive_expect_tx(&full[st], __popc(all) * 416);
    }
    __syncwarp();
    if (starts) {
      // up to the next run's start or the next key that is not copied
      const uint32_t after = lane == 31 ? 0u : (runs | ~all) >> (lane + 1);
      const int len = after ? __ffs(after) : 32 - lane;
      uint8_t* to = smem + st * STAGE_BYTES;
      bulk_load(to + lane * 256, a.cache.codes + slot * 256, len * 256, &full[st]);
      bulk_load(to + CODES + lane * 32, a.cache.scales + slot * 32, len * 32, &full[st]);
      bulk_load(to + CODES + SCALES + lane * 128, static_cast<const uint8_t*>(a.cache.keys) + slot * 128, len * 128, &full[st]);
    }
    __syncwarp();
    issued += WARPS;
    next_tile += WARPS;
    look();
  };
  look();
#pragma unroll 1
  while (issued < STAGES && more) issue();

  const uint32_t stages = smem_u32(smem);
  int n = 0;
  bool ok = true;
  while (ok && walk.next(pc)) {
    // this warp's part of the queries: the k steps' A operands, in the order of its lanes' codes
    const ll row0 = static_cast<ll>(pc.b) * a.rows + pc.r0;
    uint32_t qa[8][4], qr[4];
    {
      const uint2 zero = make_uint2(0, 0);
      const uint8_t* lo = p.query + (row0 + g) * 1152;
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
    uint32_t odd = 0;  // a bit a row: its result is NaN
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * warp + i;
      const bool there = r < pc.rows;
      const int qi = (pc.r0 + r) / a.n_h, h = pc.r0 + r - qi * a.n_h;
      seen[i] = there ? cache_row_bounds(a, pc.b, qi) : make_int2(0, 0);
      const float up = there ? __ldcg(p.up + row0 + r) : 1.f;
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
      ok = pass(&full[stage], (n / STAGES) & 1, abort_flag, 432);
      const uint32_t base = stages + stage * STAGE_BYTES;
      // ---- expand, and this warp's part of the scores. (Straight code: the four key groups' chains of
      // products run beside each other.)
      uint32_t kv[4][2][8];
      uint2 rope[4];
      const uint32_t copied = live[stage], lost = missing[stage];
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) {  // 8 keys, one a lane group
        const int key = 8 * kt + g;
        const uint2 sc = lds8(base + CODES + key * 32 + 8 * warp);
        rope[kt] = lds8(base + CODES + SCALES + key * 128 + 32 * warp + 8 * t4);
        // odd keys' groups the other way round: half as many keys meet in a bank
        const uint32_t at = base + key * 256 + 64 * warp + 8 * t4, swap = 32 * (g & 1);
        const uint2 w0 = lds8(at + swap), w1 = lds8(at + (swap ^ 32));
#pragma unroll
        for (int G = 0; G < 2; ++G) {
          const uint2 w = (g & 1) == G ? w0 : w1;
          const uint32_t s = (((G ? sc.y : sc.x) >> (8 * t4)) & 0xffu) * 0x800080u;
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
      }
      auto clear = [&](uint32_t keep) {  // zeros for the keys whose bit is not set
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) {
          const bool here = (keep >> (8 * kt + g)) & 1u;
#pragma unroll
          for (int G = 0; G < 2; ++G)
#pragma unroll
            for (int k = 0; k < 8; ++k) kv[kt][G][k] = here ? kv[kt][G][k] : 0u;
          rope[kt].x = here ? rope[kt].x : 0u;
          rope[kt].y = here ? rope[kt].y : 0u;
        }
      };
      if (copied != 0xffffffffu) clear(copied);
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
      ok = together(ok);  // the scores' parts are there; the tile, and the weights before, have been read
      if (!ok) break;
      if (((n + STAGES) & (WARPS - 1)) == warp) issue();
      // ---- weights: four rows, a key a lane. m stays while no weight passes 2^(LIFT + SLACK), so that a
      // tile needs no maximum but one vote.
      const int key0 = pc.key0 + j * KEYS, key = key0 + lane;
      float x[4], by[4];
      bool over = false, strange = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float* from = sp + (4 * warp + i) * SP_STRIDE + lane;
        float v = (from[0] + from[ROWS * SP_STRIDE]) + (from[2 * ROWS * SP_STRIDE] + from[3 * ROWS * SP_STRIDE]);
        strange = strange || !(fabsf(v) <= 3.402823466e38f);
        v *= f[i];
        if constexpr ((MOD & kModCap) != 0) v = tanh_rel(v) * p.mod.cap_log2;
        if constexpr ((MOD & kModBias) != 0) v = fmaf(-slope2[i], fabsf(pos[i] - static_cast<float>(j * KEYS)), v);
        x[i] = key >= seen[i].x && key < seen[i].y ? v : -INFINITY;
        over = over || x[i] > m[i] + (LIFT + SLACK);
        by[i] = 1.f;
      }
      // a key that is not finite: no weight, and NaN for the rows that see it
      const uint32_t not_finite = __ballot_sync(0xffffffffu, strange);
      if (lane == 0) bad[warp] = not_finite;
      if (not_finite | lost) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool hit = key >= seen[i].x && key < seen[i].y && (((not_finite | lost) >> lane) & 1u);
          if (__any_sync(0xffffffffu, hit)) odd |= 1u << i;
        }
        over = over && !((not_finite >> lane) & 1u);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = ((not_finite >> lane) & 1u) ? -INFINITY : x[i];
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
      if (lane == 0) reinterpret_cast<uint8_t*>(flags)[warp] = (changed ? 1 : 0) | (not_finite ? 2 : 0);
      together(true);
      // ---- context
      const uint32_t flag = *flags;
      if (flag & 0x02020202u) clear(~(bad[0] | bad[1] | bad[2] | bad[3]));
      if (flag & 0x01010101u) {
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
    if (!ok) break;
    together(true);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * warp + i;
      float sum = l[i];
#pragma unroll
      for (int k = 16; k > 0; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
      if ((odd >> i) & 1u) sum = __int_as_float(0x7fc00000);
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
    together(true);
    // a lane has 16 columns of each of its two groups, of rows g and g + 8
    if (pc.begins && pc.ends) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = g + 8 * half;
        const float sum = scale_by[r], inv = sum != sum ? sum : sum == 0.f ? 0.f : 1.f / sum;
        if (r < pc.rows)
#pragma unroll
          for (int G = 0; G < 2; ++G) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = pack_bf16x2(o[G][k][2 * half] * inv, o[G][k][2 * half + 1] * inv);
            uint4* to = reinterpret_cast<uint4*>(p.ctx + (row0 + r) * 512 + 128 * warp + 64 * G + 16 * t4);
            to[0] = make_uint4(w[0], w[1], w[2], w[3]);
            to[1] = make_uint4(w[4], w[5], w[6], w[7]);
          }
      }
    } else {
      float* out = a.part_o + static_cast<ll>(2 * part + (pc.begins ? 1 : 0)) * ROWS * 512;
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int r = g + 8 * half;
        if (r < pc.rows)
#pragma unroll
          for (int G = 0; G < 2; ++G) {
            float4* to = reinterpret_cast<float4*>(out + r * 512 + 128 * warp + 64 * G + 16 * t4);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              to[k] = make_float4(o[G][2 * k][2 * half], o[G][2 * k][2 * half + 1], o[G][2 * k + 1][2 * half],
                                  o[G][2 * k + 1][2 * half + 1]);
          }
      }
    }
    together(true);  // the sums have been read before the next piece's factors
  }
  if (!ok) {  // given up: let the copies under way land
    for (int i = issued - WARPS; i >= max(n, 0); i -= WARPS) mbar_drain(&full[i % STAGES], (i / STAGES) & 1);
    __syncthreads();
    if (threadIdx.x == 0) publish_abort(abort_flag, a.status);
  }
}

}  // namespace

LaunchResult cache4_mma_attn(const CacheAttn& a, const uint8_t* query, const float* up, bf16* ctx, cudaStream_t st) {
  Params p{};
  p.a = a;
  p.query = query;
  p.up = up;
  p.ctx = ctx;
  p.sl2 = a.scale * 1.4426950408889634f;
  Dims d{};
  d.scale = a.scale;
  p.mod = mod_params(d, a.mods);
  LaunchResult r;
  const int mod = mod_of(a.mods);
  auto kern = mod == 0 ? cache4_attn_mma_kernel<0> : mod == kModCap ? cache4_attn_mma_kernel<kModCap>
            : mod == kModBias ? cache4_attn_mma_kernel<kModBias> : cache4_attn_mma_kernel<kModCap | kModBias>;
  r.err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (r.err == cudaSuccess) r.err = launch_next(kern, a.parts, THREADS, SMEM_BYTES, st, p);
  if (r.err != cudaSuccess) r.what = "cache4_attn_mma";
  return r;
}

}  // namespace laga
