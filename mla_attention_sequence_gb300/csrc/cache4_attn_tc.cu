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
// context columns beside the scores, so both halves of a part compute the scores. Of the query tile (nine
// [128 x 64] boxes, 144 KB) the four of this half's values stay in TMEM as the A operand and five in shared
// memory: with all of it there too few key tiles would fit beside it, and reading A from there bounds the
// products (6 KB for every 52 cycles of an N = 64 step, near 128 bytes a cycle; from TMEM 38 cycles).
//
// A tile of 64 keys is nine [64 x 64] boxes: the four of this half's values, which the context's product
// reads long after the scores, in three places in turn; the four others, whose place is free again as soon
// as their scores are done, a pair at a time; the RoPE box, two places. The products' order is, tile by
// tile, the scores of tile n (20 steps with A in shared memory, then 16 with A in TMEM) and the context of
// tile n - 1 (4 steps), so that the softmax of a tile has the scores of the next one beside it. The products by
// themselves take 2200 of the loop's 2500 cycles a tile, 1660 of which the tensor pipe works: a step of N = 64
// waits for its operands. So no unit is full (counters: pipe 52% of the elapsed cycles, its operands' reads of
// shared memory 56%, the other warps' accesses to it 55%); fewer scores a CTA would help, faster softmax not.
//
// Warp roles: warps 0 .. 3 load the queries (TMA; what goes to TMEM by way of the place of what stays) and do
// the softmax, one row a thread (their TMEM lanes); warp 4 allocates TMEM and issues the MMAs; warps 8 .. 23
// expand the key tiles, eight the values and the RoPE box, eight the others, four lanes a key, each with its
// next tile's bytes under way.
// TMEM columns: query [0,128), S [128,192) and [192,256) in turn, P over its S, O [256,512).
//
// 24 sequences of 4000 .. 16384 tokens, 128 heads (events): 83 us for 67 GFLOP; 131072 tokens alone: 41 us. On
// the way: eight producers with two whole tiles' places 104; sixteen 88; three places for the values 86; two
// values an instruction in the softmax 83. With eight lanes a key (whole lines a load, half the load's
// wavefronts, but one barrier for both pairs) 95 .. 108, with a warp that asks for tiles ahead of time in the
// L2 no gain, with the keys on the MMA's M 176.
#include "cache4.h"
#include "cache4_tc.cuh"
#include "score_mod.cuh"

LAGA_TRACE_DEFINE(cache4)

namespace laga {
namespace {

constexpr int BQ = 128, BKV = 64;
constexpr int NBOX = 9, QBOX = 16384, KBOX = 8192;
constexpr int Q_TMEM = 4;                    // query boxes in TMEM
constexpr int V_BUFS = 3, V_BYTES = 4 * KBOX, PAIR_BYTES = 2 * KBOX;
constexpr int K_BYTES = V_BUFS * V_BYTES + 2 * PAIR_BYTES + 2 * KBOX;  // values, the other boxes in pairs, RoPE
constexpr int Q_BYTES = (NBOX - Q_TMEM) * QBOX;
constexpr int SMEM_BYTES = K_BYTES + Q_BYTES + 1024 + 512;
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
constexpr int SOFTMAX_WARPS = 4, PRODUCER_WARPS = 8, MMA_WARP = 4;
constexpr int NTHREADS = 768;  // warps 5 .. 7 have no work
// Of 80 registers a thread at launch: 136 + 24 + 4 * 80 = 6 * 80. The producers keep theirs, which is as few
// as they need: a spilled value is fetched behind the loads of the next tile, for hundreds of cycles.
constexpr int SOFTMAX_REGS = 136, MMA_REGS = 24;
constexpr uint32_t TMEM_COLS = 512, COL_S = 128, COL_O = 256;
constexpr int HALF = 256;
// kind::f16 with fp16 operands is idesc_bf16 without the two type fields
constexpr uint32_t F16 = ~((1u << 7) | (1u << 10));
constexpr uint32_t IDESC_S = idesc_bf16(BQ, BKV, false, false) & F16;
constexpr uint32_t IDESC_ROPE = idesc_bf16(BQ, BKV, false, false);
constexpr uint32_t IDESC_PV = idesc_bf16(BQ, HALF, false, true) & F16;

struct Params {
  CacheAttn a;
  CacheOperands x;
  float sl2;          // scale * log2(e)
  ModParams mod;      // u_scale, cap_log2
};

// A producer lane's key in the tile to be loaded next: its place among the sequence's pages, kept from tile
// to tile, and its page, fetched a tile before it is used (the fetch behind the loads that need it took a
// third of a producer's time).
struct KeyPlace {
  int at, page_row, loaded;  // loaded: the table's entry, not looked at before it is used (that would wait for it)
  uint32_t page_of;
  bool wanted, in;  // within the item's interval; within the table
  __device__ __forceinline__ void fetch(const CacheAttn& a, const Piece& p) {
    wanted = at >= p.hull.x && at < p.hull.y;
    in = page_of < static_cast<uint32_t>(a.pages.most);
    if (wanted && in) loaded = __ldg(a.pages.table + static_cast<ll>(p.b) * a.pages.most + page_of);
  }
  // the page; -1 for a key outside the interval, -2 for one without a page
  __device__ __forceinline__ int id(const CacheAttn& a) const {
    return !wanted ? -1 : in && loaded >= 0 && loaded < a.cache.pages ? loaded : -2;
  }
  __device__ __forceinline__ void begin(const CacheAttn& a, const Piece& p, int key) {
    at = p.key0 + key;
    page_of = static_cast<uint32_t>(at) / static_cast<uint32_t>(a.cache.page);
    page_row = at - static_cast<int>(page_of) * a.cache.page;
    fetch(a, p);
  }
  __device__ __forceinline__ void step(const CacheAttn& a, const Piece& p) {
    at += BKV;
    page_row += BKV;
    if (page_row >= a.cache.page) {
      page_row -= a.cache.page;
      ++page_of;
      if (page_row >= a.cache.page) {  // pages of less than a tile
        const int k = page_row / a.cache.page;
        page_row -= k * a.cache.page;
        page_of += k;
      }
    }
    fetch(a, p);
  }
};

// What a producer lane holds of one key tile: of each of two pairs of boxes 16 bytes of codes, two blocks,
// and their scales; for the VALUES' boxes also two of the key's eight RoPE chunks. Few wide loads: every
// load of a warp touches eight keys' lines.
template <bool VALUES>
struct Held {
  uint4 codes[2], rope[VALUES ? 2 : 1];
  uint32_t scales[2];
  bool live, bad;  // a key to expand (else zeros); a key that should be there and is not
};
template <bool VALUES>
__device__ __forceinline__ void hold(const CacheAttn& a, const KeyPlace& k, int lane4, int half, Held<VALUES>& h) {
  const int id = k.id(a);
  h.live = id >= 0;
  h.bad = id == -2;
  const ll slot = h.live ? static_cast<ll>(id) * a.cache.page + k.page_row : 0;
  const uint4* c = reinterpret_cast<const uint4*>(a.cache.codes + slot * 256 + 128 * half) + lane4;
  const uint16_t* s = reinterpret_cast<const uint16_t*>(a.cache.scales + slot * 32 + 16 * half) + lane4;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    h.codes[i] = __ldg(c + 4 * i);
    h.scales[i] = __ldg(s + 4 * i);
  }
  if constexpr (VALUES) {
    const uint4* r = reinterpret_cast<const uint4*>(static_cast<const bf16*>(a.cache.keys) + slot * 64) + 2 * lane4;
    h.rope[0] = __ldg(r);
    h.rope[1] = __ldg(r + 1);
  }
}

__device__ __forceinline__ void sts16(uint32_t at, const uint4& v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
template <int REGS, bool MORE>
__device__ __forceinline__ void take_registers() {
  if constexpr (MORE)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}

// The key tiles' places in shared memory and their barriers.
struct Tiles {
  uint8_t *values, *pairs, *rope;  // [3] of four boxes; [2], of each tile in turn the first and second pair; [2]
  uint64_t *v_full, *v_free;       // [3] values and RoPE of a tile are there; its context is done
  uint64_t *p_full, *p_free;       // [2] a pair is there; its scores are done
  uint64_t* r_free;                // [2] the tile's scores are done
  uint32_t* bad;                   // [4][16] of each producer, tiles in turn: lanes whose key is not finite
  volatile int* abort_flag;
};

// A producer warp: keys [8 pw, 8 pw + 8) of every key tile, of it the boxes of this CTA's half of the VALUES
// and the RoPE box, or the others. Four lanes a key.
template <bool VALUES>
__device__ __forceinline__ void expand_tiles(const CacheAttn& a, Walk<BQ, BKV>& walk, int pw, int vh, const Tiles& t) {
  const int lane = threadIdx.x & 31, key = 8 * pw + (lane >> 2), b4 = lane & 3, half = VALUES ? vh : 1 - vh;
  const uint32_t row = static_cast<uint32_t>(key);
  const bool turned = (b4 & 2) != 0;
  const uint32_t pick = turned ? 0x4441u : 0x4440u;  // the first stored block's scale; the other's with bit 0 turned
  // A lane's two blocks are a half of a box's row, its upper lanes' in the other order, so that eight lanes
  // (two keys) store to eight different 16-byte columns.
  const uint32_t boxes = smem_u32(VALUES ? t.values : t.pairs) + (b4 >> 1) * KBOX + sw128_offset(row, 4 * (b4 & 1) + (b4 & 2));
  Piece pc;
  Held<VALUES> cur;
  KeyPlace place;
  int left = 0;
  bool more = walk.next(pc);  // a tile whose place is known
  auto begin_piece = [&]() {
    left = pc.tiles;
    place.begin(a, pc, key);
  };
  auto take = [&]() {  // that tile's bytes, and the place of the one behind it
    hold<VALUES>(a, place, b4, half, cur);
    if (--left > 0) {
      place.step(a, pc);
    } else {
      more = walk.next(pc);
      if (more) begin_piece();
    }
  };
  if (!more) return;
  begin_piece();
  take();
  bool held = true;
  struct Pair {
    uint4 v[4];
  };
  auto expand = [&](int i) {
    const uint32_t two = cur.live ? cur.scales[i] : 0u;
    const uint32_t s0 = __byte_perm(two, 0, pick) * 0x800080u, s1 = __byte_perm(two, 0, pick ^ 1u) * 0x800080u;
    const uint4 w = cur.codes[i];
    return Pair{{expand8(turned ? w.z : w.x, s0), expand8(turned ? w.w : w.y, s0), expand8(turned ? w.x : w.z, s1),
                 expand8(turned ? w.y : w.w, s1)}};
  };
  auto store = [&](const Pair& p, uint32_t to) {  // columns c, c + 1, c ^ 2, (c ^ 2) + 1 of the box's row
#pragma unroll
    for (int x = 0; x < 4; ++x) sts16(to ^ (16 * x), p.v[x]);
  };
  auto arrive = [&](uint64_t* bar) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  };
  int buf = 0;  // n % V_BUFS
  uint32_t v_ph = 1;
#pragma unroll 1
  for (int n = 0; held; ++n) {
    LAGA_TRACE_POINT(cache4, VALUES ? 3 : 0, n);
    // A block that reads as NaN: zeros here, and every row that sees the key gets NaN. All scales at once: a
    // byte above the largest scale has its upper bit and the sum's set.
    static_assert(kCacheTopScale == 0xe2, "the sum below");
    const uint32_t s01 = cur.scales[0] | cur.scales[1] << 16;
    const uint32_t over = ((s01 & 0x7f7f7f7fu) + 0x1d1d1d1du) & s01 & 0x80808080u;
    bool fine = over == 0 || !cur.live;
    if (!VALUES) {
      fine = fine && !cur.bad;
      if (cur.bad && b4 == 0) report_page(a.status, 305);
    }
    if (__any_sync(0xffffffffu, over != 0)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if ((cur.scales[i] & 0xffu) > kCacheTopScale) cur.scales[i] &= 0xff00u;
        if ((cur.scales[i] >> 8) > kCacheTopScale) cur.scales[i] &= 0xffu;
      }
    }
    // The next tile's bytes go into the same registers, as soon as these have been expanded: a wait for one
    // of a warp's loads can be a wait for all that are under way.
    auto advance = [&]() {
      held = more;
      if (more) take();
    };
    auto report = [&]() {
      const uint32_t odd = ~__ballot_sync(0xffffffffu, fine);  // four lanes a key
      if (lane == 0) t.bad[(n & 3) * 16 + (VALUES ? 8 : 0) + pw] = odd;
    };
    if constexpr (VALUES) {
      if (!pass(&t.v_free[buf], v_ph, t.abort_flag, 402)) return;
      if (!pass(&t.r_free[n & 1], static_cast<uint32_t>(((n >> 1) & 1) ^ 1), t.abort_flag, 403)) return;
      LAGA_TRACE_POINT(cache4, 4, n);
      store(expand(0), boxes + buf * V_BYTES);
      const Pair v1 = expand(1);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool number = finite8(cur.rope[i]);
        fine = fine && (number || !cur.live);
        if (!(number && cur.live)) cur.rope[i] = make_uint4(0, 0, 0, 0);
      }
      const uint32_t rope = smem_u32(t.rope) + (n & 1) * KBOX + sw128_offset(row, 2 * b4);
      sts16(rope, cur.rope[0]);
      sts16(rope ^ 16, cur.rope[1]);
      advance();
      store(v1, boxes + buf * V_BYTES + PAIR_BYTES);
      report();
      arrive(&t.v_full[buf]);
      LAGA_TRACE_POINT(cache4, 16, n);
      if (++buf == V_BUFS) {
        buf = 0;
        v_ph ^= 1;
      }
    } else {
      if (!pass(&t.p_free[0], static_cast<uint32_t>((n & 1) ^ 1), t.abort_flag, 401)) return;
      LAGA_TRACE_POINT(cache4, 1, n);
      store(expand(0), boxes);
      arrive(&t.p_full[0]);
      const Pair v1 = expand(1);
      advance();
      LAGA_TRACE_POINT(cache4, 17, n);
      if (!pass(&t.p_free[1], static_cast<uint32_t>((n & 1) ^ 1), t.abort_flag, 404)) return;
      LAGA_TRACE_POINT(cache4, 18, n);
      store(v1, boxes + PAIR_BYTES);
      report();
      arrive(&t.p_full[1]);
      LAGA_TRACE_POINT(cache4, 2, n);
    }
  }
}

// Shared-memory descriptors differ in their low words alone (the address, and for MN-major tiles the
// distance of their atoms): blocks of four K16 steps take those, so that an MMA costs its warp the fewest
// instructions. With whole descriptors added up outside, a box of four took ~300 cycles to issue beside
// the other roles, twice what it takes to run.
constexpr uint32_t DESC_HIGH = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(const void* at, uint32_t lbo) { return (smem_u32(at) >> 4) | ((lbo >> 4) << 16); }
// D (+)= A B over four steps; a, b: low words, `b_step` between the steps of b (A's are 2, or 8 TMEM columns).
template <bool A_TMEM, uint32_t B_STEP>
__device__ __forceinline__ void mma4(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (A_TMEM)
    asm volatile(
        "{\n\t.reg .pred e, p, t;\n\t.reg .b32 x, y;\n\t.reg .b64 v;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.eq.b32 t, %3, %3;\n\t"
        "mov.b64 v, {%2, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], v, %3, p;\n\t"
        "add.u32 x, %1, 8;\n\tadd.u32 y, %2, %6;\n\tmov.b64 v, {y, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], v, %3, t;\n\t"
        "add.u32 x, %1, 16;\n\tadd.u32 y, %2, %7;\n\tmov.b64 v, {y, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], v, %3, t;\n\t"
        "add.u32 x, %1, 24;\n\tadd.u32 y, %2, %8;\n\tmov.b64 v, {y, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [x], v, %3, t;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(DESC_HIGH), "n"(B_STEP), "n"(2 * B_STEP), "n"(3 * B_STEP)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred e, p, t;\n\t.reg .b32 x, y;\n\t.reg .b64 u, v;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.eq.b32 t, %3, %3;\n\t"
        "mov.b64 u, {%1, %5};\n\tmov.b64 v, {%2, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], u, v, %3, p;\n\t"
        "add.u32 x, %1, 2;\n\tadd.u32 y, %2, %6;\n\tmov.b64 u, {x, %5};\n\tmov.b64 v, {y, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], u, v, %3, t;\n\t"
        "add.u32 x, %1, 4;\n\tadd.u32 y, %2, %7;\n\tmov.b64 u, {x, %5};\n\tmov.b64 v, {y, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], u, v, %3, t;\n\t"
        "add.u32 x, %1, 6;\n\tadd.u32 y, %2, %8;\n\tmov.b64 u, {x, %5};\n\tmov.b64 v, {y, %5};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], u, v, %3, t;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "r"(DESC_HIGH), "n"(B_STEP), "n"(2 * B_STEP), "n"(3 * B_STEP)
        : "memory");
}

// A bit for each four lanes of which some bit is set.
__device__ __forceinline__ uint32_t keys_of(uint32_t lanes) {
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) bits |= ((lanes >> (4 * i)) & 15u) ? 1u << i : 0u;
  return bits;
}

__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
template <int MOD>
__global__ void __launch_bounds__(NTHREADS, 1) cache4_attn_kernel(const __grid_constant__ CUtensorMap mQ, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint8_t* sQ = smem + K_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sQ + Q_BYTES);
  uint64_t* s_full = bars + 12;   // [2] the scores in that place are there
  uint64_t* p_full = bars + 14;
  uint64_t* pv_done = bars + 15;  // P read, O up to date
  uint64_t* q_full = bars + 16;   // the TMEM boxes are there
  uint64_t* q_stage = bars + 17;  // they are in shared memory
  uint64_t* q_rest = bars + 18;   // the other boxes are there
  uint64_t* q_idle = bars + 19;   // the softmax warps are done with the queries' place
  uint64_t* drain = bars + 20;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 21);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const Tiles t{smem, smem + V_BUFS * V_BYTES, smem + V_BUFS * V_BYTES + 2 * PAIR_BYTES, bars, bars + 3, bars + 6, bars + 8,
                bars + 10, reinterpret_cast<uint32_t*>(bars + 22), abort_flag};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const CacheAttn& a = p.a;
  const int part = blockIdx.x >> 1, vh = blockIdx.x & 1;  // vh: this CTA's half of the context's columns

  if (threadIdx.x == 0) {
    for (int i = 0; i < V_BUFS; ++i) {
      mbar_init(&t.v_full[i], PRODUCER_WARPS);
      mbar_init(&t.v_free[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&t.p_full[i], PRODUCER_WARPS);
      mbar_init(&t.p_free[i], 1);
      mbar_init(&t.r_free[i], 1);
      mbar_init(&s_full[i], 1);
    }
    mbar_init(p_full, SOFTMAX_WARPS);
    mbar_init(pv_done, 1);
    mbar_init(q_full, SOFTMAX_WARPS);
    mbar_init(q_stage, 1);
    mbar_init(q_rest, 1);
    mbar_init(q_idle, SOFTMAX_WARPS);
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
  LAGA_TRACE_CTA_BEGIN(cache4);

  Walk<BQ, BKV> walk(a, part);
  Piece pc;
  if (warp >= 8) {
    // ---------------- expand key tiles: four of each kind in turn, so that each scheduler has some of both
    const int i = warp - 8, pw = 4 * (i >> 3) + (i & 3);
    if ((i & 4) == 0)
      expand_tiles<false>(a, walk, pw, vh, t);
    else
      expand_tiles<true>(a, walk, pw, vh, t);
  } else if (warp > MMA_WARP) {
    take_registers<MMA_REGS, false>();
  } else if (warp == MMA_WARP) {
    take_registers<MMA_REGS, false>();
    // ---------------- products
    bool ok = true, issued = false;
    const uint32_t q_low = desc_low(sQ, 16), pair_low = desc_low(t.pairs, 16), rope_low = desc_low(t.rope, 16);
    const uint32_t key_low = desc_low(t.values, 16), value_low = desc_low(t.values, KBOX);
    int n = 0, seg = 0, buf = 0, before = V_BUFS - 1;  // n % V_BUFS, (n - 1) % V_BUFS
    uint32_t v_ph = 0;
    auto context = [&](int m, int at, bool first) -> bool {  // O (+)= P(m) V(m)
      if (!pass(p_full, m & 1, abort_flag, 411)) return false;
      LAGA_TRACE_POINT(cache4, 7, m);
      tc_fence_after();
      mma4<true, 2048 / 16>(tmem + COL_O, tmem + COL_S + (m & 1) * BKV, value_low + at * (V_BYTES / 16), IDESC_PV, first ? 0u : 1u);
      mma_commit_warp(&t.v_free[at]);
      mma_commit_warp(pv_done);
      return true;
    };
    while (ok && walk.next(pc)) {
      ok = pass(q_full, seg & 1, abort_flag, 412) && pass(q_rest, seg & 1, abort_flag, 416);
      ++seg;
      for (int j = 0; j < pc.tiles && ok; ++j, ++n) {
        // All of a tile's scores before the context of the tile before, so that its weights are worked out
        // beside them; first the pairs, whose places are refilled as soon as their scores are done. (P of the
        // tile two before, in this S's place, was read by a product issued earlier.) The scores of two tiles
        // can be done before a softmax warp has looked at the first, so each place has its own barrier: it is
        // over again with the tile after next, which waits for all four warps' weights of this one.
        const uint32_t s = tmem + COL_S + (n & 1) * BKV;
#pragma unroll
        for (int i = 0; i < 2 && ok; ++i) {
          ok = pass(&t.p_full[i], n & 1, abort_flag, 413 + i);
          if (!ok) break;
          tc_fence_after();
          LAGA_TRACE_POINT(cache4, 5 + i, n);
          mma4<false, 2>(s, q_low + 2 * i * (QBOX / 16), pair_low + i * (PAIR_BYTES / 16), IDESC_S, i ? 1u : 0u);
          mma4<false, 2>(s, q_low + (2 * i + 1) * (QBOX / 16), pair_low + i * (PAIR_BYTES / 16) + KBOX / 16, IDESC_S, 1u);
          mma_commit_warp(&t.p_free[i]);
          issued = true;
        }
        ok = ok && pass(&t.v_full[buf], v_ph, abort_flag, 415);
        if (!ok) break;
        tc_fence_after();
        LAGA_TRACE_POINT(cache4, 11, n);
        mma4<false, 2>(s, q_low + 4 * (QBOX / 16), rope_low + (n & 1) * (KBOX / 16), IDESC_ROPE, 1u);
#pragma unroll
        for (int c = 0; c < Q_TMEM; ++c)
          mma4<true, 2>(s, tmem + 32 * c, key_low + buf * (V_BYTES / 16) + c * (KBOX / 16), IDESC_S, 1u);
        mma_commit_warp(&t.r_free[n & 1]);
        mma_commit_warp(&s_full[n & 1]);
        LAGA_TRACE_POINT(cache4, 12, n);
        if (j > 0) ok = context(n - 1, before, j == 1);
        before = buf;
        if (++buf == V_BUFS) {
          buf = 0;
          v_ph ^= 1;
        }
      }
      if (ok) ok = context(n - 1, before, pc.tiles == 1);
    }
    if (!ok && issued) {
      mma_commit_warp(drain);
      if (lane == 0) mbar_drain(drain, 0);
      __syncwarp();
    }
  } else {
    take_registers<SOFTMAX_REGS, true>();
    // ---------------- queries and softmax: thread = row of the tile = TMEM lane
    const int r = threadIdx.x;
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    const float nan = __int_as_float(0x7fc00000);
    int n = 0, seg = 0;
    bool ok = true, staged = false, rest = false;  // warp 0: copies of this piece are under way or done
    while (ok && walk.next(pc)) {
      staged = rest = false;
      const bool there = r < pc.rows;
      const ll row = static_cast<ll>(pc.b) * a.rows + pc.r0 + (there ? r : 0);
      const int qi = (pc.r0 + r) / a.n_h, h = pc.r0 + r - qi * a.n_h;
      const int2 seen = there ? cache_row_bounds(a, pc.b, qi) : make_int2(0, 0);
      const ll row0 = static_cast<ll>(pc.b) * a.rows + pc.r0;
      // q_idle's phases: twice a piece, after the boxes for TMEM have been read and after O is out
      if (warp == 0) {
        if (seg > 0 && !pass(q_idle, 1, abort_flag, 424)) { ok = false; break; }
        if (lane == 0) {
          mbar_arrive_expect_tx(q_stage, Q_TMEM * QBOX);
          for (int c = 0; c < Q_TMEM; ++c) tma_load_2d(sQ + c * QBOX, &mQ, q_stage, 64 * (4 * vh + c), static_cast<int>(row0));
        }
        staged = true;
      }
      const float up = there ? __ldcg(p.x.up + row) : 1.f;
      bool odd = up != up && seen.x < seen.y;  // the row's result is NaN (one that sees nothing is 0 whatever it holds)
      if (!pass(q_stage, seg & 1, abort_flag, 425)) { ok = false; break; }
#pragma unroll 1
      for (int c = 0; c < Q_TMEM; ++c) {
        uint32_t u[32];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 v = *reinterpret_cast<const uint4*>(sQ + c * QBOX + sw128_offset(static_cast<uint32_t>(r), static_cast<uint32_t>(i)));
          u[4 * i] = v.x;
          u[4 * i + 1] = v.y;
          u[4 * i + 2] = v.z;
          u[4 * i + 3] = v.w;
        }
        tmem_st32(tmem + 32 * c + lane_off, u);
      }
      fence_proxy_async_smem();  // read before the next copies write there
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(q_idle);
        mbar_arrive(q_full);
      }
      if (warp == 0) {
        if (!pass(q_idle, 0, abort_flag, 426)) { ok = false; break; }
        if (lane == 0) {
          mbar_arrive_expect_tx(q_rest, Q_BYTES);
          for (int c = 0; c < 5; ++c)
            tma_load_2d(sQ + c * QBOX, &mQ, q_rest, c < 4 ? 64 * (4 * (1 - vh) + c) : 512, static_cast<int>(row0));
        }
        rest = true;
      }
      ++seg;
      LAGA_TRACE_POINT(cache4, 13, n);

      const float f = up * (MOD & kModFar ? p.mod.u_scale : MOD & kModCap ? p.mod.u_scale * 2.8853900817779268f : p.sl2);
      float slope2 = 0.f, pos = 0.f;
      if constexpr ((MOD & kModBias) != 0) {
        if (there) slope2 = __ldg(p.mod.slopes + h) * 1.4426950408889634f;
        pos = static_cast<float>(__ldg(a.lengths + pc.b) - a.Sq + qi - pc.key0);
      }
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < pc.tiles && ok; ++j, ++n) {
        if (!pass(&s_full[n & 1], (n >> 1) & 1, abort_flag, 421)) { ok = false; break; }
        LAGA_TRACE_POINT(cache4, 8, n);
        tc_fence_after();
        uint32_t x[64];
        const uint32_t s_at = tmem + COL_S + (n & 1) * BKV + lane_off;
        tmem_ld32(s_at, *reinterpret_cast<uint32_t(*)[32]>(x));
        tmem_ld32(s_at + 32, *reinterpret_cast<uint32_t(*)[32]>(x + 32));
        // lanes of the producers whose key is not finite, by eights of them; a bit a key
        uint2 bits = make_uint2(0, 0);
        {
          uint32_t w[8], any = 0;
          const uint32_t at = smem_u32(t.bad + (n & 3) * 16);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint4 x, y;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at + 16 * i));
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w) : "r"(at + 16 * i + 32));
            w[4 * i] = x.x | y.x;
            w[4 * i + 1] = x.y | y.y;
            w[4 * i + 2] = x.z | y.z;
            w[4 * i + 3] = x.w | y.w;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) any |= w[i];
          if (any)
            bits = make_uint2(keys_of(w[0]) | keys_of(w[1]) << 8 | keys_of(w[2]) << 16 | keys_of(w[3]) << 24,
                              keys_of(w[4]) | keys_of(w[5]) << 8 | keys_of(w[6]) << 16 | keys_of(w[7]) << 24);
        }
        tmem_wait_ld();
        const int k0 = pc.key0 + j * BKV;
        // f turns a product into log2 units, or with a cap c into the exponent of e^2u = 2^(f s):
        // c tanh(u) = c - 2 c / (1 + e^2u), to 1e-7 of c; far: by tanh_rel, which is small where u is
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          F2 v = mul(f2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), f2(f));
          if constexpr ((MOD & (kModCap | kModFar)) == kModCap) {
            const float2 e = parts(v);
            const float2 y = parts(add(f2(ex2_approx(e.x), ex2_approx(e.y)), f2(1.f)));
            v = fma(f2(rcp_approx(y.x), rcp_approx(y.y)), f2(-2.f * p.mod.cap_log2), f2(p.mod.cap_log2));
          }
          const float2 s = parts(v);
          x[2 * i] = __float_as_uint(s.x);
          x[2 * i + 1] = __float_as_uint(s.y);
        }
        if constexpr ((MOD & (kModFar | kModBias)) != 0) {
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            float s = __uint_as_float(x[i]);
            if constexpr ((MOD & kModFar) != 0) s = tanh_rel(s) * p.mod.cap_log2;
            if constexpr ((MOD & kModBias) != 0) s = fmaf(-slope2, fabsf(pos - static_cast<float>(j * BKV + i)), s);
            x[i] = __float_as_uint(s);
          }
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
        F2 sums = f2(0.f);
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float2 s = parts(add(f2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), f2(neg)));
          const float w0 = ex2_approx(s.x), w1 = ex2_approx(s.y);
          sums = add(sums, f2(w0, w1));
          pk[i] = pack_f16x2(w0, w1);
        }
        const float sum = parts(sums).x + parts(sums).y;
        l = fmaf(l, alpha, sum);
        LAGA_TRACE_POINT(cache4, 9, n);
        // O is the products' until the tile before is done
        if (j > 0 && !pass(pv_done, (n - 1) & 1, abort_flag, 422)) { ok = false; break; }
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
        tmem_st32(s_at, pk);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
        LAGA_TRACE_POINT(cache4, 10, n);
      }
      if (!ok || !pass(pv_done, (n - 1) & 1, abort_flag, 423)) { ok = false; break; }
      tc_fence_after();
      if (odd) l = nan;
      LAGA_TRACE_POINT(cache4, 14, n);
      // O out, 128 bytes a row at a time, turned in the queries' place (their products are done) so that a
      // store writes whole lines.
      const uint32_t o = tmem + COL_O + lane_off;
      uint8_t* stage = sQ + warp * 4096;
      const bool whole = pc.begins && pc.ends;
      const ll slot = static_cast<ll>(2 * part + (pc.begins ? 1 : 0)) * BQ;
      if (whole && l == 0.f && seen.x < seen.y) l = nan;  // every score it sees is -inf
      const float inv = l != l ? nan : l == 0.f ? 0.f : 1.f / l;
      if (there && vh == 0) {
        if (whole)
          a.lse[(static_cast<ll>(pc.b) * a.n_h + h) * a.Sq + qi] = l == 0.f ? -INFINITY : fmaf(m, 0.6931471805599453f, logf(l));
        else
          a.part_ml[slot + r] = make_float2(m, l);
      }
      float* out = (whole ? p.x.ctx + row0 * 512 : a.part_o + slot * 512) + vh * HALF;
      const float by = whole ? inv : 1.f;
#pragma unroll 1
      for (int c = 0; c < HALF / 32; ++c) {
        uint32_t u[32];
        tmem_ld32(o + c * 32, u);
        tmem_wait_ld();
#pragma unroll
        for (int v = 0; v < 8; ++v) {
          float4 w;
          w.x = __uint_as_float(u[4 * v]) * by;
          w.y = __uint_as_float(u[4 * v + 1]) * by;
          w.z = __uint_as_float(u[4 * v + 2]) * by;
          w.w = __uint_as_float(u[4 * v + 3]) * by;
          *reinterpret_cast<float4*>(stage + sw128_offset(lane, v)) = w;
        }
        // row by row of the warp's 32, 16 bytes a lane
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = 4 * i + (lane >> 3);
          const float4 v = *reinterpret_cast<const float4*>(stage + sw128_offset(static_cast<uint32_t>(rr), lane & 7u));
          if (warp * 32 + rr < pc.rows) *reinterpret_cast<float4*>(out + (warp * 32 + rr) * 512 + c * 32 + 4 * (lane & 7)) = v;
        }
        __syncwarp();
      }
      LAGA_TRACE_POINT(cache4, 15, n);
      tc_fence_before();  // O has been read before the next piece's products overwrite it (q_full, p_full)
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_idle);
    }
    if (!ok && warp == 0 && lane == 0) {  // given up: let the copies under way land
      const uint32_t ph = static_cast<uint32_t>((rest ? seg - 1 : seg) & 1);
      if (staged) mbar_drain(q_stage, ph);
      if (rest) mbar_drain(q_rest, ph);
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  LAGA_TRACE_CTA_END(cache4);
  if (threadIdx.x == 0) publish_abort(abort_flag, a.status);
  if (warp == MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

}  // namespace

LaunchResult cache4_tc_attn(const CacheAttn& a, const CacheOperands& x, cudaStream_t st) {
  const ll rows = static_cast<ll>(a.pages.B) * a.rows;
  LaunchResult r;
  CUtensorMap mQ;
  const uint64_t dims[2] = {kQueryBytes / 2, static_cast<uint64_t>(rows)}, strides[1] = {kQueryBytes};
  const uint32_t box[2] = {64, BQ};
  r.cu = make_tmap(&mQ, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x.query, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
  if (!r.ok()) {
    r.what = "tensor map cache4 queries";
    return r;
  }
  Params p{};
  p.a = a;
  p.x = x;
  p.sl2 = a.scale * 1.4426950408889634f;
  Dims d{};
  d.scale = a.scale;
  p.mod = mod_params(d, a.mods);
  auto kern = cache4_attn_kernel<0>;
  switch (mod_of(a.mods) | (a.mods.cap > kFarCap ? kModFar : 0)) {
    case 0: break;
    case kModCap: kern = cache4_attn_kernel<kModCap>; break;
    case kModBias: kern = cache4_attn_kernel<kModBias>; break;
    case kModCap | kModBias: kern = cache4_attn_kernel<kModCap | kModBias>; break;
    case kModCap | kModFar: kern = cache4_attn_kernel<kModCap | kModFar>; break;
    default: kern = cache4_attn_kernel<kModCap | kModBias | kModFar>; break;
  }
  r.err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (r.err == cudaSuccess) r.err = launch_next(kern, 2 * a.parts, NTHREADS, SMEM_BYTES, st, mQ, p);
  if (r.err != cudaSuccess) r.what = "cache4_attn";
  return r;
}

}  // namespace laga
