// Masked attention forward on the tensor cores (d_qk = 128 + 64, d_v = 128, bf16 operands,
// fp32 softmax): each query row sees an interval of keys; scores may be capped by a tanh and
// carry a bias by distance.
//
//   t2 = log2(e) * (cap tanh(scale q.K / cap) - slope |pos - j|), masked: -inf
//   P = 2^(t2 - m), l = sum P, O = sum P V, out = O / l, lse = (m + log2 l) / log2(e)
//
// A packed batch is many short key ranges: one CTA per query tile spent ~9 us a tile on its
// own start and end, around 1 to 5 key tiles of 0.7 us. So one CTA per SM stays and takes (head,
// query tile) items from a ticket, longest of a head first, and a new item's tiles enter the
// pipeline while the last one's are still in it. And the masked softmax is longer than the plain
// one (a bias: +70% of the instructions, a cap: twice), at one warp per scheduler issuing every
// third cycle: two warpgroups share the score tiles, one the even ones, one the odd ones.
// 2 x 4096 rows of 16 heads in 1 / 5 / 40 documents, us, against one CTA per query tile:
//   mask alone 179 / 90 / 51 (143 / 92 / 67)   bias 200 / 103 / 57 (234 / 124 / 78)
//   cap 262 / 134 / 69 (269 / 168 / 96)
// What bounds it: a 128 x 128 tile's products move 208 KB through shared memory, 1625 cycles at
// 128 B a cycle, and take ~2100 with their hand-offs; a warpgroup has twice that for its softmax
// and needs ~2600. S(g) -> P(g) -> S(g + 3) is the chain that sets the pace.
//
// Warp roles (384 threads):
//   warp 0      lane 0: tickets and the item ring; TMA for Q (per item) and K tiles
//   warp 1      TMEM allocation; the MMA issue loop (elected lane)
//   warp 2      lane 0: TMA for V tiles
//   warp 3      the waiter: waits on each mbarrier the next MMA group needs, then meets
//               warp 1 at a named barrier (the AND of their flags carries a timeout)
//   warps 4..7, 8..11  softmax: score tile g (counted over all items) belongs to warpgroup
//               g % 2; thread = query row = TMEM lane
// TMEM columns: three S/P buffers [0,384), O [384,512).
//
// MMA order, by tile count over all items: PV(k), then the S tiles up to k + 3; an item's
// first S waits for PV(k - 2) instead, so that its Q (one buffer) has had time to arrive.
//
// The softmax makes one pass over a score tile, a loop of four chunks of 32 columns (unrolled, it
// outgrows the instruction cache and its warps wait for instructions; a second pass for the
// maximum reads the tile from TMEM and caps it twice). Its weights
// count in 2^m for a reference m that is 0 until scores turn out to be further than 2^32 off;
// then m moves, and what was written of the tile so far is scaled. At a tile's end the warpgroup
// settles m with the one that tile g - 1 left for the row in shared memory (the larger stays;
// weights and O follow it), passes it on and hands P over. With a bias the tiles are walked from
// the last key back, so that the nearest (largest) come first. Each warpgroup sums its own tiles'
// weights; the one with the item's last tile adds the other's and writes the rows out, while the
// other has begun the next item.
#include "internal.h"
#include "ptx.cuh"
#include "score_mod.cuh"

#include <algorithm>

namespace laga {
namespace {

constexpr int BQ = 128;
constexpr int BKV = 128;
constexpr int BOX = 16384;  // one [128 rows][64 cols] bf16 box
constexpr int Q_BYTES = 3 * BOX;
constexpr int K_BYTES = 3 * BOX;
constexpr int V_BYTES = 2 * BOX;
constexpr int K_STAGES = 2;
constexpr int V_STAGES = 2;
constexpr int NBUF = 3;   // S/P buffers in TMEM
constexpr int RING = 6;   // items known to the roles at a time; the S tiles run up to 3 items ahead
constexpr int PREFETCH = 4;  // K/V tiles requested into L2 this far ahead of their load
constexpr int STAGE_BOX = 32 * 64;  // per softmax warp: [32 rows][32 cols] bf16 of the output
constexpr int OFF_K = Q_BYTES;
constexpr int OFF_V = OFF_K + K_STAGES * K_BYTES;
constexpr int OFF_STAGE = OFF_V + V_STAGES * V_BYTES;
constexpr int OFF_M = OFF_STAGE + 8 * STAGE_BOX;  // [128] the rows' reference
constexpr int OFF_L = OFF_M + 128 * 4;            // [2][128] the other warpgroup's sums, by item parity
constexpr int OFF_ITEMS = OFF_L + 2 * 128 * 4;    // [RING] int4
constexpr int OFF_BARS = OFF_ITEMS + RING * 16;
constexpr int N_BARS = 2 + 2 * K_STAGES + 2 * V_STAGES + 3 * NBUF + 2 + 2 * RING + 4 + 8;
constexpr int SMEM_BYTES = OFF_BARS + N_BARS * 8 + 8 + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
constexpr int NTHREADS = 384;
constexpr int HANDOFF_BAR = 1;  // named barrier of warp 1 and the waiter (64 threads)
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t COL_O = 384;
constexpr uint32_t IDESC_S = idesc_bf16(128, 128, false, false);
constexpr uint32_t IDESC_PV = idesc_bf16(128, 128, false, true);
constexpr float LOG2E = 1.4426950408889634f;
// The weights are 2^(t2 - m) for a reference m that need not be the maximum, only near enough:
// bf16 and fp32 have the same exponents, so 2^32 rounds no worse than 1. But O holds weights times
// V in fp32: with 2^FAR at most, 2^16 keys of a V up to 2^80 stay finite, and with 2^-FAR at least
// a V down to 2^-80 keeps its bits. (A FAR of 100 lost both ends at V of 2^36 and 2^-40 and was no
// faster: 2 x 4096 rows with a bias take 478 us the step with either.) Below 32, scores of ordinary size would
// move the reference. A row starts with m = 0; m is always a whole number, so that a move to another m
// scales weights by a power of two, exactly.
constexpr float FAR = 32.f;  // scores further off than this move the reference
// The bounded waits of this kernel, kept short: a wait is inlined a dozen times, and the control
// warps' code competes for the instruction cache with the softmax (with the clock-reading form
// the issue loop took some 1750 cycles a tile, most of it waiting for instructions). The limit
// counts tries; a try suspends the thread for a while, so it is at least tens of milliseconds.
constexpr uint32_t kTries = 1u << 22;
__device__ __forceinline__ bool wait1(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int where) {
  const uint32_t addr = smem_u32(bar);
#pragma unroll 1
  for (uint32_t it = 0; it < kTries; ++it) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(addr), "r"(parity)
        : "memory");
    if (ok) return true;
    if (*abort_flag) return false;
  }
  *abort_flag = kStatusTimeout | (where << 8);
  return false;
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int where) {
  bool w = true;
  if ((threadIdx.x & 31) == 0) w = wait1(bar, parity, abort_flag, where);
  const bool all = __shfl_sync(0xffffffffu, w ? 1 : 0, 0) != 0;
  __syncwarp();  // order lane 0's acquire before the other lanes' reads
  return all;
}

struct Params {
  int* status;
  int Sq, n_h, q_offset, q_split, q_offset2, skv_pad, n_q_tiles;
  int total;  // items: B * n_h * n_q_tiles
  float scale_log2;
  float* lse;
  const int2* rows;  // [B][n_q_tiles * 128] visible interval of each query row
  const int4* work;  // [B][n_q_tiles] {query tile, first key tile, key tiles}, longest first
  int* ticket;
  ModParams mod;
};

// 32 raw scores -> exponents t2, -inf where masked. [first, end): the visible keys among
// them, where not all are (partial); dist: to the first of them.
template <bool CAP, bool BIAS>
__device__ __forceinline__ void exponents(uint32_t (&x)[32], bool partial, int first, int end,
                                          const Params& p, float slope2, float dist) {
  if (CAP && partial) {  // a masked score must not decide how the row's others are capped
    const uint32_t bits = visible_bits(first, end);
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (!((bits >> k) & 1u)) x[k] = 0u;
  }
  if constexpr (CAP) {
    if (all_small<32>(x, p.mod.u_scale)) {
      const F2 us = f2(p.mod.u_scale), c2 = f2(p.mod.cap_log2);
#pragma unroll
      for (int k = 0; k < 32; k += 2) {
        const F2 u = mul(f2(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), us);
        const float2 t = parts(mul(mul(u, c2), tanh_over_u(mul(u, u))));
        x[k] = __float_as_uint(t.x);
        x[k + 1] = __float_as_uint(t.y);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        x[k] = __float_as_uint(p.mod.cap_log2 * tanh_abs(__uint_as_float(x[k]) * p.mod.u_scale));
    }
  }
  if constexpr (BIAS) {
    const float scale = CAP ? 1.f : p.scale_log2;
    const float last = dist - 31.f;
    const bool up = dist >= 0.f && last >= 0.f, down = dist <= 0.f && last <= 0.f;
    if (__all_sync(0xffffffffu, up || down)) {  // linear in k: -slope2 |dist - k| = s dist - s k
      const float s = up ? -slope2 : slope2, base = s * dist;
#pragma unroll
      for (int k = 0; k < 32; ++k)
        x[k] = __float_as_uint(fmaf(__uint_as_float(x[k]), scale, fmaf(-s, static_cast<float>(k), base)));
    } else {
#pragma unroll
      for (int k = 0; k < 32; ++k)
        x[k] = __float_as_uint(fmaf(-slope2, fabsf(dist - static_cast<float>(k)), __uint_as_float(x[k]) * scale));
    }
  }
  if (partial) {
    const uint32_t bits = visible_bits(first, end);
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if (!((bits >> k) & 1u)) x[k] = 0xff800000u;  // -inf
  }
}

// 2^d for a whole d <= 0 as two factors: what is scaled may be as large as 2^FAR times a sum, so
// that 2^d alone, below the smallest fp32, would lose it.
struct Pow2 {
  float a, b;
  __device__ __forceinline__ explicit Pow2(float d) {
    const int n = static_cast<int>(fmaxf(d, -252.f)), h = n / 2;
    a = __int_as_float((h + 127) << 23);
    b = __int_as_float((n - h + 127) << 23);
  }
  __device__ __forceinline__ float operator()(float x) const { return x * a * b; }
};

struct Item {
  int bh, t, j0, n;  // n < 0: no more items
};

// Absolute position of local query row i (a query tile never straddles the segments).
__device__ __forceinline__ int q_pos(const Params& p, int i) {
  return (p.q_split > 0 && i >= p.q_split) ? p.q_offset2 + (i - p.q_split) : p.q_offset + i;
}

// One hand-off: PV(k) (item ip's tile jp) and / or S(g) (item is's tile js).
struct Step {
  bool pv, s;
  int k, ip, jp, g, is, js, n;  // n: key tiles of item is
};

// The order of the tensor products, walked alike by the waiter and the MMA warp: step() ends
// at the named barrier and returns what it says; read(i, item, last use) waits for an item. A
// warp that leaves for any reason but the barrier's own answer meets the other there once more
// (finish), so that neither stays behind.
enum class Walk { kDone, kHandoffFailed, kReadFailed };
template <class Read, class Do>
__device__ __forceinline__ Walk walk(Read&& read, Do&& step) {
  Item si{}, pi{};
  int is = 0, js = 0, gs = 0, ip = 0, jp = 0;
  bool s_end = false;
  for (int k = -1;; ++k) {
    bool pv = k >= 0;
    if (pv && jp == 0) {
      if (!read(ip, pi, true)) return Walk::kReadFailed;
      if (pi.n < 0) return Walk::kDone;
    }
    for (;;) {  // PV(k) with the first S due, then the others
      bool s = !s_end && gs <= k + (js == 0 && gs > 0 ? 2 : 3);
      if (s && js == 0) {
        if (!read(is, si, false)) return Walk::kReadFailed;
        if (si.n < 0) {
          s_end = true;
          s = false;
        }
      }
      if (!pv && !s) break;
      if (!step(Step{pv, s, k, ip, jp, gs, is, js, si.n})) return Walk::kHandoffFailed;
      if (pv) {
        if (++jp == pi.n) {
          jp = 0;
          ++ip;
        }
        pv = false;
      }
      if (!s) break;
      ++gs;
      if (++js == si.n) {
        js = 0;
        ++is;
      }
    }
  }
}

__device__ __forceinline__ bool finish(Walk w) {
  return w != Walk::kHandoffFailed && bar_and(HANDOFF_BAR, 64, w == Walk::kDone);
}

template <int MOD>
__global__ void __launch_bounds__(NTHREADS, 1)
    attn_fwd_masked_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                           const __grid_constant__ CUtensorMap mR, const __grid_constant__ CUtensorMap mV,
                           const __grid_constant__ CUtensorMap mO, const Params p) {
  constexpr bool CAP = (MOD & kModCap) != 0, BIAS = (MOD & kModBias) != 0;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint8_t* sQ = smem;
  uint8_t* sK = smem + OFF_K;
  uint8_t* sV = smem + OFF_V;
  float* m_ref = reinterpret_cast<float*>(smem + OFF_M);
  float* l_other = reinterpret_cast<float*>(smem + OFF_L);
  int4* items = reinterpret_cast<int4*>(smem + OFF_ITEMS);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BARS);
  uint64_t* q_full = bars + 0;
  uint64_t* q_empty = bars + 1;
  uint64_t* k_full = bars + 2;               // [K_STAGES]
  uint64_t* k_empty = k_full + K_STAGES;     // [K_STAGES]
  uint64_t* v_full = k_empty + K_STAGES;     // [V_STAGES]
  uint64_t* v_empty = v_full + V_STAGES;     // [V_STAGES]
  uint64_t* s_full = v_empty + V_STAGES;     // [NBUF] S(g) -> s_full[g % NBUF]
  uint64_t* p_full = s_full + NBUF;          // [NBUF]
  uint64_t* pv_done = p_full + NBUF;         // [NBUF]
  uint64_t* o_free = pv_done + NBUF;         // an item's O has been read out
  uint64_t* drain = o_free + 1;
  uint64_t* item_full = drain + 1;           // [RING]
  uint64_t* item_empty = item_full + RING;   // [RING]
  uint64_t* m_done = item_empty + RING;      // [4] a quarter's reference after tile g
  uint64_t* l_full = m_done + 4;             // [2][4] a quarter's other sums, by count of items that have them
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(l_full + 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int i = 0; i < K_STAGES; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < V_STAGES; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < NBUF; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&pv_done[i], 1);
    }
    mbar_init(o_free, 4);
    mbar_init(drain, 1);
    for (int i = 0; i < RING; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], 11);  // the V producer, the waiter, the MMA warp, eight softmax warps
    }
    for (int i = 0; i < 4; ++i) mbar_init(&m_done[i], 1);
    for (int i = 0; i < 8; ++i) mbar_init(&l_full[i], 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  after_previous();

  // Item i from the ring, by a whole warp; `last`: this reader is done with the slot.
  auto warp_item = [&](int i, Item& it, bool last, int where) -> bool {
    const int s = i % RING;
    if (!wait_warp(&item_full[s], (i / RING) & 1, abort_flag, where)) return false;
    const int4 v = items[s];
    it = Item{v.x, v.y, v.z, v.w};
    __syncwarp();
    if (last && lane == 0) mbar_arrive(&item_empty[s]);
    return true;
  };

  if (warp < 4) {
    if (warp == 0) {
      if (lane == 0) {
        tma_prefetch_desc(&mQ);
        tma_prefetch_desc(&mK);
        tma_prefetch_desc(&mR);
        auto entry = [&](int idx, int& bh) -> int4 {
          bh = idx / p.n_q_tiles;
          return idx < p.total ? p.work[(bh / p.n_h) * p.n_q_tiles + (idx - bh * p.n_q_tiles)] : make_int4(0, 0, -1, 0);
        };
        // the next item's entry and the ticket after it are on their way while this item's tiles load
        int bh;
        int4 w = entry(atomicAdd(p.ticket, 1), bh);
        int ticket = atomicAdd(p.ticket, 1);
        int gk = 0, i = 0, loads = 0;
        bool ok = true;
        for (;; ++i) {
          const int slot = i % RING;
          if (!wait1(&item_empty[slot], ((i / RING) & 1) ^ 1, abort_flag, 301)) { ok = false; break; }
          items[slot] = make_int4(bh, w.x, w.y, w.z);
          mbar_arrive(&item_full[slot]);
          if (w.z < 0) break;
          int next_bh;
          const int4 next = entry(ticket, next_bh);
          ticket = atomicAdd(p.ticket, 1);
          const int b = bh / p.n_h, h = bh - b * p.n_h;
          if (!wait1(q_empty, (i & 1) ^ 1, abort_flag, 302)) { ok = false; break; }
          mbar_arrive_expect_tx(q_full, Q_BYTES);
          tma_load_3d(sQ, &mQ, q_full, h * 192, w.x * BQ, b);
          tma_load_3d(sQ + BOX, &mQ, q_full, h * 192 + 64, w.x * BQ, b);
          tma_load_3d(sQ + 2 * BOX, &mQ, q_full, h * 192 + 128, w.x * BQ, b);
          ++loads;
          for (int j = 0; j < w.z; ++j, ++gk) {
            const int s = gk % K_STAGES;
            if (!wait1(&k_empty[s], ((gk / K_STAGES) & 1) ^ 1, abort_flag, 303)) { ok = false; break; }
            uint8_t* dst = sK + s * K_BYTES;
            mbar_arrive_expect_tx(&k_full[s], K_BYTES);
            const int kt = BIAS ? w.y + w.z - 1 - j : w.y + j, row = b * p.skv_pad + kt * BKV;
            tma_load_2d(dst, &mK, &k_full[s], h * 128, row);
            tma_load_2d(dst + BOX, &mK, &k_full[s], h * 128 + 64, row);
            tma_load_3d(dst + 2 * BOX, &mR, &k_full[s], 0, kt * BKV, b);
            if (j + PREFETCH < w.z) {
              const int ahead = BIAS ? row - PREFETCH * BKV : row + PREFETCH * BKV;
              tma_prefetch_2d(&mK, h * 128, ahead);
              tma_prefetch_2d(&mK, h * 128 + 64, ahead);
            }
          }
          if (!ok) break;
          w = next;
          bh = next_bh;
        }
        if (!ok) {  // aborted: let issued copies land
          if (loads > 0) mbar_drain(q_full, (loads - 1) & 1);
          for (int k = gk - K_STAGES < 0 ? 0 : gk - K_STAGES; k < gk; ++k)
            mbar_drain(&k_full[k % K_STAGES], (k / K_STAGES) & 1);
        }
      }
    } else if (warp == 2) {
      if (lane == 0) {
        tma_prefetch_desc(&mV);
        int gv = 0;
        bool ok = true;
        for (int i = 0; ok; ++i) {
          const int slot = i % RING;
          if (!wait1(&item_full[slot], (i / RING) & 1, abort_flag, 304)) { ok = false; break; }
          const int4 v = items[slot];
          mbar_arrive(&item_empty[slot]);
          if (v.w < 0) break;
          const int b = v.x / p.n_h, h = v.x - b * p.n_h;
          for (int j = 0; j < v.w; ++j, ++gv) {
            const int s = gv % V_STAGES;
            if (!wait1(&v_empty[s], ((gv / V_STAGES) & 1) ^ 1, abort_flag, 305)) { ok = false; break; }
            uint8_t* dst = sV + s * V_BYTES;
            mbar_arrive_expect_tx(&v_full[s], V_BYTES);
            const int row = b * p.skv_pad + (BIAS ? v.z + v.w - 1 - j : v.z + j) * BKV;
            tma_load_2d(dst, &mV, &v_full[s], h * 128, row);
            tma_load_2d(dst + BOX, &mV, &v_full[s], h * 128 + 64, row);
            if (j + PREFETCH < v.w) {
              const int ahead = BIAS ? row - PREFETCH * BKV : row + PREFETCH * BKV;
              tma_prefetch_2d(&mV, h * 128, ahead);
              tma_prefetch_2d(&mV, h * 128 + 64, ahead);
            }
          }
        }
        if (!ok)
          for (int k = gv - V_STAGES < 0 ? 0 : gv - V_STAGES; k < gv; ++k)
            mbar_drain(&v_full[k % V_STAGES], (k / V_STAGES) & 1);
      }
    } else if (warp == 3) {
      // The waiter: a hand-off's waits side by side, a barrier a lane (one after the other, each a
      // round trip of some 300 cycles beside the MMAs' own traffic, they set the pace of the loop).
      finish(walk([&](int i, Item& it, bool last) { return warp_item(i, it, last, 306); },
                  [&](const Step& t) -> bool {
                    uint64_t* bar = nullptr;
                    uint32_t parity = 0;
                    if (lane == 0 && t.pv) {
                      bar = &p_full[t.k % NBUF];
                      parity = (t.k / NBUF) & 1;
                    } else if (lane == 1 && t.pv) {
                      bar = &v_full[t.k % V_STAGES];
                      parity = (t.k / V_STAGES) & 1;
                    } else if (lane == 2 && t.pv && t.jp == 0 && t.ip > 0) {
                      bar = o_free;
                      parity = (t.ip - 1) & 1;
                    } else if (lane == 3 && t.s) {
                      bar = &k_full[t.g % K_STAGES];
                      parity = (t.g / K_STAGES) & 1;
                    } else if (lane == 4 && t.s && t.js == 0) {
                      bar = q_full;
                      parity = t.is & 1;
                    }
                    bool ok = bar == nullptr;
                    uint32_t it = 0;
                    for (; it < kTries; ++it) {
                      if (!ok) ok = mbar_try_wait(bar, parity);
                      if (__all_sync(0xffffffffu, ok)) break;
                      if (__any_sync(0xffffffffu, *abort_flag != 0)) break;
                    }
                    if (it == kTries) *abort_flag = kStatusTimeout | (308 << 8);
                    return bar_and(HANDOFF_BAR, 64, ok);
                  }));
    } else {
      bool issued = false;
      const uint64_t q_desc = sdesc_sw128(smem_u32(sQ), 16, 1024);
      auto ready = [&]() -> bool {
        const bool r = bar_and(HANDOFF_BAR, 64, true);
        tc_fence_after();
        return r;
      };
      const bool all = finish(walk(
          [&](int i, Item& it, bool last) { return warp_item(i, it, last, 313); },
          [&](const Step& t) -> bool {
            if (!ready()) return false;
            if (t.pv) {
              const int vs = t.k % V_STAGES;
              const uint64_t v_desc = sdesc_sw128(smem_u32(sV + vs * V_BYTES), BOX, 1024);
              const uint32_t p_tmem = tmem + (t.k % NBUF) * 128;
#pragma unroll
              for (int g = 0; g < BKV / 64; ++g) {  // keys [64g, 64g + 64): four K16 steps
                const int kk = 4 * g;
                mma4_ts_warp(tmem + COL_O, p_tmem + kk * 8, p_tmem + kk * 8 + 8, p_tmem + kk * 8 + 16,
                             p_tmem + kk * 8 + 24, v_desc + ((kk * 2048) >> 4), v_desc + (((kk + 1) * 2048) >> 4),
                             v_desc + (((kk + 2) * 2048) >> 4), v_desc + (((kk + 3) * 2048) >> 4), IDESC_PV,
                             (t.jp > 0 || g > 0) ? 1u : 0u);
              }
              mma_commit_warp(&pv_done[t.k % NBUF]);
              mma_commit_warp(&v_empty[vs]);
            }
            if (t.s) {
              const int ks = t.g % K_STAGES;
              const uint64_t k_desc = sdesc_sw128(smem_u32(sK + ks * K_BYTES), 16, 1024);
#pragma unroll
              for (int c = 0; c < 3; ++c) {  // head dims [64c, 64c + 64): four K16 steps in box c
                const uint32_t o = (c * BOX) >> 4;
                mma4_ss_warp(tmem + (t.g % NBUF) * 128, q_desc + o, q_desc + o + 2, q_desc + o + 4, q_desc + o + 6,
                             k_desc + o, k_desc + o + 2, k_desc + o + 4, k_desc + o + 6, IDESC_S, c > 0 ? 1u : 0u);
              }
              issued = true;
              mma_commit_warp(&s_full[t.g % NBUF]);
              mma_commit_warp(&k_empty[ks]);
              if (t.js + 1 == t.n) mma_commit_warp(q_empty);
            }
            return true;
          }));
      if (!all && issued) {
        mma_commit_warp(drain);
        if (lane == 0) mbar_drain(drain, 0);
        __syncwarp();
      }
    }
  } else {
    // ---------------- softmax warpgroups
    const int wg = (warp >> 2) - 1;  // warpgroup: tiles g with g % 2 == wg
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const float sl2 = p.scale_log2;
    uint8_t* stage = smem + OFF_STAGE + (warp - 4) * STAGE_BOX;
    bool ok = true;
    int g0 = 0;      // the item's first tile
    int shared = 0;  // items so far that both warpgroups had tiles of
    for (int i = 0; ok; ++i) {
      Item it;
      if (!warp_item(i, it, true, 314)) { ok = false; break; }
      if (it.n < 0) break;
      const int b = it.bh / p.n_h, h = it.bh - b * p.n_h;
      const int q_row = it.t * BQ + r;
      const int2 v = p.rows[static_cast<long long>(b) * (p.n_q_tiles * BQ) + q_row];
      const bool poisoned = v.x < 0;
      const int lo = v.x & 0x7fffffff, hi = v.y;
      float slope2 = 0.f, pos = 0.f;
      if constexpr (BIAS) {
        slope2 = p.mod.slopes[h] * LOG2E;
        pos = static_cast<float>(q_pos(p, q_row) - it.j0 * BKV);
      }
      const int last_g = g0 + it.n - 1;
      float m = 0.f;      // this warpgroup's reference for the row
      float m_in = 0.f;   // the one that tile g - 1 (the other warpgroup's) left
      bool seen = false;  // some key before this tile was visible, as far as this warpgroup knows
      float l_run = 0.f;  // in units of 2^m
      for (int g = g0 + ((g0 ^ wg) & 1); g <= last_g; g += 2) {
        const int buf = g % NBUF;
        // S(g) is issued after PV(g - 3), so its completion also means P(g - 3) in this
        // buffer has been read.
        if (!wait_warp(&s_full[buf], (g / NBUF) & 1, abort_flag, 315)) { ok = false; break; }
        tc_fence_after();
        const uint32_t s_addr = tmem + buf * 128 + lane_off;
        const int kt = BIAS ? it.n - 1 - (g - g0) : g - g0;  // key tile of the walk
        const int kv0 = (it.j0 + kt) * BKV;
        bool tile_seen = false;
        // weights already written (chunks of 16 columns before `end`) times 2^by
        auto scale_weights = [&](int end, const Pow2& factor) {
          tmem_wait_st();
#pragma unroll 1
          for (int c = 0; c < end; ++c) {
            uint32_t u[16];
            tmem_ld16(s_addr + 16 * c, u);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k)
              u[k] = pack_bf16x2(factor(__uint_as_float(u[k] << 16)), factor(__uint_as_float(u[k] & 0xffff0000u)));
            tmem_st16(s_addr + 16 * c, u);
            tmem_wait_st();
          }
        };
        float left = INFINITY;  // the row's reference after tile g - 1; INFINITY: nothing seen yet
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t x[32];
          tmem_ld32(s_addr + 32 * c, x);
          if (c == 3) {  // read under the last chunk's arithmetic; tile g - 1 has ended half a tile ago
            if (g > 0 && !wait_warp(&m_done[quarter], (g - 1) & 1, abort_flag, 316)) ok = false;
            if (g > g0) left = m_ref[r];
          }
          tmem_wait_ld();
          const int k0 = kv0 + 32 * c;
          const bool partial = !__all_sync(0xffffffffu, lo <= k0 && hi >= k0 + 32);
          exponents<CAP, BIAS>(x, partial, lo - k0, hi - k0, p, slope2,
                               pos - static_cast<float>(kt * BKV + 32 * c));
          float a0 = max3f(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2])), a1 = __uint_as_float(x[3]);
#pragma unroll
          for (int k = 4; k < 32; k += 4) {
            a0 = max3f(a0, __uint_as_float(x[k]), __uint_as_float(x[k + 1]));
            a1 = max3f(a1, __uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
          }
          const float mx = fmaxf(a0, a1) * (CAP || BIAS ? 1.f : sl2);
          const bool before = seen || tile_seen;
          const bool far = mx > m + FAR || (!before && mx < m - FAR && mx > -INFINITY);
          if (__any_sync(0xffffffffu, far)) {
            const float to = far ? rintf(mx) : m;
            const Pow2 factor(before ? m - to : 0.f);  // nothing before: weights and sum are 0
            l_run = factor(l_run);
            scale_weights(c, factor);
            m = to;
          }
          tile_seen = tile_seen || mx > -INFINITY;
          const float neg_m = -m;
          float2 sum2 = make_float2(0.f, 0.f);
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float s0 = __uint_as_float(x[2 * k]), s1 = __uint_as_float(x[2 * k + 1]);
            const float p0 = ex2_approx(CAP || BIAS ? s0 + neg_m : fmaf(s0, sl2, neg_m));
            const float p1 = ex2_approx(CAP || BIAS ? s1 + neg_m : fmaf(s1, sl2, neg_m));
            sum2 = add_f32x2(sum2, make_float2(p0, p1));
            pk[k] = pack_bf16x2(p0, p1);  // rounded once, the MMA's operand type; the sum is not
          }
          l_run += sum2.x + sum2.y;
          tmem_st16(s_addr + 16 * c, pk);  // over score columns that have been read
        }
        if (!ok) break;
        // settle the reference with what tile g - 1 left
        float to = m;
        m_in = 0.f;
        if (left != INFINITY) {
          m_in = left;
          to = tile_seen || seen ? fmaxf(left, m) : left;
          seen = true;
        }
        const bool move_o = left != INFINITY && left != to;
        if (__any_sync(0xffffffffu, to != m)) {
          const Pow2 factor(fminf(m - to, 0.f));  // m > to only where the row has seen nothing here
          l_run = factor(l_run);
          scale_weights(4, factor);
          m = to;
        }
        seen = seen || tile_seen;
        m_ref[r] = seen ? m : INFINITY;
        __syncwarp();
        if (lane == 0) mbar_arrive(&m_done[quarter]);
        if (__any_sync(0xffffffffu, move_o)) {  // O may only be touched once PV(g - 1) has landed
          if (!wait_warp(&pv_done[(g - 1) % NBUF], ((g - 1) / NBUF) & 1, abort_flag, 317)) { ok = false; break; }
          tc_fence_after();
          const uint32_t o_addr = tmem + COL_O + lane_off;
          const Pow2 factor(move_o ? left - to : 0.f);
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t u[16];
            tmem_ld16(o_addr + c * 16, u);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) u[k] = __float_as_uint(factor(__uint_as_float(u[k])));
            tmem_st16(o_addr + c * 16, u);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buf]);
      }
      if (!ok) break;
      const bool mine = (last_g & 1) == wg;  // the item's last tile: this warpgroup writes it out
      if (it.n > 1) {
        // the other warpgroup's last tile was last_g - 1, whose reference is this one's m_in
        float* slot = l_other + (shared & 1) * 128;
        uint64_t* bar = &l_full[(shared & 1) * 4 + quarter];
        if (!mine) {
          slot[r] = l_run;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar);
        } else {
          if (!wait_warp(bar, (shared >> 1) & 1, abort_flag, 318)) { ok = false; break; }
          const float other = slot[r];
          l_run += Pow2(fminf(m_in - m, 0.f))(other);
        }
        ++shared;
      }
      if (mine) {
        if (!wait_warp(&pv_done[last_g % NBUF], (last_g / NBUF) & 1, abort_flag, 319)) { ok = false; break; }
        tc_fence_after();
        const uint32_t o_addr = tmem + COL_O + lane_off;
        // a row that sees nothing: out = 0, lse = -inf; one that sees a non-finite key, or whose
        // scores are all -inf (an infinite q): NaN
        const bool bad = poisoned || (lo < hi && l_run == 0.f);
        const float inv = bad ? NAN : l_run == 0.f ? 0.f : 1.f / l_run;
        uint32_t o[64];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t u[32];
          tmem_ld32(o_addr + c * 32, u);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k)
            o[16 * c + k] = pack_bf16x2(__uint_as_float(u[2 * k]) * inv, __uint_as_float(u[2 * k + 1]) * inv);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(o_free);  // the next item's PV may overwrite O
        if (q_row < p.Sq) {
          const float lse = bad ? NAN : l_run == 0.f ? -INFINITY : (m + __log2f(l_run)) * 0.6931471805599453f;
          p.lse[(static_cast<long long>(b) * p.n_h + h) * p.Sq + q_row] = lse;
        }
        // the warp's 32 rows as four [32 rows][64 B] boxes (64-byte swizzle) through its buffer and
        // tensor-map stores; rows past Sq are clipped by the map
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (lane == 0) bulk_wait_read_all();
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(stage + sw64_offset(lane, k)) =
                make_uint4(o[16 * c + 4 * k], o[16 * c + 4 * k + 1], o[16 * c + 4 * k + 2], o[16 * c + 4 * k + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&mO, stage, h * 128 + 32 * c, it.t * BQ + quarter * 32, b);
            bulk_commit_group();
          }
        }
      }
      g0 += it.n;
    }
    if (lane == 0) bulk_wait_read_all();  // shared memory must not go away under a store
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) publish_abort(abort_flag, p.status);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

}  // namespace

LaunchResult tc_masked_attn_fwd(const Dims& d, const MaskArgs& mask, const bf16* q, const bf16* k_ws, const bf16* v_ws,
                                const bf16* k_rope, bf16* out, float* lse, cudaStream_t st) {
  LaunchResult r;
  CUtensorMap mQ, mK, mR, mV, mO;
  auto rows3 = [&](CUtensorMap* m, const void* base, uint64_t inner, uint64_t rows, uint32_t box_x, uint32_t box_y,
                   CUtensorMapSwizzle swizzle) {
    if (r.cu != CUDA_SUCCESS) return;
    const uint64_t dims[3] = {inner, rows, static_cast<uint64_t>(d.B)};
    const uint64_t strides[2] = {inner * 2, inner * 2 * rows};
    const uint32_t box[3] = {box_x, box_y, 1};
    r.cu = make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, swizzle);
  };
  rows3(&mQ, q, static_cast<uint64_t>(d.n_h) * 192, d.Sq, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B);
  rows3(&mR, k_rope, 64, d.S, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B);
  rows3(&mO, out, static_cast<uint64_t>(d.n_h) * 128, d.Sq, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
  const uint64_t kv_inner = static_cast<uint64_t>(d.n_h) * 128;
  const uint64_t kv_dims[2] = {kv_inner, static_cast<uint64_t>(d.B) * d.skv_pad};
  const uint64_t kv_strides[1] = {kv_inner * 2};
  const uint32_t kv_box[2] = {64, 128};
  if (r.cu == CUDA_SUCCESS)
    r.cu = make_tmap(&mK, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, k_ws, kv_dims, kv_strides, kv_box,
                     CU_TENSOR_MAP_SWIZZLE_128B);
  if (r.cu == CUDA_SUCCESS)
    r.cu = make_tmap(&mV, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, v_ws, kv_dims, kv_strides, kv_box,
                     CU_TENSOR_MAP_SWIZZLE_128B);
  if (r.cu != CUDA_SUCCESS) {
    r.what = "tensor maps masked attention forward";
    return r;
  }
  Params p{};
  p.status = device_status_ptr();
  p.Sq = d.Sq;
  p.n_h = d.n_h;
  p.q_offset = d.q_offset;
  p.q_split = d.q_split;
  p.q_offset2 = d.q_offset2;
  p.skv_pad = d.skv_pad;
  p.n_q_tiles = d.sq_pad / BQ;
  p.total = d.B * d.n_h * p.n_q_tiles;
  p.scale_log2 = d.scale * LOG2E;
  p.lse = lse;
  p.rows = mask.meta.rows;
  p.work = mask.meta.work;
  p.ticket = mask.meta.fwd_ticket;
  p.mod = mod_params(d, mask.mods);
  using M = CUtensorMap;
  void (*kern)(M, M, M, M, M, Params) = attn_fwd_masked_kernel<0>;
  switch (mod_of(mask.mods)) {
    case 0: break;
    case kModCap: kern = attn_fwd_masked_kernel<kModCap>; break;
    case kModBias: kern = attn_fwd_masked_kernel<kModBias>; break;
    default: kern = attn_fwd_masked_kernel<kModCap | kModBias>; break;
  }
  r.err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
  if (r.err != cudaSuccess) {
    r.what = "cudaFuncSetAttribute(attn_fwd_masked)";
    return r;
  }
  r.err = launch_next(kern, std::min(p.total, sm_count()), NTHREADS, SMEM_BYTES, st, mQ, mK, mR, mV, mO, p);
  if (r.err != cudaSuccess) r.what = "attn_fwd_masked_kernel launch";
  return r;
}

}  // namespace laga
