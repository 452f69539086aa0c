// The paged cache of latents in 4 bits: its layout, and the interfaces of the kernels that write it,
// read it and attend over it.
#pragma once
#include "rope.h"

namespace laga {

constexpr int kCacheBlock = 16;      // latent values that share a scale
constexpr int kCacheTopScale = 226;  // largest scale, 1.25 * 2^13: 6 of them are the largest value, 61440
constexpr int kCacheNanScale = 255;  // a block that held a value that is not finite

// A scale byte is the upper 8 of an fp16's 15 bits below the sign. A code of at most two significant
// bits times a scale of at most four is a multiple of 2^-18 of at most 61440: exact in fp16 (and in
// bf16 and fp32), so that what the cache stands for needs no rounding as an operand of a product.
struct CacheView {
  uint8_t* codes;   // [pages][page][ceil(d_c / 2)], the even column in the low half of a byte
  uint8_t* scales;  // [pages][page][ceil(d_c / 16)]
  void* keys;       // [pages][page][d_rope]
  long long pages;
  int page, d_c, d_rope;
  bool is_bf16;  // the keys' type
  __host__ __device__ int code_bytes() const { return (d_c + 1) / 2; }
  __host__ __device__ int blocks() const { return (d_c + kCacheBlock - 1) / kCacheBlock; }
};

// Which pages a sequence's positions lie in: page k of sequence b is table[b][k].
struct PageTable {
  const int* table;  // [B][most]
  int B, most;
};

struct CacheRows {  // rows of a padded batch, at positions starts[b] + i for i < counts[b]
  PageTable pages;
  int rows;           // per sequence
  const int* starts;  // [B]
  const int* counts;  // [B], or null: all
};

struct CacheAppend {
  CacheView cache;
  CacheRows at;
  const void *c_kv, *k_rope;  // [B][rows][d_c], [B][rows][d_rope]
  const void* w_k;            // null: no norm
  float eps;
  bool turn;         // rotate the keys
  bool own_pos;      // by rope.pos, else by the position itself
  RopeArgs rope;     // tokens, d_rope, layout, positions
  int* status;
};
LaunchResult cache4_append(const CacheAppend& a, const RopeTable& t, cudaStream_t st);

struct CacheRead {
  CacheView cache;
  CacheRows at;
  void *c_kv, *k_rope;
  int* status;
};
LaunchResult cache4_read(const CacheRead& a, cudaStream_t st);

// ---- attention over the cache
//
// The rows of a sequence are its Sq queries times n_h heads, row i n_h + h; an item is a tile of `tile`
// of them. The keys an item's rows see lie in one interval; its key tiles of `keys` and those of all
// items, one after the other, are shared out evenly among `parts` groups of CTAs. An item that one
// part holds whole is written at once; of a split one each part leaves its piece in a slot (2 part if
// it began earlier, 2 part + 1 otherwise), and a second kernel joins the pieces.
struct CacheAttn {
  CacheView cache;
  PageTable pages;
  const int* lengths;  // [B] cached tokens
  const int *key_lo, *key_hi;  // [B][Sq] or null
  int Sq, n_h, rows;   // rows = Sq * n_h
  int tile, row_tiles, keys, parts;
  bool causal;
  float scale;
  ScoreMods mods;
  int* first;    // [items + 1] first key tile of each item in the order of all
  int* part_item;  // [parts] the item in which a part's share begins
  int2* hull;    // [items] keys seen by some row, of those past the table's room the first few
  float* part_o;     // [2 parts][tile][d_c]
  float2* part_ml;   // [2 parts][tile] {running maximum, sum}
  float* lse;        // [B][n_h][Sq]
  int* status;
  __host__ __device__ int items() const { return pages.B * row_tiles; }
};

// CUDA cores, any widths: q_lat and ctx in fp32. The join joins split items (maxima in natural units) and
// fills the rows of empty ones.
constexpr int kSimtRows = 8, kSimtKeys = 32;
LaunchResult cache4_simt_prepare(const CacheAttn& a, bool is_bf16, int d_nope, const void* q, const void* W_UK,
                                 float* q_lat, cudaStream_t st);
LaunchResult cache4_simt_attn(const CacheAttn& a, bool is_bf16, int d_nope, const void* q, const float* q_lat, float* ctx,
                              cudaStream_t st);
LaunchResult cache4_join(const CacheAttn& a, float* ctx, cudaStream_t st);
LaunchResult cache4_simt_out(const CacheAttn& a, bool is_bf16, int d_v, const float* ctx, const void* W_UV, void* out,
                             cudaStream_t st);

// Tensor cores, bf16 with d_c = 512, d_nope = d_v = 128, d_rope = 64: a plan and operands of the queries,
// the attention (maxima in units of log2, whole items' context normalised in fp32), the joining with the
// output's product. A row of `query` is 512 fp16 and 64 bf16, times the power of two whose inverse is
// the row's `up` (NaN: the row's result is).
struct CacheOperands {
  uint8_t* query;  // [B * rows][1152]
  float* up;       // [B * rows]
  float* ctx;      // [B * rows][512]
};
constexpr int kQueryBytes = 1152;
LaunchResult cache4_tc_prepare(const CacheAttn& a, const bf16* q, const bf16* W_UK, const CacheOperands& x, cudaStream_t st);
constexpr int kTcRows = 128, kTcKeys = 64;  // tcgen05
LaunchResult cache4_tc_attn(const CacheAttn& a, const CacheOperands& x, cudaStream_t st);
constexpr int kMmaRows = 16, kMmaKeys = 32;  // mma.sync, for few rows
LaunchResult cache4_mma_attn(const CacheAttn& a, const CacheOperands& x, cudaStream_t st);
LaunchResult cache4_tc_finish(const CacheAttn& a, const CacheOperands& x, const bf16* W_UV, bf16* out, cudaStream_t st);

#ifdef __CUDACC__
// The pool's row of position p of sequence b, or -1 where the table has none.
__device__ __forceinline__ long long cache_slot(const CacheView& c, const PageTable& t, int b, long long p) {
  if (p < 0) return -1;
  const long long k = p / c.page;
  if (k >= t.most) return -1;
  const int id = __ldg(t.table + static_cast<long long>(b) * t.most + k);
  if (id < 0 || id >= c.pages) return -1;
  return static_cast<long long>(id) * c.page + (p - k * c.page);
}

constexpr int kStatusBadPage = 1;  // LAGA_ERR_INVALID_ARG in the device's status word
__device__ __forceinline__ void report_page(int* status, int where) {
  if (status) atomicCAS(status, 0, kStatusBadPage | (where << 8));
}

// The keys [lo, hi) that query i of sequence b sees.
__device__ __forceinline__ int2 cache_row_bounds(const CacheAttn& a, int b, int i) {
  const int len = __ldg(a.lengths + b);
  const long long at = static_cast<long long>(b) * a.Sq + i;
  int lo = a.key_lo ? max(0, __ldg(a.key_lo + at)) : 0;
  int hi = a.key_hi ? min(len, __ldg(a.key_hi + at)) : len;
  if (a.causal) hi = min(hi, len - a.Sq + i + 1);
  return lo < hi ? make_int2(lo, hi) : make_int2(0, 0);
}

// A part's share of all key tiles.
struct CacheShare {
  int quota, begin, end;
};
__device__ __forceinline__ CacheShare cache_share(const CacheAttn& a, int part) {
  const int total = __ldcg(a.first + a.items());
  const int quota = max(1, (total + a.parts - 1) / a.parts);
  const long long begin = static_cast<long long>(part) * quota;
  return CacheShare{quota, static_cast<int>(min(begin, static_cast<long long>(total))),
                    static_cast<int>(min(begin + quota, static_cast<long long>(total)))};
}
// A row's sum of weights at its end: 0 of a row that sees keys (whose scores were all -inf) is NaN.
__device__ __forceinline__ float row_sum(float l, int2 seen) {
  return l == 0.f && seen.x < seen.y ? __int_as_float(0x7fc00000) : l;
}
// The result of a row of an item without key tiles: 0, or NaN where it sees keys, all past the table's room.
__device__ __forceinline__ float lost_row(int2 seen) { return seen.x < seen.y ? __int_as_float(0x7fc00000) : 0.f; }

// One CTA: the items' intervals of keys, and the running sum of their key tiles.
template <int THREADS>
__device__ __forceinline__ void cache4_plan_items(const CacheAttn& a) {
  __shared__ int sums[32];
  const int items = a.items(), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long room = static_cast<long long>(a.pages.most) * a.cache.page;
  int before = 0;
  for (int j0 = 0; j0 < items; j0 += THREADS) {
    const int j = j0 + threadIdx.x;
    int tiles = 0;
    if (j < items) {
      const int b = j / a.row_tiles, r0 = (j - b * a.row_tiles) * a.tile, r1 = min(r0 + a.tile, a.rows) - 1;
      int lo = 0x7fffffff, hi = 0;
      for (int i = r0 / a.n_h; i <= r1 / a.n_h; ++i) {
        const int2 s = cache_row_bounds(a, b, i);
        if (s.x >= s.y) continue;
        lo = min(lo, s.x);
        hi = max(hi, s.y);
      }
      // Keys that the table has no room for: those up to the end of the first one's tile stay in the interval,
      // as keys without a page to the rows that see them (a key past the interval, in its last tile, would pass
      // for one of zeros). A row that sees only others ends without a weight (row_sum), or its whole item
      // without a tile (lost_row).
      if (hi > room) {
        report_page(a.status, 303);
        hi = min(hi, (static_cast<int>(room) / a.keys + 1) * a.keys);
      }
      if (lo >= hi) lo = hi = 0;
      a.hull[j] = make_int2(lo, hi);
      if (lo < hi) tiles = (hi - 1) / a.keys - lo / a.keys + 1;
    }
    int run = tiles;  // inclusive sum over the warp, then over the warps
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, run, m);
      if (lane >= m) run += o;
    }
    if (lane == 31) sums[warp] = run;
    __syncthreads();
    if (warp == 0) {
      int s = lane < THREADS / 32 ? sums[lane] : 0;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, s, m);
        if (lane >= m) s += o;
      }
      sums[lane] = s;
    }
    __syncthreads();
    if (j < items) a.first[j] = before + (warp ? sums[warp - 1] : 0) + run - tiles;
    before += sums[31];
    __syncthreads();
  }
  if (threadIdx.x == 0) a.first[items] = before;
  // the item in which each part's share begins: the last one that begins at or before it
  __syncthreads();
  const int quota = max(1, (before + a.parts - 1) / a.parts);
  for (int p = threadIdx.x; p < a.parts; p += THREADS) {
    const long long t = static_cast<long long>(p) * quota;
    int lo = 0, hi = items;  // first[lo] <= t < first[hi], if t is within them
    while (t < before && hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.first[mid] <= t) lo = mid;
      else hi = mid;
    }
    a.part_item[p] = lo;
  }
}
#endif

}  // namespace laga
