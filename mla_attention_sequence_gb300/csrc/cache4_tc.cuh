// What the two tensor-core forms of the attention over the 4-bit cache share: the walk over a part's
// key tiles, the expansion of codes, the softmax's constants.
#pragma once
#include "cache4.h"
#include "score_mod.cuh"

#include <cuda_fp16.h>

namespace laga {

using ll = long long;
constexpr float LIFT = 6.f, SLACK = 8.f;  // weights: the maximum's 2^6 when m is set, up to 2^14 before m is moved

// One part's piece of an item: its key tiles, in the order of the walk.
struct Piece {
  int item, b, r0, rows, tiles, key0;
  int2 hull;
  bool begins, ends;
};
template <int ROWS, int KEYS>
struct Walk {
  const CacheAttn& a;
  CacheShare share;
  int t, item;
  __device__ __forceinline__ Walk(const CacheAttn& a_, int part) : a(a_), share(cache_share(a_, part)) {
    t = share.begin;
    item = __ldcg(a.part_item + part) - 1;
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
    p.r0 = (item - p.b * a.row_tiles) * ROWS;
    p.rows = min(ROWS, a.rows - p.r0);
    p.hull = __ldcg(a.hull + item);
    p.key0 = (p.hull.x / KEYS + (t - begin)) * KEYS;
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
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// 2^-e brings a row's largest size to between 2^8 and 2^9 (within what a power of two can).
__device__ __forceinline__ int row_exponent(float top) {
  return min(max(static_cast<int>(__float_as_uint(top) >> 23) - 127 - 8, -118), 118);
}
// Eight bf16 values, all finite (0 times an infinity or a NaN is a NaN).
__device__ __forceinline__ bool finite4(uint2 v) {
  return (times_zero_plus_bf16x2(v.y, times_zero_plus_bf16x2(v.x, 0u)) & 0x7fff7fffu) == 0;
}
__device__ __forceinline__ bool finite8(uint4 v) {
  uint32_t z = times_zero_plus_bf16x2(v.x, 0u);
  z = times_zero_plus_bf16x2(v.y, z);
  z = times_zero_plus_bf16x2(v.z, z);
  z = times_zero_plus_bf16x2(v.w, z);
  return (z & 0x7fff7fffu) == 0;
}
__device__ __forceinline__ uint4 ldg4(const void* p) { return __ldcg(static_cast<const uint4*>(p)); }
// A warp's wait for a phase, all lanes together: the phase that is over costs a test and a vote. (One
// lane waiting for the others costs two more convergence points and their taken branches; the waits of
// a warp that comes by once a tile took hundreds of cycles then, even for phases long over.)
__device__ __forceinline__ bool pass(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int where) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  const unsigned long long t0 = global_ns();
  for (uint32_t it = 1;; ++it) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if ((it & 63u) == 0) {
      const bool late = global_ns() - t0 > kWaitLimitNs;
      if (__any_sync(0xffffffffu, late || *abort_flag != 0)) {
        if (late) *abort_flag = kStatusTimeout | (where << 8);
        __syncwarp();
        return false;
      }
    }
  }
}

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
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, m));
  return v;
}

}  // namespace laga
