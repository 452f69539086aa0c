// Interfaces of the masked attention's preparation, its CUDA-core kernels and the 8-bit
// checkpoints it can read.
#pragma once
#include "internal.h"

#include <cuda_fp8.h>

namespace laga {

// A checkpoint in 8 bits: e4m3 codes [rows][cols] and, per block of 32 columns, one biased
// power-of-two exponent [rows][ceil(cols / 32)]: value = code * 2^(scale - 127).
struct Packed {
  const uint8_t* codes;
  const uint8_t* scales;
};
constexpr int kPackBlock = 32;

#ifdef __CUDACC__
__device__ __forceinline__ float scale_value(uint8_t e) {  // 2^(e - 127); e = 0 is a subnormal
  return __uint_as_float(e == 0 ? 0x00400000u : static_cast<uint32_t>(e) << 23);
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t v) {  // exact
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(v, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Eight values (chunk `c` of the row) as packed bf16, for cols a multiple of 32: exact but for
// values below bf16's normal range.
__device__ __forceinline__ uint4 unpack8_bf16x8(const Packed& p, long long row, int cols, int c) {
  const uint2 v = __ldcg(reinterpret_cast<const uint2*>(p.codes + row * cols + c * 8));
  const float s = scale_value(__ldcg(p.scales + row * (cols / kPackBlock) + (c >> 2)));
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 f = e4m3x2_to_float2(static_cast<uint16_t>((k < 2 ? v.x : v.y) >> (16 * (k & 1))));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
    w[k] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float unpack8_value(const Packed& p, long long row, int cols, int k) {
  const int blocks = (cols + kPackBlock - 1) / kPackBlock;
  return e4m3x2_to_float2(__ldcg(p.codes + row * cols + k)).x * scale_value(__ldcg(p.scales + row * blocks + k / kPackBlock));
}

// Whether one of the keys [lo, hi) has its bit set: words step by step from `from`, every `step`th.
__device__ __forceinline__ bool sees_bad_key(const uint32_t* words, int lo, int hi, int from, int step) {
  if (lo >= hi) return false;
  const int w0 = lo >> 5, w1 = (hi - 1) >> 5;
  for (int w = w0 + from; w <= w1; w += step) {
    uint32_t m = words[w];
    if (w == w0) m &= ~0u << (lo & 31);
    if (w == w1) m &= ~0u >> (31 - ((hi - 1) & 31));
    if (m) return true;
  }
  return false;
}
#endif

// The preparation's part of a masked call's workspace.
struct MaskBuffers {
  int2 *rows, *q_tiles, *q_hull;
  int *kt_count, *kt_list, *q_bad;
  int *seen, *seen_list;  // [B * kt]: whether a key tile is walked; the walked ones, in order
  int* counters;          // {tiles in seen_list, CTAs done, forward ticket}
  int4* work;
  uint32_t* bad;  // [B][ceil(S / 32)] bit per key: its latent row does not count as finite
  char* c_kv;     // [B][S][d_c] with such rows zero, in the inputs' type
  char* k_rope;   // [B][S][d_rope]
  MaskMeta meta() const { return MaskMeta{rows, q_hull, kt_count, kt_list, q_bad, seen, seen_list, counters,
                                             work, counters + 2}; }
};
size_t mask_bytes(const Dims& d, int elem);
MaskBuffers mask_carve(const Dims& d, int elem, char*& p);  // advances p

LaunchResult mask_prepare(const Dims& d, bool is_bf16, const int* key_lo, const int* key_hi, const void* c_kv,
                          const void* k_rope, const MaskBuffers& m, bool key_tiles, cudaStream_t st);
LaunchResult mask_key_bounds(const Dims& d, const int* starts, int n_docs, const int* prefix, int window, int* key_lo,
                             int* key_hi, cudaStream_t st);

// Row statistics of the masked backward (w.lse2, w.delta) and, if some q or dout row is not
// finite, clean copies; with q8 / out8, q and out come from checkpoints and q_clean is written.
// check_q: a non-finite q may have a finite lse (capped scores). beside: the kernel launched just
// before is the rebuild, which writes nothing that this reads.
LaunchResult tc_mask_bwd_pre(const Dims& d, const bf16* q, const bf16* out, const Packed* q8, const Packed* out8,
                             const bf16* dout, const float* lse, const BwdWorkspace& w, bf16* q_clean,
                             bf16* dout_clean, int* q_bad, bool check_q, bool beside, cudaStream_t st);

// ---- CUDA cores, any widths up to 256: fp32 K/V, fp32 arithmetic.
LaunchResult simt_mask_bwd_pre(const Dims& d, bool is_bf16, const void* q, const void* out, const Packed* q8,
                               const Packed* out8, const void* dout, const float* lse, float* lse_row, float* delta,
                               float* q_clean, float* dout_clean, bool beside, cudaStream_t st);
size_t simt_masked_fwd_workspace(const Dims& d, int elem);
size_t simt_masked_bwd_workspace(const Dims& d, int elem);
LaunchResult simt_masked_fwd(const Dims& d, bool is_bf16, const ScoreMods& mods, const int* key_lo, const int* key_hi,
                             const void* q, const void* c_kv, const void* k_rope, const void* W_UK, const void* W_UV,
                             void* out, float* lse, void* ws, cudaStream_t st);
struct BwdGrads {
  void *dq, *dc_kv, *dk_rope, *dW_UK, *dW_UV;
};
LaunchResult simt_masked_bwd(const Dims& d, bool is_bf16, const ScoreMods& mods, const int* key_lo, const int* key_hi,
                             const void* q, const void* c_kv, const void* k_rope, const void* W_UK, const void* W_UV,
                             const void* out, const Packed* q8, const Packed* out8, const float* lse,
                             const void* dout, const BwdGrads& g, void* ws, bool reuse_kv, cudaStream_t st);

}  // namespace laga
