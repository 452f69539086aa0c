// Interface of the rotary positions' kernels, alone and with the norms before them.
#pragma once
#include "internal.h"

namespace laga {

constexpr int kRopePairs = 128;  // most rotated pairs (d_rope <= 256)
constexpr int kNormWidth = 1024;  // widest normed head

struct RopeTable {
  uint64_t turns[kRopePairs];  // pair i: turns per position step, as a fraction of 2^64
  uint8_t axis[kRopePairs];    // pair i turns with this axis' position
};

struct RopeArgs {
  long long tokens;  // B * S rows of q, k_rope and of each axis of pos
  int n_h, d_nope, d_rope;
  bool interleaved, inverse, pos64, is_bf16;
  const void* pos;  // [axes][tokens], int32 or int64
  const void *q, *k;  // [tokens][n_h][d_nope + d_rope], [tokens][d_rope]; either may be null
  void *q_out, *k_out;
};

LaunchResult rope(const RopeArgs& a, const RopeTable& table, cudaStream_t st);

// Norms and rotation: a.q, a.k the rows before the norm; a.q_out, a.k_out the results.
struct NormArgs {
  RopeArgs rope;
  float eps;
  const void *w_q, *w_k;  // [d_nope + d_rope], [d_rope]
  // backward: the gradients of the results; rope.q_out, rope.k_out are then those of the rows
  const void *z_q, *z_k;
  void *dw_q, *dw_k;
  float* partials;  // norm_rope_bwd_partials(..) values of scratch
};
LaunchResult norm_rope(const NormArgs& a, const RopeTable& table, cudaStream_t st);
LaunchResult norm_rope_bwd(const NormArgs& a, const RopeTable& table, cudaStream_t st);
size_t norm_rope_bwd_partials(const RopeArgs& a);

}  // namespace laga
