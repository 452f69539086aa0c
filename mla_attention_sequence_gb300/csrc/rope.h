// Interface of the rotary positions' kernel.
#pragma once
#include "internal.h"

namespace laga {

constexpr int kRopePairs = 128;  // most rotated pairs (d_rope <= 256)

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

}  // namespace laga
