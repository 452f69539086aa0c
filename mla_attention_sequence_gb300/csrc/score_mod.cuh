// Per-score arithmetic of the masked attention kernels, in the log2 domain: with x the raw
// product q . K, a score's exponent is
//   t2 = log2(e) * (cap tanh(scale x / cap) - slope |position - key|)
// without a cap: scale x in place of cap tanh(.); without slopes: no second term.
#pragma once
#include "internal.h"
#include "ptx.cuh"

namespace laga {

struct ModParams {
  float u_scale;        // scale / cap
  float cap_log2;       // cap * log2(e)
  const float* slopes;  // [n_h]
};

inline ModParams mod_params(const Dims& d, const ScoreMods& m) {
  ModParams p{};
  if (m.cap > 0.f) {
    p.u_scale = d.scale / m.cap;
    p.cap_log2 = m.cap * 1.4426950408889634f;
  }
  p.slopes = m.slopes;
  return p;
}

// tanh(u) = 1 - 2 / (1 + e^(2u)), to ~1e-7 absolute: it is multiplied by the cap, so the
// absolute error is the one that counts. e^(2u) = inf gives 1, 0 gives -1.
__device__ __forceinline__ float tanh_abs(float u) {
  return 1.f - __fdividef(2.f, 1.f + ex2_approx(u * 2.8853900817779268f));
}

}  // namespace laga
