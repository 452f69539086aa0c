// What the C ABI's entry points share: status reporting, argument checks, the choice of
// a path for a descriptor, opt-in timing.
#pragma once
#include "../../include/laga_mla.h"
#include "internal.h"

#include <cstddef>

namespace laga {

// Sets the last error's text (fmt's %s is `detail`) and returns s.
laga_status fail(laga_status s, const char* fmt, const char* detail = nullptr);
laga_status from_launch(const LaunchResult& r);
bool aligned16(const void* p);

void prof_begin(const char* name, cudaStream_t s);
void prof_end(cudaStream_t s);

// Run one launcher between two profiling marks.
template <class F>
LaunchResult timed(const char* name, cudaStream_t s, F&& f) {
  prof_begin(name, s);
  LaunchResult r = f();
  prof_end(s);
  return r;
}

enum class Path { Invalid, Simt, TensorCore, TensorCoreFused };

// Validate the descriptor; fill dims; choose a path. On error, sets *st.
Path plan(const laga_mla_desc* desc, Dims* d, laga_status* st, bool for_bwd);

}  // namespace laga
