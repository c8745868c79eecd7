// Argument checks shared by the C ABI sources: byte ranges and their overlap.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rwkv7_wkv.h"

namespace rwkv7 {

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
  bool empty() const { return hi <= lo; }
};

inline bool overlap(Range x, Range y) { return !x.empty() && !y.empty() && x.lo < y.hi && y.lo < x.hi; }

inline Range range_of(const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, p ? lo + (uintptr_t)bytes : lo};
}

inline bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// Whether an output overlaps an input or another output. `same`: an input that the last output may
// be exactly (an update in place), or null.
inline bool outputs_overlap(const Range* out, int nout, const Range* in, int nin, const Range* same) {
  for (int o = 0; o < nout; ++o) {
    for (int i = 0; i < nin; ++i) {
      const bool in_place = o == nout - 1 && &in[i] == same && in[i].lo == out[o].lo;
      if (!in_place && overlap(out[o], in[i])) return true;
    }
    for (int e = o + 1; e < nout; ++e)
      if (overlap(out[o], out[e])) return true;
  }
  return false;
}

// A launch's status. It may allocate on the host or take a lock; nothing that these throw leaves a C entry point.
template <class Launch>
int status_of(Launch launch) {
  try {
    return launch() == hipSuccess ? RWKV7_OK : RWKV7_ERR_HIP;
  } catch (...) {
    return RWKV7_ERR_HIP;
  }
}

}  // namespace rwkv7
