// Argument checks that the entry points of the operators share (host only).
#pragma once

#include <stdint.h>

#include <hip/hip_runtime_api.h>

#include "../../include/msm.h"

namespace msm {
namespace check {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t align_up(size_t v) { return (v + 255) & ~(size_t)255; }
inline size_t elem_bytes(msm_dtype io) { return io == MSM_BF16 ? 2 : 4; }
inline msm_status status_of(hipError_t e) { return e == hipSuccess ? MSM_OK : MSM_ERR_LAUNCH; }

struct Range {
  uintptr_t lo, hi;
};
inline Range rng(const void* p, size_t bytes) {
  return p ? Range{(uintptr_t)p, (uintptr_t)p + bytes} : Range{0, 0};
}
inline bool overlaps(Range a, Range b) {
  if (a.lo == a.hi || b.lo == b.hi) return false;
  return a.lo < b.hi && b.lo < a.hi;
}
inline bool any_overlap(const Range* outs, int nout, const Range* ins, int nin) {
  for (int i = 0; i < nout; ++i) {
    for (int j = 0; j < nin; ++j)
      if (overlaps(outs[i], ins[j])) return true;
    for (int j = i + 1; j < nout; ++j)
      if (overlaps(outs[i], outs[j])) return true;
  }
  return false;
}
inline bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

}  // namespace check
}  // namespace msm
