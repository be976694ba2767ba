// abi_checks.h -- what the host sides of the training operators and of the residual block check arguments with.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../../include/ssm_scan.h"

namespace ssm {
namespace abi {

constexpr int64_t kMaxSize = int64_t(1) << 40;
constexpr int64_t kMaxElems = int64_t(1) << 61;
constexpr int64_t kMaxGrid = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxBlocks = (int64_t(1) << 24) - 1;  // of 256 threads, in a launch of one dimension

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

inline Range span(const void* p, int64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Range{a, p ? a + static_cast<uintptr_t>(bytes) : a};
}

inline bool overlaps(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

inline bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

inline bool mul_ok(int64_t a, int64_t b, int64_t* out) {
  if (a <= 0 || b <= 0 || a > kMaxElems / b) return false;
  *out = a * b;
  return true;
}

inline bool dtype_ok(int32_t t) { return t == SSM_F32 || t == SSM_BF16; }
inline int64_t dtype_size(int32_t t) { return t == SSM_BF16 ? 2 : 4; }

inline ssm_status launch_status(hipError_t e) { return e == hipSuccess ? SSM_OK : SSM_ERR_LAUNCH; }

// any of the outputs over an input or another output
inline bool any_overlap(const Range* outs, size_t nout, const Range* ins, size_t nin) {
  for (size_t i = 0; i < nout; ++i) {
    for (size_t j = 0; j < nin; ++j)
      if (overlaps(outs[i], ins[j])) return true;
    for (size_t j = i + 1; j < nout; ++j)
      if (overlaps(outs[i], outs[j])) return true;
  }
  return false;
}

}  // namespace abi
}  // namespace ssm
