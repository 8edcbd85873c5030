// Argument checks that the C entry points of the operators around the layer share.
#pragma once
#include "common.h"

namespace moe {

// Workgroups times threads of a launch stay below 2^32.
constexpr int64_t kMaxTokens = 4194303;

inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool need(const void* p, size_t n) { return p && aligned_to(p, n); }

inline moe_status check_scratch(const void* ws, size_t bytes, size_t required) {
  if (required && (!ws || bytes < required)) return MOE_EWORKSPACE;
  return aligned_to(ws, 16) ? MOE_OK : MOE_EINVAL;
}

inline moe_status done(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_EHIP; }

}  // namespace moe

#define MOE_TRY(expr)              \
  do {                             \
    moe_status st_ = (expr);       \
    if (st_ != MOE_OK) return st_; \
  } while (0)
