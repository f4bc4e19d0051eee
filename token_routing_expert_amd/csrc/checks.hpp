// checks.hpp -- host-side argument checks shared by the C entry points.
#pragma once

#include "../../include/moe.h"
#include "common.hpp"

namespace tre {

constexpr int64_t kMaxElems = (int64_t)1 << 31;  // per-array element limit

inline size_t elem_size(moe_dtype dt) { return dt == MOE_F32 ? 4 : 2; }
inline bool dtype_ok(int dt) { return dt == MOE_F32 || dt == MOE_BF16; }
inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

inline moe_status from_hip(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

inline moe_status check_experts(int32_t E) {
  if (E < 1) return MOE_ERR_ARG;
  if (E > kMaxExperts) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

inline moe_status check_width(int32_t n) {
  if (n < 1) return MOE_ERR_ARG;
  if (n % 64 != 0) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace tre

#define TRY(expr)                    \
  do {                               \
    const moe_status st_ = (expr);   \
    if (st_ != MOE_OK) return st_;   \
  } while (0)
