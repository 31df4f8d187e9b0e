// Host helpers shared by the library's C ABI sources (pool.cpp, step.cpp,
// weight.cpp, kvs_mask.cpp, train.cpp).
#pragma once

#include <cmath>

#include "../../include/leyline.h"

namespace ll {

// Record a message for ll_last_error() on the calling thread; returns s.
ll_status fail(ll_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
const char* last_error();

// The scale of an attention's scores, and the cap that bounds them (0: none).  The
// kernels keep scores in base 2 and work out the tanh of scale / cap times a product,
// so both stay far from the ends of float32.
inline ll_status check_scale(float scale, float cap) {
  if (!std::isfinite(scale * 1.4426950408889634f)) return fail(LL_EINVAL, "scale, times log2 e, is not finite");
  if (cap == 0.f) return LL_OK;
  if (!(cap >= 0x1p-40f && cap <= 0x1p40f)) return fail(LL_EINVAL, "cap must be 0 or lie in [2^-40, 2^40]");
  const float ratio = std::fabs(scale / cap);
  if (scale != 0.f && !(ratio >= 0x1p-64f && ratio <= 0x1p64f))
    return fail(LL_EINVAL, "scale must be 0 or lie in [cap * 2^-64, cap * 2^64]");
  return LL_OK;
}

}  // namespace ll
