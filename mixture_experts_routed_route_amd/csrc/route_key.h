// Order of router logits, shared by the kernels that choose experts.
#pragma once

#include "moe_internal.h"

namespace moe {

// Order-preserving map of a float onto uint32: larger float -> larger key.
// +0 and -0 map to one key; NaN maps to 0, below -inf (0x007FFFFF).
__device__ __forceinline__ uint32_t order_key(float f) {
  uint32_t b = __float_as_uint(f);
  if ((b & 0x7FFFFFFFu) == 0u) b = 0u;
  if ((b & 0x7F800000u) == 0x7F800000u && (b & 0x007FFFFFu)) return 0u;
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k) {
  uint32_t b = (k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k;
  return __uint_as_float(b);
}

}  // namespace moe
