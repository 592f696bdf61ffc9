// The division of slots by x_row_div, set on the host.
#pragma once

#include <stdint.h>

namespace moe {

// With l = ceil(log2 d) and m = ceil(2^(31+l) / d), floor(s / d) = (s m) >> (31 + l)
// (Granlund and Montgomery, 1994, Theorem 4.2 with N = 31).
inline void lora_set_division(int32_t d, uint32_t& magic, int32_t& shift) {
  int l = 0;
  while (((int64_t)1 << l) < d) ++l;
  magic = (uint32_t)((((uint64_t)1 << (31 + l)) + (uint64_t)d - 1) / (uint64_t)d);
  shift = 31 + l;
}

}  // namespace moe
