// Division by a number that the host knows.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace seedlm {

// x / d for 0 <= x < 2^31, with 2^(L-1) < d <= 2^L: ceil(2^(31+L) / d) is less
// than 1 above 2^(31+L) / d, so the product is less than x / 2^(31+L) < 2^-L
// above x / d.  That is at most 1/d, which no quotient's fraction lacks less
// than to the next whole number, so the floor is the quotient's.
struct Divisor {
  uint32_t mul, shift;
  __device__ uint32_t of(uint32_t x) const { return (uint32_t)(((uint64_t)x * mul) >> shift); }
};
inline Divisor divisor(uint32_t d) {
  uint32_t L = 0;
  while (((uint64_t)1 << L) < d) ++L;
  return {(uint32_t)((((uint64_t)1 << (31 + L)) + d - 1) / d), 31 + L};
}

}  // namespace seedlm
