// Integer division by numbers that the host knows.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace w4a4 {

// Division by a number fixed for a launch: m = floor(2^32 / d) + 1 gives the
// quotient or one more (2^32 - 1 for d = 1: or one less).
struct Divisor {
  uint32_t d, m;
};
inline Divisor divisor(int64_t d) {
  return {(uint32_t)d, d == 1 ? 0xFFFFFFFFu : (uint32_t)((1ull << 32) / (uint64_t)d + 1)};
}
__device__ __forceinline__ int div_by(int x, const Divisor& v, int& rem) {
  int q = (int)__umulhi((uint32_t)x, v.m), r = x - q * (int)v.d;
  if (r < 0) --q, r += (int)v.d;
  if (r >= (int)v.d) ++q, r -= (int)v.d;
  rem = r;
  return q;
}

}  // namespace w4a4
