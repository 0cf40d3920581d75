// fast_div.cuh -- quotients by a divisor that the host knows.
#pragma once

#include <cstdint>

namespace qk {

// n / d for n < 2^31 by a multiplication: 2^p / d rounded up, p = 31 + ceil(log2 d), is
// off by less than 2^(p - 31) / n in the quotient.
struct FastDiv {
  uint32_t m, p;
  int d;
};
inline FastDiv fast_div(int d) {
  uint32_t l = 0;
  while ((1ull << l) < (uint64_t)d) ++l;
  const uint64_t two_p = 1ull << (31 + l);
  return FastDiv{(uint32_t)((two_p + (uint64_t)d - 1) / (uint64_t)d), 31 + l, d};
}
__device__ __forceinline__ int quot(int n, const FastDiv& f) {
  return (int)(((uint64_t)(uint32_t)n * f.m) >> f.p);
}

}  // namespace qk
