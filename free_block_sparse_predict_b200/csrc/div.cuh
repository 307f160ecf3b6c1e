// Division by a number that the host knows, as a multiply.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace sparge {

// n / d = umulhi(n, mul) >> shift
// for n < 2^31 (Granlund and Montgomery's round-up method, 32 + 1 bits of
// precision for a 31-bit numerator).
struct Div {
  uint32_t d, mul, shift;
  __device__ __forceinline__ int32_t quot(int32_t n) const {
    return d == 1 ? n : int32_t(__umulhi(uint32_t(n), mul) >> shift);
  }
};
inline Div make_div(uint32_t d) {
  Div x{d, 0, 0};
  if (d > 1) {
    uint32_t log = 0;
    while ((uint64_t(1) << log) < d) ++log;  // ceil(log2 d)
    x.shift = log - 1;
    x.mul = uint32_t(((uint64_t(1) << (31 + log)) + d - 1) / d);
  }
  return x;
}

}  // namespace sparge
