// usp_div.cuh -- division by numbers that a launch fixes, by a multiplication (a
// dependent chain of a few steps where the integer division takes tens).
#pragma once

#include <cstdint>

namespace usp {

// n / d for n < 2^31: with m = 2^31 / d rounded up to 32 + shift bits, the
// product's upper part is the quotient.
struct Div {
  uint32_t d, mul, shift;
};
inline Div make_div(uint32_t d) {
  uint32_t shift = 0;
  while ((1ull << shift) < d) ++shift;
  const uint64_t m = ((1ull << (31 + shift)) + d - 1) / d;
  return Div{d, static_cast<uint32_t>(m), shift};
}
__device__ __forceinline__ uint32_t quot(const Div& v, uint32_t n) {
  return static_cast<uint32_t>((static_cast<uint64_t>(n) * v.mul) >> (31 + v.shift));
}

}  // namespace usp
