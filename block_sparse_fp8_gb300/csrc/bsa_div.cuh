// Division of an index by a number that the host knows: q = floor(n / d) for n < 2^31, from a product's
// upper half (T. Granlund, P. L. Montgomery, "Division by invariant integers using multiplication", PLDI
// 1994).  With s = ceil(log2 d) and m = ceil(2^(32 + s) / d) - 2^32, n (2^32 + m) / 2^(32 + s) lies
// above n / d by less than n / 2^32 / d, less than the distance to the next whole number.
#pragma once

#include <cstdint>

namespace bsa {

struct Divisor {
  uint32_t d, m, s;

  static Divisor of(uint32_t d) {  // d >= 1
    Divisor x;
    x.d = d;
    x.s = 0;
    while ((1ull << x.s) < d) ++x.s;
    x.m = (uint32_t)(((1ull << 32) * ((1ull << x.s) - d)) / d + 1);
    return x;
  }
#ifdef __CUDACC__
  __device__ __forceinline__ uint32_t quotient(uint32_t n) const { return (__umulhi(n, m) + n) >> s; }
#endif
};

}  // namespace bsa
