// Exact sums of fp64 values in digits of the long accumulator, for sums whose
// terms come in any order, from any split.
#ifndef DETGEMM_EXACT_SUM_H
#define DETGEMM_EXACT_SUM_H

#include "rowops.h"

namespace rowops {

// Digit 0 of NDIG weighs 2^-170 (digit 4 of the long accumulator, 2^(32 DIG0 - 298)).
constexpr int DIG0 = 4, NDIG = 10;

// A finite fp64 value below 2^152 (a sum of up to 2^24 fp32 values) as two or three
// digits: add(j, v) for digit j; what lies below digit 0's unit is cut off.  The
// top digit (2^118) takes all that is above it, up to 2^34 a value, so that
// 2^22 values stay far below 2^62.
template <class Add>
__device__ __forceinline__ void add_digits(double v, Add add) {
  const uint64_t u = static_cast<uint64_t>(__double_as_longlong(v));
  const int ef = static_cast<int>(u >> 52) & 0x7FF;
  uint64_t sig = u & ((1ull << 52) - 1ull);
  if (ef != 0) sig |= 1ull << 52;
  int o = max(ef, 1) - 1075 + 298 - 32 * DIG0;                // the bit of digit 0 that sig starts at
  if (o < 0) {
    sig = o > -64 ? sig >> -o : 0ull;
    o = 0;
  }
  if (sig == 0ull) return;
  const int s = o & 31, j = o >> 5;
  const uint64_t low = sig << s, high = s > 0 ? sig >> (64 - s) : 0ull;
  int64_t d0 = static_cast<int64_t>(low & 0xFFFFFFFFull), d1 = static_cast<int64_t>(low >> 32);
  int64_t d2 = static_cast<int64_t>(high);
  if (j + 2 >= NDIG) {
    d1 |= d2 << 32;
    d2 = 0;
  }
  if (u >> 63) { d0 = -d0; d1 = -d1; d2 = -d2; }
  add(j, d0);
  add(j + 1, d1);
  if (d2 != 0) add(j + 2, d2);
}

// digits to an fp64 value: the top three words, 65 bits or more, each of the two
// steps rounded to 53
template <class D>
__device__ __forceinline__ double sum_of_digits(D digit) {
  uint32_t w[NDIG + 1];
  int64_t carry = 0;
#pragma unroll
  for (int j = 0; j < NDIG; ++j) {
    const int64_t v = digit(j) + carry;
    w[j] = static_cast<uint32_t>(v);
    carry = v >> 32;
  }
  const bool neg = carry < 0;
  w[NDIG] = static_cast<uint32_t>(carry);                     // |carry| < 2^31
  if (neg) {
    uint32_t c = 1u;
#pragma unroll
    for (int j = 0; j <= NDIG; ++j) {
      const uint32_t v = ~w[j] + c;
      c = (c != 0u && v == 0u) ? 1u : 0u;
      w[j] = v;
    }
  }
  int top = 0;
  uint32_t a = 0u, b = 0u, c = 0u;                            // the highest nonzero word and the two below it
#pragma unroll
  for (int j = 0; j <= NDIG; ++j)
    if (w[j] != 0u) {
      top = j;
      a = w[j];
      b = j > 0 ? w[j > 0 ? j - 1 : 0] : 0u;
      c = j > 1 ? w[j > 1 ? j - 2 : 0] : 0u;
    }
  const double two = static_cast<double>((static_cast<uint64_t>(a) << 32) | b);
  const double mag = ldexp(fma(two, 4294967296.0, static_cast<double>(c)), 32 * (DIG0 + top - 2) - 298);
  return neg ? -mag : mag;
}

}  // namespace rowops

#endif  // DETGEMM_EXACT_SUM_H
