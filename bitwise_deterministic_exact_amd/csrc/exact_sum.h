// Exact sums of fp32 and of fp64 values in the digits of the long accumulator,
// and their one rounding: for sums whose terms come in any order, from any split.
#ifndef DETGEMM_EXACT_SUM_H
#define DETGEMM_EXACT_SUM_H

#include "rowops.h"

namespace rowops {

// An fp32 value is sig 2^(e - 150) with e = max(exponent field, 1): it starts
// at bit o = e + 148 of the accumulator (digit 0 weighs 2^-298) and its 24
// bits touch digits o/32 and o/32 + 1, 4..13 of the 18.
constexpr int DIG0 = 4, NDIG = 10;

// the finite value of bits u as one or two digits: add(j, v) for digit DIG0 + j
template <class Add>
__device__ __forceinline__ void add_digits(uint32_t u, Add add) {
  if ((u << 1) == 0u) return;
  const uint32_t ef = (u >> 23) & 0xFFu;
  uint32_t sig = u & 0x7FFFFFu;
  if (ef != 0u) sig |= 0x800000u;
  const uint32_t o = max(ef, 1u) + 148u;
  const uint64_t wide = static_cast<uint64_t>(sig) << (o & 31u);
  int64_t lo = static_cast<int64_t>(wide & 0xFFFFFFFFull), hi = static_cast<int64_t>(wide >> 32);
  if (u >> 31) { lo = -lo; hi = -hi; }
  const int j = static_cast<int>(o >> 5) - DIG0;
  add(j, lo);
  if (hi != 0) add(j + 1, hi);
}

// digits to an fp32 value or a bf16 one (as fp32), rounded once (nearest-even):
// carries first, then the top 24 bits (bf16: 8) with the rest as a sticky bit.
// By way of fp32 a bf16 gradient would be rounded twice: 1 + 2^-8 + 2^-30 to 1.
template <class D>
__device__ __forceinline__ float round_digits(D digit, bool bf16) {
  uint32_t w[NDIG + 1];
  int64_t carry = 0;
#pragma unroll
  for (int j = 0; j < NDIG; ++j) {
    const int64_t v = digit(j) + carry;
    w[j] = static_cast<uint32_t>(v);
    carry = v >> 32;
  }
  const bool neg = carry < 0;
  w[NDIG] = static_cast<uint32_t>(carry);                     // |carry| < 2^31: the sums stay far below 2^62
  if (neg) {
    uint32_t c = 1u;
#pragma unroll
    for (int j = 0; j <= NDIG; ++j) {
      const uint32_t v = ~w[j] + c;
      c = (c != 0u && v == 0u) ? 1u : 0u;
      w[j] = v;
    }
  }
  int top = -1;
  uint32_t hi = 0u, lo = 0u;                                  // the highest nonzero word and the one below it
#pragma unroll
  for (int j = 0; j <= NDIG; ++j)
    if (w[j] != 0u) {
      top = j;
      hi = w[j];
      lo = j > 0 ? w[j > 0 ? j - 1 : 0] : 0u;
    }
  bool sticky = false;                                        // any bit below those two
#pragma unroll
  for (int j = 0; j <= NDIG; ++j)
    if (j < top - 1 && w[j] != 0u) sticky = true;
  if (top < 0) return 0.0f;
  uint64_t win = (static_cast<uint64_t>(hi) << 32) | lo;      // its bit 0 weighs 2^(32 (DIG0 + top - 1) - 298)
  int q = 32 * (DIG0 + top - 1) - 298;
  const int n = 64 - __builtin_clzll(win);                    // n >= 33
  // the bits below the kept ones; subnormal results keep 2^-149 (bf16: 2^-133)
  const int cut = bf16 ? max(n - 8, -133 - q) : max(n - 24, -149 - q);
  if (cut > 64) return neg ? -0.0f : 0.0f;                    // bf16, top = 0: 69, and less than 2^-138
  if (cut > 0) {
    const uint64_t rest = win & ((1ull << cut) - 1ull), half = 1ull << (cut - 1);
    win >>= cut;
    q += cut;
    if (rest > half || (rest == half && (sticky || (win & 1ull)))) win += 1ull;
  }
  const float mag = ldexpf(static_cast<float>(static_cast<uint32_t>(win)), q);
  return neg ? -mag : mag;
}

// The same for a finite fp64 value below 2^152, a sum of up to 2^24 fp32 values:
// two or three digits; what lies below 2^-170, digit 0's unit, is cut off.  The
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
