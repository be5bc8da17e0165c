// The 8-bit checkpoint format, shared by the kernels that write and read it:
// 32 consecutive elements of a row (the last block may be shorter) share a
// power of two 2^e; element = code 2^e with int8 codes.
//
//   A = the block's largest magnitude
//   e = the least exponent with A < 127.5 2^e, within [-126, 121]
//   code = x / 2^e to nearest, ties to even, clamped to +-127
//
// so a value is off by at most half a unit 2^e <= A / 63.75 (a whole one above
// 127.5 2^121), and code 2^e is exact in bf16 and fp32: an exact product of
// what is read back needs no further rounding.  A block that holds a NaN or an
// infinity has the exponent byte DET_INT8_NAN and reads back as NaN throughout.
#ifndef DETGEMM_INT8_BLOCK_H
#define DETGEMM_INT8_BLOCK_H

#include "rowops.h"

namespace rowops {

constexpr int INT8_BLOCK = 32;

// magnitudes are compared as bit patterns: NaN and inf are above all that is finite
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ bool not_finite(uint32_t m) { return m >= 0x7F800000u; }

// adding 2^16 to the bits carries into the exponent from a significand of
// 1.9921875 = 127.5 / 64 on
__device__ __forceinline__ int block_exponent(uint32_t m) {
  const int e = static_cast<int>((m + 0x10000u) >> 23) - 133;
  return min(max(e, -126), 121);
}
__device__ __forceinline__ float power_of_two(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// the largest of 8 adjacent lanes
__device__ __forceinline__ uint32_t top_of_8(uint32_t m) {
  // lane ^ 1
  m = max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0xB1, 0xF, 0xF, false)));
  // lane ^ 2
  m = max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0x4E, 0xF, 0xF, false)));
  // mirrored in 8
  return max(m, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(m), 0x141, 0xF, 0xF, false)));
}

// four values as codes of the unit 1 / inv, in one word (bad: a block that is not finite)
__device__ __forceinline__ uint32_t codes_of(const float (&v)[4], float inv, bool bad) {
  uint32_t w = 0;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const float k = __builtin_amdgcn_fmed3f(rintf(v[r] * inv), -127.0f, 127.0f);
    w |= (static_cast<uint32_t>(static_cast<int>(k)) & 0xFFu) << (8 * r);
  }
  return bad ? 0u : w;
}
__device__ __forceinline__ void values_of(uint32_t w, float unit, float (&v)[4]) {
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] = static_cast<float>(static_cast<int8_t>(w >> (8 * r))) * unit;
}
// 2^e of an exponent byte, NaN for a block that was not finite
__device__ __forceinline__ float unit_of(int8_t e) { return e == DET_INT8_NAN ? NAN : power_of_two(max<int>(e, -126)); }

// words of four codes that start at any byte
struct __attribute__((packed, aligned(1))) CodeWord {
  uint32_t w;
};
// four codes at p, n of them inside the row
__device__ __forceinline__ void store_codes(int8_t* p, uint32_t w, int n) {
  if (n >= 4) {
    reinterpret_cast<CodeWord*>(p)->w = w;
  } else {
#pragma unroll
    for (int r = 0; r < 3; ++r)
      if (r < n) p[r] = static_cast<int8_t>(w >> (8 * r));
  }
}
__device__ __forceinline__ uint32_t load_codes(const int8_t* p, int n) {
  if (n >= 4) return reinterpret_cast<const CodeWord*>(p)->w;
  uint32_t w = 0;
#pragma unroll
  for (int r = 0; r < 3; ++r)
    if (r < n) w |= static_cast<uint32_t>(static_cast<uint8_t>(p[r])) << (8 * r);
  return w;
}

// The same blocks with fp16 elements, for what is kept in 16 bits: element =
// half 2^e, e the exponent that brings the block's largest finite magnitude into
// [2^14, 2^15).  11 bits each over 29 binades below that (bf16: 8 bits, and the
// gradients that are formed from it would show it), no overflow; infinities and
// NaN stay themselves.
__device__ __forceinline__ uint32_t finite_magnitude(float v) {
  const uint32_t m = magnitude(v);
  return not_finite(m) ? 0u : m;
}
__device__ __forceinline__ int half_exponent(uint32_t m) {
  const int e = static_cast<int>(m >> 23) - 141;
  return max(e, -126);
}
using f16x2 = _Float16 __attribute__((ext_vector_type(2)));
using half_words = uint32_t __attribute__((ext_vector_type(2), aligned(2)));
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, f16x2{static_cast<_Float16>(lo), static_cast<_Float16>(hi)});
}
// four adjacent elements at p, n of them inside the row
__device__ __forceinline__ void store_halves(uint16_t* p, const float (&v)[4], float inv, int n) {
  const half_words w = {pack_half(v[0] * inv, v[1] * inv), pack_half(v[2] * inv, v[3] * inv)};
  if (n >= 4) {
    *reinterpret_cast<half_words*>(p) = w;
  } else {
#pragma unroll
    for (int r = 0; r < 3; ++r)
      if (r < n) p[r] = static_cast<uint16_t>(w[r / 2] >> (16 * (r & 1)));
  }
}
__device__ __forceinline__ void load_halves(const uint16_t* p, float unit, float (&v)[4], int n) {
  half_words w = {0u, 0u};
  if (n >= 4) {
    w = *reinterpret_cast<const half_words*>(p);
  } else {
#pragma unroll
    for (int r = 0; r < 3; ++r)
      if (r < n) w[r / 2] |= static_cast<uint32_t>(p[r]) << (16 * (r & 1));
  }
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const uint32_t word = w[r];           // a bit cast of w[r] itself takes the vector's first element
    const f16x2 h = __builtin_bit_cast(f16x2, word);
    v[2 * r] = static_cast<float>(h[0]) * unit;
    v[2 * r + 1] = static_cast<float>(h[1]) * unit;
  }
}

// four adjacent elements at element i, n of them inside the row (the others 0)
__device__ __forceinline__ void load4(int dt, const void* p, int64_t i, float (&v)[4], int n) {
  if (n >= 4) {
    if (dt == DET_F32) load_vec<DET_F32, 4>(p, i, v);
    else load_vec<DET_BF16, 4>(p, i, v);
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = r < n ? load_elem(dt, p, i + r) : 0.0f;
  }
}
__device__ __forceinline__ void store4(int dt, void* p, int64_t i, const float (&v)[4], int n) {
  if (n >= 4) {
    if (dt == DET_F32) store_vec<DET_F32, 4>(p, i, v);
    else store_vec<DET_BF16, 4>(p, i, v);
  } else {
#pragma unroll
    for (int r = 0; r < 3; ++r)
      if (r < n) store_elem(dt, p, i + r, v[r]);
  }
}

}  // namespace rowops

#endif  // DETGEMM_INT8_BLOCK_H
