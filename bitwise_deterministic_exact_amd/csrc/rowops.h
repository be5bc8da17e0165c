// Shared device and host helpers of the row kernels (head.hip, norm.hip):
// element loads and stores of any alignment, wave reductions in one fixed
// order, and the argument checks of their C entry points.
#ifndef DETGEMM_ROWOPS_H
#define DETGEMM_ROWOPS_H

#include <hip/hip_runtime.h>

#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include "detgemm.h"

namespace rowops {

// ---------------------------------------------------------------- host side

// det_last_error's buffer of the calling thread (512 bytes, owned by the
// library's first source file): every entry point reports through it.
inline det_status fail(det_status st, const char* fmt, ...) {
  char* const buf = const_cast<char*>(det_last_error());
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, 512, fmt, ap);
  va_end(ap);
  return st;
}

inline det_status hip_check(hipError_t e, const char* what) {
  if (e != hipSuccess) return fail(DET_EHIP, "%s: %s", what, hipGetErrorString(e));
  return DET_OK;
}

inline bool known_dtype(int dt) { return dt == DET_F32 || dt == DET_BF16; }
inline bool aligned_for(const void* p, int dt) {
  return (reinterpret_cast<uintptr_t>(p) & (dt == DET_F32 ? 3u : 1u)) == 0;
}
inline bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---------------------------------------------------------------- elements
//
// A thread moves 16 bytes at a time: VE elements of its type.  The accesses
// carry the element's alignment only, so a row may start anywhere (odd
// vocabularies and widths, sliced views) and the thread-to-element map, and
// with it every sum's order, is the same for every alignment.

template <int DT>
struct Elem;
template <>
struct Elem<DET_F32> {
  static constexpr int VE = 4, BYTES = 4;
};
template <>
struct Elem<DET_BF16> {
  static constexpr int VE = 8, BYTES = 2;
};

// 16 and 8 bytes that start at any element
using u32x4_a2 = uint32_t __attribute__((ext_vector_type(4), aligned(2)));
using u32x4_a4 = uint32_t __attribute__((ext_vector_type(4), aligned(4)));
using u32x2_a2 = uint32_t __attribute__((ext_vector_type(2), aligned(2)));
// NT: data that is read once and is not wanted in the caches
template <bool NT, class T>
__device__ __forceinline__ T load_as(const T* p) {
  if constexpr (NT) return __builtin_nontemporal_load(p);
  else return *p;
}

using bf16x2 = __bf16 __attribute__((ext_vector_type(2)));
using f32x2 = float __attribute__((ext_vector_type(2)));

// two floats rounded (nearest, ties to even) to a pair of bf16
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const f32x2 f = {lo, hi};
  const bf16x2 b = __builtin_convertvector(f, bf16x2);
  return __builtin_bit_cast(uint32_t, b);
}

template <int DT>
__device__ __forceinline__ float load_elem(const void* p, int64_t i) {
  if constexpr (DT == DET_F32) return static_cast<const float*>(p)[i];
  else return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
}
__device__ __forceinline__ float load_elem(int dt, const void* p, int64_t i) {
  return dt == DET_F32 ? load_elem<DET_F32>(p, i) : load_elem<DET_BF16>(p, i);
}
template <int DT>
__device__ __forceinline__ void store_elem(void* p, int64_t i, float v) {
  if constexpr (DT == DET_F32) static_cast<float*>(p)[i] = v;
  else static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(pack_bf16(v, 0.0f));
}
__device__ __forceinline__ void store_elem(int dt, void* p, int64_t i, float v) {
  if (dt == DET_F32) store_elem<DET_F32>(p, i, v);
  else store_elem<DET_BF16>(p, i, v);
}

// W consecutive elements from element i on, W a multiple of a 16-byte access's
// VE or (bf16) half of one
template <int DT, int W, bool NT = false>
__device__ __forceinline__ void load_vec(const void* p, int64_t i, float (&v)[W]) {
  const char* const q = static_cast<const char*>(p) + i * Elem<DT>::BYTES;
  if constexpr (DT == DET_F32) {
#pragma unroll
    for (int j = 0; j < W / 4; ++j) {
      const u32x4_a4 u = load_as<NT>(reinterpret_cast<const u32x4_a4*>(q) + j);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * j + e] = __uint_as_float(u[e]);
    }
  } else if constexpr (W == 4) {
    const u32x2_a2 u = load_as<NT>(reinterpret_cast<const u32x2_a2*>(q));
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      v[2 * e] = __uint_as_float(u[e] << 16);
      v[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < W / 8; ++j) {
      const u32x4_a2 u = load_as<NT>(reinterpret_cast<const u32x4_a2*>(q) + j);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[8 * j + 2 * e] = __uint_as_float(u[e] << 16);
        v[8 * j + 2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
      }
    }
  }
}
template <int DT, int W>
__device__ __forceinline__ void store_vec(void* p, int64_t i, const float (&v)[W]) {
  char* const q = static_cast<char*>(p) + i * Elem<DT>::BYTES;
  if constexpr (DT == DET_F32) {
#pragma unroll
    for (int j = 0; j < W / 4; ++j) {
      u32x4_a4 u;
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = __float_as_uint(v[4 * j + e]);
      *(reinterpret_cast<u32x4_a4*>(q) + j) = u;
    }
  } else if constexpr (W == 4) {
    const u32x2_a2 u = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    *(reinterpret_cast<u32x2_a2*>(q)) = u;
  } else {
#pragma unroll
    for (int j = 0; j < W / 8; ++j) {
      u32x4_a2 u;
#pragma unroll
      for (int e = 0; e < 4; ++e) u[e] = pack_bf16(v[8 * j + 2 * e], v[8 * j + 2 * e + 1]);
      *(reinterpret_cast<u32x4_a2*>(q) + j) = u;
    }
  }
}

// ---------------------------------------------------------------- reductions
//
// Over the 64 lanes of a wave, as the DPP chain row_shr 1, 2, 4, 8,
// row_bcast 15, row_bcast 31: lane 63 ends with the total, read back to a
// scalar.  The chain is one fixed tree, so a sum's bits are fixed.
template <int CTRL>
__device__ __forceinline__ float dpp(float old, float v) {
  return __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
      static_cast<int>(__float_as_uint(old)), static_cast<int>(__float_as_uint(v)), CTRL, 0xF, 0xF, false)));
}
__device__ __forceinline__ float lane63(float v) {
  return __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(__float_as_uint(v)), 63)));
}
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp<0x111>(0.0f, v);
  v += dpp<0x112>(0.0f, v);
  v += dpp<0x114>(0.0f, v);
  v += dpp<0x118>(0.0f, v);
  // row_bcast: lanes without a source add the 0 of `old`
  v += __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(__float_as_uint(v)), 0x142, 0xA, 0xF, false)));
  v += __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(__float_as_uint(v)), 0x143, 0xC, 0xF, false)));
  return lane63(v);
}
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp<0x111>(v, v));
  v = fmaxf(v, dpp<0x112>(v, v));
  v = fmaxf(v, dpp<0x114>(v, v));
  v = fmaxf(v, dpp<0x118>(v, v));
  v = fmaxf(v, dpp<0x142>(v, v));
  v = fmaxf(v, dpp<0x143>(v, v));
  return lane63(v);
}
// in 64 bits, for the few values that join partial results: a butterfly
__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// LDS written by lanes of a wave becomes visible to its other lanes (the LDS
// serves one wave's instructions in order; this keeps the compiler to it)
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

}  // namespace rowops

#endif  // DETGEMM_ROWOPS_H
