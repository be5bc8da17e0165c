// Elementary functions that several kernels share.
#ifndef DETGEMM_ELEMENTARY_H
#define DETGEMM_ELEMENTARY_H

#include "rowops.h"

#pragma clang fp contract(off)

namespace rowops {

// e^x to about 2 units: the product with log2 e is carried in two parts, or its
// rounding would cost |x| units.  Of a NaN: 0; its callers keep the NaN.
__device__ __forceinline__ float exp_of(float x) {
  x = __builtin_amdgcn_fmed3f(x, -200.0f, 200.0f);            // e^+-200 is inf or 0 in 32 bits all the same
  const float hi = x * 1.44269502f;
  const float lo = fmaf(x, 1.92596299e-8f, fmaf(x, 1.44269502f, -hi));
  const float e = __builtin_amdgcn_exp2f(hi);
  return e == INFINITY ? e : fmaf(e, lo * 0.693147182f, e);
}

}  // namespace rowops

#endif  // DETGEMM_ELEMENTARY_H
