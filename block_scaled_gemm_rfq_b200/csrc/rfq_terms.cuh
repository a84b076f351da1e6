// rfq_terms.cuh -- an fp32 number as a sum of bf16 terms (8 bits each), as the adapters' second products take it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace rfq {

// The leading bf16 term of v, taken off it.  What rounds past bf16's range is cut off instead (the next term has the
// rest), and an infinite v is one infinite term: as inf - inf the rest would be NaN, and so would every sum with it.
__device__ __forceinline__ __nv_bfloat16 take_term(float& v) {
  float f = __bfloat162float(__float2bfloat16_rn(v));
  if (isinf(f)) f = __uint_as_float(__float_as_uint(v) & 0xffff0000u);
  v = f == v ? 0.f : v - f;
  return __float2bfloat16_rn(f);
}

}  // namespace rfq
