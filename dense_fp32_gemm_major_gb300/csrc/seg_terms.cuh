// seg_terms.cuh -- a result held as two bf16 terms (SegArgs::C, C_lo).
#pragma once

#include <cuda_bf16.h>

namespace gemm {

// The second term of f beside the first, h = bf16(f). Of an infinite h there is
// none: f - h would be NaN, or infinite the other way where f is finite, and
// the sum of the terms' products NaN instead of infinite.
__device__ __forceinline__ __nv_bfloat16 second_term(float f, __nv_bfloat16 h) {
  const float first = static_cast<float>(h);
  return __float2bfloat16_rn(isinf(first) ? 0.0f : f - first);
}

}  // namespace gemm
