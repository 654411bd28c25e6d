// Activations of the linear epilogue, in 32 bits.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/kaio.h"

namespace kaio {

// Forms that neither cancel nor overflow into a NaN for large finite inputs:
// gelu through erfc (1 + erf loses the tail for negative y), the tanh form and
// silu as y times a logistic function, y / (1 + exp(-z)), whose exp overflows
// to infinity and gives -0 there.
template <int ACT>
__device__ __forceinline__ float activation(float y) {
  if constexpr (ACT == KAIO_ACT_RELU) {
    return y < 0.f ? 0.f : y;   // NaN stays NaN
  } else if constexpr (ACT == KAIO_ACT_GELU) {
    return 0.5f * y * erfcf(-0.70710678118654752f * y);
  } else if constexpr (ACT == KAIO_ACT_GELU_TANH) {
    // tanh(u) + 1 = 2 / (1 + exp(-2u)), u = sqrt(2 / pi) (y + 0.044715 y^3)
    return y / (1.f + __expf(-1.5957691216057308f * (y + 0.044715f * y * y * y)));
  } else if constexpr (ACT == KAIO_ACT_SILU) {
    return y / (1.f + __expf(-y));
  } else {
    return y;
  }
}

}  // namespace kaio
