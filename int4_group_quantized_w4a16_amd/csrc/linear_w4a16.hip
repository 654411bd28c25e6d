// W4A16 product with bias, activation and residual in its epilogue.
//
//   y[m, n] = act( sum_k x[m, k] * int4(W, k, n) * S[k / 128, n] + b[n] ) + r[m, n]
//
// One wave per 16 x 16 tile of y: per group of 128 k four MFMAs over exact
// integers into a fresh partial, then acc += partial * scale, as in the QKV
// kernels.

#include "common.hpp"
#include "epilogue.hpp"
#include "launch.hpp"

namespace kaio {
namespace {

template <int ACT>
__global__ void __launch_bounds__(64) linear_w4a16_kernel(LinearProblem p, uint32_t ntiles) {
  const uint32_t lane = threadIdx.x, kb = lane >> 4, l16 = lane & 15;
  const uint32_t m0 = blockIdx.x / ntiles * 16, n0 = blockIdx.x % ntiles * 16;
  const uint32_t row = m0 + l16 < p.m ? m0 + l16 : p.m - 1, col = n0 + l16 < p.n ? n0 + l16 : p.n - 1;
  floatx4 acc = {0.f, 0.f, 0.f, 0.f};
  for (uint32_t g = 0; g < p.k / kGroup; ++g) {
    floatx4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      const half8_t a = *reinterpret_cast<const half8_t*>(p.x + (size_t)row * p.k + g * kGroup + ks * 32 + kb * 8);
      part = mfma16x16x32(a, unpack_int4x8(p.w[((size_t)g * 16 + ks * 4 + kb) * p.n + col]), part);
    }
    const float s = h2f(p.s[(size_t)g * p.n + col]);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = __builtin_fmaf(part[i], s, acc[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t r = m0 + 4 * kb + i;
    if (r < p.m && n0 + l16 < p.n) {
      const size_t at = (size_t)r * p.n + n0 + l16;
      float y = acc[i] + (p.bias ? h2f(p.bias[n0 + l16]) : 0.f);
      y = activation<ACT>(y);
      if (p.residual) y += h2f(p.residual[at]);
      p.y[at] = __builtin_bit_cast(uint16_t, (_Float16)y);
    }
  }
}

template <int ACT>
hipError_t launch(const LinearProblem& p, hipStream_t stream) {
  const uint32_t ntiles = (p.n + 15) / 16;
  hipLaunchKernelGGL((linear_w4a16_kernel<ACT>), dim3((p.m + 15) / 16 * ntiles), dim3(64), 0, stream, p, ntiles);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_w4a16(const LinearProblem& p, hipStream_t stream) {
  switch (p.act) {
    case KAIO_ACT_NONE: return launch<KAIO_ACT_NONE>(p, stream);
    case KAIO_ACT_RELU: return launch<KAIO_ACT_RELU>(p, stream);
    case KAIO_ACT_GELU: return launch<KAIO_ACT_GELU>(p, stream);
    case KAIO_ACT_GELU_TANH: return launch<KAIO_ACT_GELU_TANH>(p, stream);
    case KAIO_ACT_SILU: return launch<KAIO_ACT_SILU>(p, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace kaio
