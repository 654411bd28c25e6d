// Product in 8-bit integers with a scale for each token and each channel:
//
//   y[i, j] = act( xs[i] ws[j] sum_k xq[i, k] wq[j, k] + b[j] ) + r[i, j]
//
// Both operands hold 16 consecutive k per lane of a 16x16x64 i8 MFMA, so both
// are read as they lie, [index][k].  Sums are exact in i32 (k < 2^17).

#include "common.hpp"
#include "epilogue.hpp"
#include "launch.hpp"
#include "paged.hpp"

namespace kaio {
namespace {

typedef int intx4 __attribute__((ext_vector_type(4)));

// one output from its integer sum
template <bool kBf16>
__device__ __forceinline__ uint16_t output(const Linear8& p, int acc, uint32_t row, uint32_t col) {
  // the channel's scale first: what is left out of range then is out of range in the result
  float y[1] = {(float)acc * p.ws[col] * p.xs[row]};
  if (p.bias) y[0] += to_f32<kBf16>(p.bias[col]);
  activations<1>(y, p.act);
  if (p.residual) y[0] += to_f32<kBf16>(p.residual[(size_t)row * p.n + col]);
  return from_f32<kBf16>(y[0]);
}

// 64 x 64 outputs per workgroup, 32 x 32 per wave, operands straight from memory.
template <bool kBf16>
__global__ void __launch_bounds__(256) linear8_plain_kernel(Linear8 p, uint32_t mtiles) {
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l16 = lane & 15, kq = lane >> 4;
  const uint32_t m0 = blockIdx.x % mtiles * 64 + (wave & 1) * 32, n0 = blockIdx.x / mtiles * 64 + (wave >> 1) * 32;
  const int8_t *a[2], *b[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t r = m0 + 16 * i + l16, c = n0 + 16 * i + l16;
    a[i] = p.x + (size_t)(r < p.m ? r : p.m - 1) * p.k;
    b[i] = p.w + (size_t)(c < p.n ? c : p.n - 1) * p.k;
  }
  intx4 acc[2][2] = {};
  for (uint32_t k = 16 * kq; k - 16 * kq < p.k; k += 64) {
    intx4 va[2] = {}, vb[2] = {};
    if (k < p.k)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        va[i] = *reinterpret_cast<const intx4*>(a[i] + k);
        vb[i] = *reinterpret_cast<const intx4*>(b[i] + k);
      }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(va[i], vb[j], acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t row = m0 + 16 * i + 4 * kq + e, col = n0 + 16 * j + l16;
        if (row < p.m && col < p.n) p.y[(size_t)row * p.n + col] = output<kBf16>(p, acc[i][j][e], row, col);
      }
}

}  // namespace

hipError_t launch_linear_w8a8(const Linear8& p, hipStream_t stream) {
  const uint32_t mtiles = (p.m + 63) / 64, ntiles = (p.n + 63) / 64;
  if (p.bf16) hipLaunchKernelGGL(linear8_plain_kernel<true>, dim3(mtiles * ntiles), dim3(256), 0, stream, p, mtiles);
  else hipLaunchKernelGGL(linear8_plain_kernel<false>, dim3(mtiles * ntiles), dim3(256), 0, stream, p, mtiles);
  return hipGetLastError();
}

}  // namespace kaio
