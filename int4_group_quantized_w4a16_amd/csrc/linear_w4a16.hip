// W4A16 product with bias, activation and residual in its epilogue:
//
//   y[m, n] = act( sum_k x[m, k] * int4(W, k, n) * S[k / 128, n] + b[n] ) + r[m, n]
//
// The QKV projection's two kernels on one matrix (w4a16_split_k.hpp,
// w4a16_tile.hpp; qkv_decode.hip and qkv_prefill.hip describe them), with the
// sums kept in f32 through the epilogue and rounded once.
//
// Measured, weights from HBM: 8 x 4096 x 4096 with bias and residual 5.0 us
// (a launch is 4); 61 x 11004 x 4096 with silu 14.2 us (22.5 MB of weights are 5
// us): 172 tiles leave 84 compute units idle, and on the others no unit is the
// bound (vector unit 45% busy, LDS 34%, MFMA 27%): the waves wait 43% of their
// cycles for loads and barriers, one four-set tile per compute unit; 2048 x 4096
// x 4096 with everything 62.5 to 65 us by card, 1057 to 1099 TFLOP/s, MFMA and
// vector unit 51% and 52% busy.

#include "w4a16_split_k.hpp"
#include "w4a16_tile.hpp"

namespace kaio {
namespace {

template <int RT, int RSPLIT, int VEC, int WAVES, bool kFull, int XR, bool kTrim, int NG>
__global__ void __launch_bounds__(WAVES * 64, 1) linear_split_k_kernel(LinearProblem p, uint32_t nstrips) {
  w4a16_split_k<4, RT, RSPLIT, VEC, WAVES, kFull, XR, kTrim, NG>(p, nstrips);
}

template <int WAVES, bool kAligned, int BM, int KS, int NQ>
__global__ void __launch_bounds__(KS * WAVES * 64, 1) linear_tile_kernel(LinearProblem p, uint32_t mtiles) {
  w4a16_tile<4, WAVES, 1, kAligned, BM, KS, NQ>(p, mtiles);
}

template <int RT, int RSPLIT, int VEC, int WAVES, int XR>
hipError_t launch_strips(const LinearProblem& p, hipStream_t stream) {
  constexpr uint32_t BN = 16 * VEC;
  const uint32_t nstrips = (p.n + BN - 1) / BN;
  const bool straight = p.k / kGroup == 2 * WAVES / RSPLIT;   // every wave with exactly two groups
#define KAIO_STRIPS(FULL, TRIM)                                                                                \
  hipLaunchKernelGGL((linear_split_k_kernel<RT, RSPLIT, VEC, WAVES, FULL, XR, TRIM, 0>), dim3(nstrips),        \
                     dim3(WAVES * kWave), 0, stream, p, nstrips)
  if constexpr (WAVES == 16) {
    if (!straight && p.n % VEC == 0) {
      if (p.n % BN == 0) KAIO_STRIPS(true, true);
      else KAIO_STRIPS(false, true);
      return hipGetLastError();
    }
  }
  if (p.n % BN == 0) KAIO_STRIPS(true, false);
  else KAIO_STRIPS(false, false);
#undef KAIO_STRIPS
  return hipGetLastError();
}

template <int WAVES, bool kAligned, int BM, int KS, int NQ>
hipError_t launch_tile(const LinearProblem& p, hipStream_t stream) {
  constexpr uint32_t BN = 16 * WAVES * NQ;
  const uint32_t mtiles = (p.m + BM - 1) / BM, ntiles = (p.n + BN - 1) / BN;
  const size_t lds = (size_t)KS * SetRing<4, WAVES, 1, BM, KS, NQ>::kSize * 16;
  auto* kern = &linear_tile_kernel<WAVES, kAligned, BM, KS, NQ>;
  static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL(kern, dim3(mtiles * ntiles), dim3(KS * WAVES * 64), lds, stream, p, mtiles);
  return hipGetLastError();
}
template <int WAVES, int BM, int KS, int NQ>
hipError_t launch_form(const LinearProblem& p, hipStream_t stream) {
  return p.n % 8 == 0 ? launch_tile<WAVES, true, BM, KS, NQ>(p, stream) : launch_tile<WAVES, false, BM, KS, NQ>(p, stream);
}

// k == 0: the product is zero, the epilogue remains
__global__ void __launch_bounds__(256) linear_empty_kernel(LinearProblem p) {
  const uint64_t total = (uint64_t)p.m * p.n;
  for (uint64_t e = (uint64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (uint64_t)gridDim.x * 256)
    p.y[e] = linear_out(p, 0.f, e / p.n, (uint32_t)(e % p.n));
}

// the kernel of a form; every form that linear_form picks is here
hipError_t launch_linear_form(const LinearProblem& p, LinearForm f, hipStream_t stream) {
  constexpr auto strips = [](uint32_t vec, uint32_t waves, uint32_t rows) { return LinearForm{vec, waves, rows, 1, 1}.code(); };
  constexpr auto tile = [](uint32_t waves, uint32_t rows, uint32_t sets, uint32_t blocks) {
    return LinearForm{0, waves, rows, sets, blocks}.code();
  };
  switch (f.code()) {
    case strips(1, 16, 8): return launch_strips<1, 1, 1, 16, 8>(p, stream);
    case strips(2, 16, 8): return launch_strips<1, 1, 2, 16, 8>(p, stream);
    case strips(4, 16, 8): return launch_strips<1, 1, 4, 16, 8>(p, stream);
    case strips(1, 16, 16): return launch_strips<1, 1, 1, 16, 16>(p, stream);
    case strips(2, 16, 16): return launch_strips<1, 1, 2, 16, 16>(p, stream);
    case strips(4, 16, 16): return launch_strips<1, 1, 4, 16, 16>(p, stream);
    case strips(1, 8, 32): return launch_strips<2, 1, 1, 8, 32>(p, stream);
    case strips(2, 8, 32): return launch_strips<2, 1, 2, 8, 32>(p, stream);
    case strips(4, 8, 32): return launch_strips<2, 1, 4, 8, 32>(p, stream);
    case strips(1, 8, 64): return launch_strips<2, 2, 1, 8, 32>(p, stream);
    case strips(2, 8, 64): return launch_strips<2, 2, 2, 8, 32>(p, stream);
    case tile(4, 64, 4, 1): return launch_form<4, 64, 4, 1>(p, stream);
    case tile(4, 64, 2, 1): return launch_form<4, 64, 2, 1>(p, stream);
    case tile(4, 96, 2, 1): return launch_form<4, 96, 2, 1>(p, stream);
    case tile(4, 64, 2, 2): return launch_form<4, 64, 2, 2>(p, stream);
    case tile(4, 96, 2, 2): return launch_form<4, 96, 2, 2>(p, stream);
    case tile(4, 128, 2, 2): return launch_form<4, 128, 2, 2>(p, stream);
    case tile(8, 96, 1, 2): return launch_form<8, 96, 1, 2>(p, stream);
    case tile(8, 128, 1, 2): return launch_form<8, 128, 1, 2>(p, stream);
    case tile(8, 128, 1, 3): return launch_form<8, 128, 1, 3>(p, stream);
    case tile(4, 64, 1, 1): return launch_form<4, 64, 1, 1>(p, stream);
    case tile(4, 64, 1, 2): return launch_form<4, 64, 1, 2>(p, stream);
    case tile(4, 96, 1, 1): return launch_form<4, 96, 1, 1>(p, stream);
    default: break;
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_linear_w4a16(const LinearProblem& p, hipStream_t stream) {
  if (p.k == 0) {
    const uint64_t wgs = ((uint64_t)p.m * p.n + 255) / 256;
    hipLaunchKernelGGL(linear_empty_kernel, dim3((uint32_t)(wgs < 4096 ? wgs : 4096)), dim3(256), 0, stream, p);
    return hipGetLastError();
  }
  return launch_linear_form(p, linear_form(p.m, p.n, p.k), stream);
}

}  // namespace kaio
