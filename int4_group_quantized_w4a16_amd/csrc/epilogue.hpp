// The epilogue of the linear product: bias, activation and residual in 32
// bits, then one rounding to f16.
#pragma once

#include <hip/hip_runtime.h>

#include "common.hpp"
#include "launch.hpp"

namespace kaio {

// Forms that neither cancel nor overflow into a NaN for large finite inputs:
// gelu through erfc (1 + erf loses the tail for negative y), the tanh form and
// silu as y times a logistic function, y / (1 + exp(-z)), whose exp overflows
// to infinity and gives -0 there.
// The logistic's reciprocal is the hardware's (1 step of f32 off at most).
template <int N>
__device__ __forceinline__ void activations(float (&y)[N], int act) {   // act: wave-uniform
  if (act == KAIO_ACT_RELU) {
#pragma unroll
    for (int e = 0; e < N; ++e) y[e] = y[e] < 0.f ? 0.f : y[e];   // NaN stays NaN
  } else if (act == KAIO_ACT_GELU) {
#pragma unroll
    for (int e = 0; e < N; ++e) y[e] = 0.5f * y[e] * erfcf(-0.70710678118654752f * y[e]);
  } else if (act == KAIO_ACT_GELU_TANH) {
    // tanh(u) + 1 = 2 / (1 + exp(-2u)), u = sqrt(2 / pi) (y + 0.044715 y^3)
#pragma unroll
    for (int e = 0; e < N; ++e)
      y[e] *= __builtin_amdgcn_rcpf(1.f + __expf(-1.5957691216057308f * (y[e] + 0.044715f * y[e] * y[e] * y[e])));
  } else if (act == KAIO_ACT_SILU) {
#pragma unroll
    for (int e = 0; e < N; ++e) y[e] *= __builtin_amdgcn_rcpf(1.f + __expf(-y[e]));
  }
}

__device__ __forceinline__ uint16_t linear_out(const LinearProblem& p, float y, size_t row, uint32_t col) {
  float v[1] = {y + (p.bias ? h2f(p.bias[col]) : 0.f)};
  activations<1>(v, p.act);
  if (p.residual) v[0] += h2f(p.residual[row * p.n + col]);
  return __builtin_bit_cast(uint16_t, (_Float16)v[0]);
}

// Stores a BM x BN f32 tile (LDS, row stride BN, column c of row r at
// place(r, c), which keeps 8-column chunks together) at (m0, n0) of y, with TT
// threads.
// In 16-byte chunks of 8 columns, whose bias and residual are loaded ahead.
// Where n % 8 != 0 a chunk starts at any even address (which global accesses
// may), and the last one of a row goes element by element.
template <bool kAligned, int BM, int BN, int TT>
struct LinearChunks {
  static constexpr int CPR = BN / 8, NCH = BM * CPR, PER = (NCH + TT - 1) / TT;
  half8_t bias[PER], residual[PER];
  static __device__ __forceinline__ half8_t fetch(const uint16_t* src) {
    half8_t v;
    __builtin_memcpy(&v, __builtin_assume_aligned(src, kAligned ? 16 : 2), 16);
    return v;
  }
  // one row's chunk; short: fewer than 8 columns are left of n
  static __device__ __forceinline__ half8_t row_chunk(const uint16_t* row, uint32_t gc, uint32_t n) {
    if (kAligned || gc + 8 <= n) return fetch(row + gc);
    half8_t v = {};
#pragma unroll
    for (int e = 0; e < 7; ++e)
      if (gc + e < n) v[e] = __builtin_bit_cast(_Float16, row[gc + e]);
    return v;
  }
  __device__ __forceinline__ void load(const LinearProblem& p, uint32_t m0, uint32_t n0, uint32_t tid) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t c = i * TT + tid, row = c / CPR, last = kAligned ? p.n - 8 : p.n - 1;
      const uint32_t gr = m0 + row < p.m ? m0 + row : p.m - 1, gc = n0 + c % CPR * 8 < p.n ? n0 + c % CPR * 8 : last;
      bias[i] = residual[i] = half8_t{};
      if (p.bias) bias[i] = row_chunk(p.bias, gc, p.n);
      if (p.residual) residual[i] = row_chunk(p.residual + (size_t)gr * p.n, gc, p.n);
    }
  }
  template <typename Place>
  __device__ __forceinline__ void store(const LinearProblem& p, const float* tile, uint32_t m0, uint32_t n0,
                                        uint32_t tid, Place place) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint32_t c = i * TT + tid, row = c / CPR, cc = c % CPR * 8;
      const uint32_t gr = m0 + row, gc = n0 + cc;
      if ((NCH % TT != 0 && c >= (uint32_t)NCH) || gr >= p.m || gc >= p.n) continue;
      const float* const src = tile + row * BN + place(row, cc);
      const floatx4 lo = *reinterpret_cast<const floatx4*>(src), hi = *reinterpret_cast<const floatx4*>(src + 4);
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = (e < 4 ? lo[e & 3] : hi[e & 3]) + (float)bias[i][e];
      activations<8>(y, p.act);
      half8_t o;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = (_Float16)(y[e] + (float)residual[i][e]);
      uint16_t* const dst = p.y + (size_t)gr * p.n + gc;
      if (kAligned || gc + 8 <= p.n) {
        __builtin_memcpy(__builtin_assume_aligned(dst, kAligned ? 16 : 2), &o, 16);
      } else {
#pragma unroll
        for (int e = 0; e < 7; ++e)
          if (gc + e < p.n) dst[e] = __builtin_bit_cast(uint16_t, (_Float16)o[e]);
      }
    }
  }
};

}  // namespace kaio
