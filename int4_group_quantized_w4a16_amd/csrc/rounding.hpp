// Rounding of rows of 16-bit numbers to 8 bits:
//
//   a_i = max_j |x_ij|,  s_i = a_i / 127,  q_ij = round(127 x_ij / a_i)   (ties to even)
//
// Exactness.  With x and a of 11 (f16) or 8 (bf16) bits 127 x has at most 18
// and is exact in f32.  Where 127 x / a is not n + 1/2 itself it lies at least
// 2^-(d + 12) from it (a ratio of integers; d: how many powers of two x lies
// below a), 32 times half a step of f32 of that quotient: a quotient off by one
// step rounds to the same integer.  An n + 1/2 has to come out as itself, which
// one correction of the approximate quotient does: what it leaves is 2^-44.
//
// A row of zeros has s = 0 and q = 0.  A row with an infinity or a NaN has
// s = NaN and q = 0, so that every product with it is NaN.
#pragma once

#include "paged.hpp"

namespace kaio {

typedef uint16_t ushort2_t __attribute__((ext_vector_type(2)));

// largest magnitude of a row of 16-bit numbers, as bits: those of magnitudes are in their order, infinity and NaN last
__device__ __forceinline__ uint32_t max_bits(uint32_t a, uint32_t pair) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(ushort2_t, a),
                                                                __builtin_bit_cast(ushort2_t, pair & 0x7FFF7FFFu)));
}
__device__ __forceinline__ uint32_t max_bits(uint32_t a, uint4 v) {
  return max_bits(max_bits(max_bits(max_bits(a, v.x), v.y), v.z), v.w);
}

// What a row is rounded with: f brings numbers of bf16's far ranges near 1 (powers of two; what that pushes out of the
// range is under 2^-100 of the row's largest and rounds to zero).
struct Rounding {
  float times, most, inverse;   // 127 f, a f, about 1 / (a f); times 0 where q is 0 throughout
  template <bool kBf16>
  __device__ __forceinline__ static Rounding of(uint32_t bits) {
    const float a = to_f32<kBf16>((uint16_t)bits);
    const bool none = bits == 0 || bits >= (kBf16 ? 0x7F80u : 0x7C00u);
    const float f = !kBf16 ? 1.f : a > 0x1p60f ? 0x1p-68f : a < 0x1p-60f ? 0x1p73f : 1.f;
    const float most = none ? 1.f : a * f;
    return Rounding{none ? 0.f : 127.f * f, most, __builtin_amdgcn_rcpf(most)};
  }
  template <bool kBf16>
  __device__ __forceinline__ static float scale(uint32_t bits) {
    return bits >= (kBf16 ? 0x7F80u : 0x7C00u) ? NAN : to_f32<kBf16>((uint16_t)bits) / 127.f;
  }
  // the integer in the low byte: adding 1.5 * 2^23 rounds to one
  template <bool kBf16>
  __device__ __forceinline__ uint32_t operator()(uint16_t x) const {
    const float t = to_f32<kBf16>(x) * times;
    float q = t * inverse;
    q = __builtin_fmaf(__builtin_fmaf(-q, most, t), inverse, q);
    return __builtin_bit_cast(uint32_t, q + 12582912.f);
  }
  template <bool kBf16>
  __device__ __forceinline__ uint32_t four(uint32_t lo, uint32_t hi) const {
    const uint32_t a = __builtin_amdgcn_perm((*this).operator()<kBf16>((uint16_t)(lo >> 16)), (*this).operator()<kBf16>((uint16_t)lo), 0x0C0C0400u);
    const uint32_t b = __builtin_amdgcn_perm((*this).operator()<kBf16>((uint16_t)(hi >> 16)), (*this).operator()<kBf16>((uint16_t)hi), 0x0C0C0400u);
    return a | (b << 16);
  }
  template <bool kBf16>
  __device__ __forceinline__ uint4 sixteen(uint4 a, uint4 b) const {
    // infinities and NaN of a row that has none in q: 0 * inf would be NaN, whose low byte is not zero
    if (times == 0.f) return uint4{0, 0, 0, 0};
    return uint4{four<kBf16>(a.x, a.y), four<kBf16>(a.z, a.w), four<kBf16>(b.x, b.y), four<kBf16>(b.z, b.w)};
  }
};

}  // namespace kaio
