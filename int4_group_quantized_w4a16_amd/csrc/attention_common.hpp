// Pieces shared by the matrix-instruction attention kernels.
#pragma once

#include "attention_schedule.hpp"
#include "common.hpp"

namespace kaio {

typedef short short8_t __attribute__((ext_vector_type(8)));
typedef short short4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bhalf8_t __attribute__((ext_vector_type(8)));

// D = A.B + C on 16-bit operands of either type (bit patterns in short8_t).
template <bool kBf16>
__device__ __forceinline__ floatx16 mfma32(short8_t a, short8_t b, floatx16 c) {
  if constexpr (kBf16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bhalf8_t, a), __builtin_bit_cast(bhalf8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
}
template <bool kBf16>
__device__ __forceinline__ floatx4 mfma16(short8_t a, short8_t b, floatx4 c) {
  if constexpr (kBf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bhalf8_t, a), __builtin_bit_cast(bhalf8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8_t, a), __builtin_bit_cast(half8_t, b), c, 0, 0, 0);
}

// Two f32 -> two 16-bit values (nearest even) in one dword, one instruction.
template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (kBf16) {
    typedef __bf16 v2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, v2{(__bf16)a, (__bf16)b});
  } else {
    return __builtin_bit_cast(uint32_t, half2_t{(_Float16)a, (_Float16)b});
  }
}

// Transposed read of four rows (keys) x 16 columns of 16-bit values per group
// of 16 lanes: lane i of the group points at 8 bytes, columns 4 (i % 4) .. + 3
// of row i / 4, and receives column i of the four rows.
__device__ __forceinline__ short4_t read_tr(const void* lds) {
  return __builtin_bit_cast(short4_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) short4_t*)(const_cast<void*>(lds))));
}

// The value of the same lane % 32 (other half of the wave) combined with ours.
__device__ __forceinline__ float max_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1]));
}
__device__ __forceinline__ float add_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
  return __builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]);
}
// the same over lanes l % 16 of the four 16-lane rows
__device__ __forceinline__ float max_rows16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
  return max_halves(fmaxf(__builtin_bit_cast(float, (uint32_t)r[0]), __builtin_bit_cast(float, (uint32_t)r[1])));
}
__device__ __forceinline__ float add_rows16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, x), __builtin_bit_cast(uint32_t, x), false, false);
  return add_halves(__builtin_bit_cast(float, (uint32_t)r[0]) + __builtin_bit_cast(float, (uint32_t)r[1]));
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// The running maximum may lag behind the true one by this much (in powers of
// two) before the sums are rescaled: weights then reach 2^8 instead of 1, far
// inside f16's range, and rescaling, which touches every accumulator, becomes
// rare after the first blocks.  The result is the same quotient.
constexpr float kLag = 8.0f;

// Non-finite 16-bit values in a dword (any half with all exponent bits set).
template <bool kBf16>
__device__ __forceinline__ bool any_special(uint32_t w) {
  constexpr uint32_t e = kBf16 ? 0x7F807F80u : 0x7C007C00u, lsb = kBf16 ? 0x00800080u : 0x04000400u;
  return ((((w & e) + lsb) & 0x80008000u) != 0);   // the exponent field carries out only when full
}
// the same dword with its non-finite halves zeroed
template <bool kBf16>
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
  constexpr uint32_t e = kBf16 ? 0x7F80u : 0x7C00u;
  return ((w & e) == e ? 0u : w & 0xFFFFu) | (((w >> 16) & e) == e ? 0u : w & 0xFFFF0000u);
}
template <bool kBf16>
struct Special {   // split of eight values: the finite ones, and ones where NaN, +inf, -inf stand
  short8_t fin, nan, pos, neg;
  __device__ __forceinline__ explicit Special(short8_t v) {
    constexpr short one = kBf16 ? 0x3F80 : 0x3C00;
    constexpr uint16_t inf = kBf16 ? 0x7F80 : 0x7C00;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint16_t b = (uint16_t)v[i], m = b & 0x7FFF;
      fin[i] = m < inf ? v[i] : (short)0;
      nan[i] = m > inf ? one : (short)0;
      pos[i] = b == inf ? one : (short)0;
      neg[i] = b == (inf | 0x8000u) ? one : (short)0;
    }
  }
};
__device__ __forceinline__ float with_special(float x, float nan, float pos, float neg) {
  x += pos > 0.f ? INFINITY : 0.f;
  x -= neg > 0.f ? INFINITY : 0.f;
  return nan > 0.f ? NAN : x;
}

// Direct global -> LDS load of 16 bytes per lane: from base + off (base
// wave-uniform) to lds + 16 * lane.  The buffer form, whose pending loads the
// compiler does not hold against LDS reads; callers wait by wait_vm_barrier.
__device__ __forceinline__ void dma16(const char* base, uint32_t off, char* lds) {
  const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, -1, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, off, 0, 0, 0);
}
// Waits until at most N vector-memory operations of the wave are outstanding, then meets the others.
template <int N>
__device__ __forceinline__ void wait_vm_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

__device__ __forceinline__ short8_t join(short4_t a, short4_t b) {
  return short8_t{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// Workspace: a note per workgroup, then the partial results, per slot R rows
// of D f32, R maxima and R sums.
template <uint32_t R, uint32_t D>
__device__ __forceinline__ float* partial_of(const PagedAttention& p, uint32_t workers, uint32_t slot) {
  return reinterpret_cast<float*>(static_cast<JoinNote*>(p.workspace) + workers) + (size_t)slot * (R * (D + 2));
}

// Zeros for the rows of q that no sequence has: before q_start[0] and from
// q_start[seqs] on.  (At a kernel's end, where its loads wait for nobody.)
__device__ __forceinline__ void zero_unowned(const PagedAttention& p, uint32_t wg, uint32_t wgs) {
  const uint32_t T = p.kv.tokens;
  const uint32_t a = p.kv.seqs ? (uint32_t)clamp_row(p.kv.q_start[0], T) : T;
  uint32_t b = p.kv.seqs ? (uint32_t)clamp_row(p.kv.q_start[p.kv.seqs], T) : T;
  if (a == 0 && b == T) return;
  const uint32_t row = p.q_heads * p.kv.head_dim;
  for (uint32_t t = wg; t < T; t += wgs) {
    if (t >= a && t < b) {
      t += (b - 1 - t) / wgs * wgs;   // skip the owned rows
      continue;
    }
    for (uint32_t e = threadIdx.x * 8; e < row; e += blockDim.x * 8)
      *reinterpret_cast<uint4*>(p.out + (size_t)t * row + e) = uint4{0, 0, 0, 0};
  }
}

}  // namespace kaio
