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

// The two 16-bit values of pack2 added to acc (f32, subnormals kept).
template <bool kBf16>
__device__ __forceinline__ float add2(uint32_t pair, float acc) {
  if constexpr (kBf16) {
    typedef __bf16 v2 __attribute__((ext_vector_type(2)));
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(v2, pair), v2{(__bf16)1.0f, (__bf16)1.0f}, acc, false);
  } else {
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(half2_t, pair), half2_t{(_Float16)1.0f, (_Float16)1.0f}, acc, false);
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
// two) before the sums are rescaled: weights then reach 2^5 instead of 1, and
// rescaling, which touches every accumulator, becomes rare after the first
// blocks.  The result is the same quotient.
constexpr float kLag = 5.0f;

// Added to every weight's exponent, so that f16, whose normal numbers end at
// 2^-14, keeps all bits of weights down to 2^-21 of the largest and rounds only
// those under 2^-32 of it to zero (of a long axis they could be many).  With
// kLag the largest weight is 2^12; f16 ends at 2^16, which leaves room for the
// steps of f32 in a score, up to 4 for scores of 2^26.  bf16 has f32's range.
template <bool kBf16>
constexpr float kLift = kBf16 ? 0.0f : 7.0f;

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

__device__ __forceinline__ u32x4 raw_rsrc(const char* base) {   // raw buffer, no range limit
  const uint64_t b = reinterpret_cast<uint64_t>(base);
  return u32x4{(uint32_t)b, (uint32_t)(b >> 32), 0xFFFFFFFFu, 0x00020000u};
}
// Direct global -> LDS load of 16 bytes per lane: from base + off (base
// wave-uniform) to lds + 16 * lane.  In assembly (no register is written): from
// the builtin the compiler knows that LDS changes, cannot tell the buffers of a
// ring apart, and waits for every load in flight before a read of any.  Callers
// wait by wait_vm_barrier; the compiler's own counts for other loads only get
// stricter by loads that it does not see.  The wait states cover m0 (one) and a
// descriptor that a lane read has just written (five); the compiler, which does
// not see what the assembly reads, adds none.
template <int kBytes>
__device__ __forceinline__ void dma(const char* base, uint32_t off, void* lds) {
  const u32x4 rsrc = raw_rsrc(base);
  const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
  if constexpr (kBytes == 16)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(at), "v"(off), "s"(rsrc) : "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(at), "v"(off), "s"(rsrc) : "m0");
}
// A K and a V load of the same cache rows: from the descriptors' bases + slot *
// row_bytes (32 bits) + the lane's offsets to lds and lds + kApart.  Five wait
// states before the first load, as in dma; the second's descriptor has more.
template <int kApart>
__device__ __forceinline__ void dma16_pair(u32x4 krsrc, uint32_t koff, u32x4 vrsrc, uint32_t voff, uint32_t slot,
                                           uint32_t row_bytes, void* lds) {
  const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
  uint32_t row;
  asm volatile("s_mul_i32 %0, %1, %2\n\ts_mov_b32 m0, %3\n\ts_nop 2\n\tbuffer_load_dwordx4 %5, %6, %0 offen lds\n\t"
               "s_add_u32 m0, %3, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %7, %8, %0 offen lds"
               : "=&s"(row)
               : "s"(slot), "s"(row_bytes), "s"(at), "n"(kApart), "v"(koff), "s"(krsrc), "v"(voff), "s"(vrsrc)
               : "m0", "scc");
}
__device__ __forceinline__ void dma16(const char* base, uint32_t off, void* lds) { dma<16>(base, off, lds); }
__device__ __forceinline__ void dma4(const char* base, uint32_t off, void* lds) { dma<4>(base, off, lds); }
// Waits until at most N vector-memory operations of the wave are outstanding,
// and its LDS operations are done.  By the builtin (vmcnt in bits 0-3 and
// 14-15, expcnt 4-6, lgkmcnt 8-11): the compiler then knows that older loads
// have landed and adds no waits of its own for them.
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | ((N >> 4) << 14));
  asm volatile("" ::: "memory");
}
// At most N LDS operations outstanding (vector memory aside).
template <int N>
__device__ __forceinline__ void wait_lds() {
  __builtin_amdgcn_s_waitcnt(15 | (7 << 4) | (N << 8) | (3 << 14));
}
// wait_vm, and meets the other waves.
template <int N>
__device__ __forceinline__ void wait_vm_barrier() {
  wait_vm<N>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
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

// Where the tile form puts columns col .. col + 3 of row r of a partial result:
// as its lanes hold them, so that each store of a wave is one piece of 1 KiB
// (row by row its 64 lanes wrote 16 bytes each to 32 rows).
template <int D>
__device__ __forceinline__ uint32_t fragment_of(uint32_t r, uint32_t col) {
  return ((r / 32 * (D / 32) + col / 32) * 4 + col % 32 / 8) * 256 + (col % 8 / 4 * 32 + r % 32) * 4;
}

// Zeros for the rows of q that no sequence has: outside [a, b).
__device__ __forceinline__ void zero_unowned(const PagedAttention& p, uint32_t wg, uint32_t wgs, uint32_t a, uint32_t b) {
  const uint32_t T = p.kv.tokens;
  if (a == 0 && b == T) return;
  const uint32_t row = p.q_heads * p.kv.head_dim;
  for (uint32_t t = wg; t < T; t += wgs) {
    if (t >= a && t < b) {
      t += (b - 1 - t) / wgs * wgs;   // skip the others
      continue;
    }
    for (uint32_t e = threadIdx.x * 8; e < row; e += blockDim.x * 8)
      *reinterpret_cast<uint4*>(p.out + (size_t)t * row + e) = uint4{0, 0, 0, 0};
  }
}

}  // namespace kaio
