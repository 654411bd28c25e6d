// The paged key/value cache as the kernels see it, shared by rope_append.hip
// and the attention kernels.
//
// A batch holds `seqs` sequences.  Sequence s has new tokens in rows
// q_start[s] .. q_start[s+1] of q and lens[s] tokens in the cache, the new
// ones last: row t of it sits at position lens[s] - (q_start[s+1] - t).  The
// token at position c lies in slot c % page_size of page
// table[s][c / page_size]; a page id outside [0, pages) stands for a page
// that is not there (nothing is read from it or written to it).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kaio {

// c / d for 0 <= c < 2^31 by one 64-bit multiply: mul = floor(2^(31+l) / d) + 1
// with 2^(l-1) < d <= 2^l, whose excess over 2^(31+l) / d is at most 2^l / d *
// 2^-(31+l) * 2^31 < 1 quotient step for every such c.
struct FastDiv {
  uint32_t d, mul, shift;
  __host__ static FastDiv of(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    return FastDiv{d, (uint32_t)((1ull << (31 + l)) / d + 1), 31 + l};
  }
  __device__ __forceinline__ uint32_t div(uint32_t c) const { return (uint32_t)(((uint64_t)c * mul) >> shift); }
};

struct PagedKV {
  uint16_t* k;              // [pages, page_size, kv_heads, head_dim], 16-bit elements
  uint16_t* v;
  const int32_t* table;     // [seqs, width]
  const int32_t* q_start;   // [seqs + 1]
  const int32_t* lens;      // [seqs]
  uint32_t pages, kv_heads, head_dim, seqs, width;
  uint32_t cap;             // width * page_size, at most 2^31 - 1: positions the table covers
  FastDiv page;
  uint32_t tokens;          // rows of q
};

// Slot (row of the cache) of position c of sequence s, or -1 if it is not there.
__device__ __forceinline__ int32_t slot_of(const PagedKV& kv, uint32_t s, int32_t c) {
  if (c < 0 || (uint32_t)c >= kv.cap) return -1;
  const uint32_t p = kv.page.div((uint32_t)c);
  const uint32_t id = (uint32_t)kv.table[(size_t)s * kv.width + p];
  return id < kv.pages ? (int32_t)(id * kv.page.d + ((uint32_t)c - p * kv.page.d)) : -1;
}

// Sequence of row t of q and its position; seq = seqs where no sequence has
// the row (a batch padded past q_start[seqs]).  Wave-uniform t; every lane
// compares one bound per pass, so 64 sequences cost one load.
__device__ __forceinline__ void find_row(const PagedKV& kv, uint32_t t, uint32_t lane, uint32_t& seq, int32_t& pos) {
  seq = kv.seqs;
  pos = -1;
  for (uint32_t s0 = 0; s0 < kv.seqs; s0 += 64) {
    const uint32_t s = s0 + lane;
    const bool in = s < kv.seqs;
    const int32_t lo = in ? kv.q_start[s] : 0, hi = in ? kv.q_start[s + 1] : 0, len = in ? kv.lens[s] : 0;
    const uint64_t hit = __ballot(in && lo <= (int32_t)t && (int32_t)t < hi);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      seq = s0 + l;
      pos = __builtin_amdgcn_readlane(len, l) - (__builtin_amdgcn_readlane(hi, l) - (int32_t)t);
      return;
    }
  }
}

// f32 <-> the 16-bit element types, by template parameter
template <bool kBf16>
__device__ __forceinline__ float to_f32(uint16_t b) {
  if constexpr (kBf16) return __builtin_bit_cast(float, (uint32_t)b << 16);
  else return (float)__builtin_bit_cast(_Float16, b);
}
template <bool kBf16>
__device__ __forceinline__ uint16_t from_f32(float f) {
  if constexpr (kBf16) return __builtin_bit_cast(uint16_t, (__bf16)f);
  else return __builtin_bit_cast(uint16_t, (_Float16)f);
}

}  // namespace kaio
