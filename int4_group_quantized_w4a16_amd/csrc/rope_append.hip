// Rotary positions on Q and K, with K and V written to a paged cache.
//
// Pair j of a head (j < half; elements 2j and 2j + 1 when interleaved, j and
// j + half otherwise) turns by a = positions[axis(j)][t] * inv_freq[j], where
// the first sections[0] pairs belong to axis 0, the next sections[1] to axis
// 1, and so on: (x, y) -> (x cos a - y sin a, x sin a + y cos a).  Elements
// past 2 * half pass through unchanged.
//
// The angle is a product in 64 bits, brought to a fraction of a turn in 64
// bits (at position 2^31 a 32-bit angle would be off by whole turns), and only
// the fraction in [-1/2, 1/2] is rounded to 32 bits for the sine and cosine:
// 2^-25 of a turn, 2e-7 rad.  The rotation runs in 32 bits and is rounded once.
//
// Bound by memory: every element is read and written once.  A workgroup takes
// one token, up to four where a token's heads do not keep its threads busy, or
// a part of a token's heads when there are few tokens.  Its threads issue their
// loads first; the sines and cosines, computed once per token into LDS by one
// thread each, and the tokens' slots, found by one wave each, pass under the
// loads' latency.

#include "launch.hpp"
#include "paged.hpp"

namespace kaio {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr int kBatch = 2;      // items whose loads a thread has in flight
constexpr uint32_t kTokens = 4;   // tokens of a workgroup at most: one wave finds each one's slot

__device__ __forceinline__ void turn_of(const RopeAppend& p, uint32_t t, uint32_t j, float& c, float& s) {
  uint32_t axis = 0;
  for (uint32_t a = 1; a < kMaxAxes; ++a) axis += a < p.axes && j >= p.first_pair[a];
  // revolutions = position * (inv_freq / 2 pi); 1 / 2 pi rounded to 64 bits
  const double rev = (double)p.positions[(size_t)axis * p.kv.tokens + t] * p.inv_freq[j] * 0.15915494309189533577;
  sincospif(2.0f * (float)(rev - rint(rev)), &s, &c);
}

// Vector form: head_dim % 16 == 0 and half % 8 == 0.  An item is two 16-byte
// chunks of one head: of a turned part, chunks i and i + half / 8 (so that a
// thread holds both elements of its eight pairs) or, interleaved, neighbours;
// elsewhere two neighbouring chunks.
// kMulti: several tokens per workgroup.  One token's form is without their indexing (16384 tokens of 384 items: 67.6 us
// against 74.4 with it).
template <bool kBf16, bool kInter, bool kMulti>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(RopeAppend p, uint32_t parts, uint32_t per_part, uint32_t tokens,
                                                               FastDiv per_token) {
  extern __shared__ float cs[];   // per token: cos [half], sin [half]
  __shared__ int32_t slots[kTokens];
  const PagedKV& kv = p.kv;
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const uint32_t t0 = blockIdx.x / parts * tokens, part = blockIdx.x % parts;
  const uint32_t nt = !kMulti ? 1 : kv.tokens - t0 < tokens ? kv.tokens - t0 : tokens;
  const uint32_t d = kv.head_dim, half = p.half;
  const uint32_t qitems = p.q_heads * p.per_head.d, kitems = kv.kv_heads * p.per_head.d;
  const uint32_t items = qitems + 2 * kitems;
  // items of the workgroup: of its part of one token, or of all its tokens
  const uint32_t first = kMulti ? 0 : part * per_part;
  const uint32_t last = kMulti ? nt * items : first + per_part < items ? first + per_part : items;

  const uint16_t* const qsrc = p.q + (size_t)t0 * p.q_heads * d;
  const uint16_t* const ksrc = p.k_new + (size_t)t0 * kv.kv_heads * d;
  const uint16_t* const vsrc = p.v_new + (size_t)t0 * kv.kv_heads * d;

  // offsets (elements) of an item's two chunks within its tensor, and which tensor (0 q, 1 k, 2 v)
  auto place = [&](uint32_t n, uint32_t& token, uint32_t& which, uint32_t& a, uint32_t& b, uint32_t& pair) {
    token = kMulti ? per_token.div(n) : 0;
    const uint32_t item = n - token * items;
    which = item < qitems ? 0 : item < qitems + kitems ? 1 : 2;
    const uint32_t r = item - (which == 0 ? 0 : which == 1 ? qitems : qitems + kitems);
    const uint32_t h = p.per_head.div(r), i = r - h * p.per_head.d;
    uint32_t e;
    if (kInter || which == 2) {
      e = 16 * i;
      b = 8;
      pair = which == 2 || 8 * i >= half ? half : 8 * i;
    } else if (i < half / 8) {
      e = pair = 8 * i;
      b = half;
    } else {
      e = 2 * half + 16 * (i - half / 8);
      b = 8;
      pair = half;
    }
    a = h * d + e;
    b += a;
  };

  u32x4_t xa[kBatch], xb[kBatch];
  auto load = [&](uint32_t base) {
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      const uint32_t item = base + n * kThreads + tid;
      uint32_t token, which, a, b, pair;
      place(item < last ? item : first, token, which, a, b, pair);
      const uint16_t* src = which == 0 ? qsrc : which == 1 ? ksrc : vsrc;
      if constexpr (kMulti) src += token * (which == 0 ? p.q_heads : kv.kv_heads) * d;
      xa[n] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(src + a));
      xb[n] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(src + b));
    }
  };
  load(first);
  int32_t slot1 = -1;   // of the one token
  if constexpr (kMulti) {
    for (uint32_t n = tid; n < nt * half; n += kThreads) {
      const uint32_t token = n / half, j = n - token * half;
      float* const c = cs + token * 2 * half;
      turn_of(p, t0 + token, j, c[j], c[half + j]);
    }
  } else {
    for (uint32_t j = tid; j < half; j += kThreads) turn_of(p, t0, j, cs[j], cs[half + j]);
  }
  if (!kMulti || wave < nt) {
    uint32_t seq;
    int32_t pos;
    find_row(kv, kMulti ? t0 + wave : t0, lane, seq, pos);
    slot1 = seq < kv.seqs ? slot_of(kv, seq, pos) : -1;
    if (kMulti && lane == 0) slots[wave] = slot1;
  }
  __syncthreads();
  uint16_t* const qdst = p.q_out + (size_t)t0 * p.q_heads * d;
  uint16_t* const kdst = kv.k + (size_t)(slot1 < 0 ? 0 : slot1) * kv.kv_heads * d;
  uint16_t* const vdst = kv.v + (size_t)(slot1 < 0 ? 0 : slot1) * kv.kv_heads * d;

  for (uint32_t base = first; base < last; base += kBatch * kThreads) {
    if (base != first) load(base);
#pragma unroll
    for (int n = 0; n < kBatch; ++n) {
      const uint32_t item = base + n * kThreads + tid;
      if (item >= last) continue;
      uint32_t token, which, a, b, pair;
      place(item, token, which, a, b, pair);
      const float* const cst = cs + token * 2 * half;
      if (pair < half) {
        uint16_t x[16], y[16];
        __builtin_memcpy(x, &xa[n], 16);
        __builtin_memcpy(x + 8, &xb[n], 16);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i0 = kInter ? 2 * e : e, i1 = kInter ? 2 * e + 1 : 8 + e;
          const uint32_t j = pair + e;
          // interleaved pairs past half pass through (half % 8 == 0: none within an item)
          const float c = cst[j], s = cst[half + j];
          const float u = to_f32<kBf16>(x[i0]), w = to_f32<kBf16>(x[i1]);
          y[i0] = from_f32<kBf16>(u * c - w * s);
          y[i1] = from_f32<kBf16>(u * s + w * c);
        }
        __builtin_memcpy(&xa[n], y, 16);
        __builtin_memcpy(&xb[n], y + 8, 16);
      }
      const int32_t slot = kMulti ? slots[token] : slot1;
      if (which != 0 && slot < 0) continue;
      uint16_t* dst;
      if constexpr (kMulti)
        dst = which == 0 ? qdst + token * p.q_heads * d : (which == 1 ? kv.k : kv.v) + (size_t)slot * kv.kv_heads * d;
      else
        dst = which == 0 ? qdst : which == 1 ? kdst : vdst;
      *reinterpret_cast<u32x4_t*>(dst + a) = xa[n];
      *reinterpret_cast<u32x4_t*>(dst + b) = xb[n];
    }
  }
}

// Element form for the other sizes: one thread per pair or pass-through element,
// 2-byte accesses (16384 tokens, 32 + 2 x 8 heads of 80 columns: 175 us with 20
// pairs, against 52 us of the vector form with 40; 4 tokens, 96 heads of 72: 11).
template <bool kBf16, bool kInter>
__global__ void __launch_bounds__(kThreads) rope_append_any_kernel(RopeAppend p) {
  extern __shared__ float cs[];
  const PagedKV& kv = p.kv;
  const uint32_t tid = threadIdx.x, t = blockIdx.x;
  const uint32_t d = kv.head_dim, half = p.half;
  for (uint32_t j = tid; j < half; j += kThreads) turn_of(p, t, j, cs[j], cs[half + j]);
  uint32_t seq;
  int32_t pos;
  find_row(kv, t, tid & 63, seq, pos);
  const int32_t slot = seq < kv.seqs ? slot_of(kv, seq, pos) : -1;
  __syncthreads();
  const uint32_t heads = p.q_heads + 2 * kv.kv_heads;
  for (uint32_t i = tid; i < heads * d; i += kThreads) {
    const uint32_t hd = i / d, e = i - hd * d;
    const bool q = hd < p.q_heads, v = hd >= p.q_heads + kv.kv_heads;
    const uint32_t h = q ? hd : hd - p.q_heads - (v ? kv.kv_heads : 0);
    const uint16_t* src = (q ? p.q : v ? p.v_new : p.k_new) + ((size_t)t * (q ? p.q_heads : kv.kv_heads) + h) * d;
    if (!q && slot < 0) continue;
    uint16_t* dst = q ? p.q_out + ((size_t)t * p.q_heads + h) * d
                      : (v ? kv.v : kv.k) + ((size_t)slot * kv.kv_heads + h) * d;
    if (v || e >= 2 * half) {
      dst[e] = src[e];
      continue;
    }
    // the thread of a pair's first element turns the pair
    const bool lead = kInter ? (e & 1) == 0 : e < half;
    if (!lead) continue;
    const uint32_t j = kInter ? e / 2 : e, e1 = kInter ? e + 1 : e + half;
    const float u = to_f32<kBf16>(src[e]), w = to_f32<kBf16>(src[e1]);
    dst[e] = from_f32<kBf16>(u * cs[j] - w * cs[half + j]);
    dst[e1] = from_f32<kBf16>(u * cs[half + j] + w * cs[j]);
  }
}

template <bool kBf16, bool kInter>
hipError_t launch(const RopeAppend& p, hipStream_t stream) {
  const uint32_t d = p.kv.head_dim, t = p.kv.tokens;
  const size_t lds = 2 * sizeof(float) * (p.half ? p.half : 1);
  if (d % 16 != 0 || p.half % 8 != 0) {
    hipLaunchKernelGGL((rope_append_any_kernel<kBf16, kInter>), dim3(t), dim3(kThreads), lds, stream, p);
    return hipGetLastError();
  }
  const uint32_t items = (p.q_heads + 2 * p.kv.kv_heads) * (d / 16);
  // few tokens: one item per thread, the token's heads spread over workgroups
  const uint32_t most = (items + kThreads - 1) / kThreads;
  const uint32_t parts = (uint64_t)t * most <= kComputeUnits * 4 ? most : 1;
  const uint32_t per = (items + parts - 1) / parts;
  // many tokens with few items each share a workgroup, as long as there are workgroups for every compute unit
  // (2357 tokens of 96 items: 6.8 us with one token each, 5.9 with four)
  uint32_t tokens = parts == 1 && items ? kBatch * kThreads / items : 1;
  tokens = tokens < 1 ? 1 : tokens > kTokens ? kTokens : tokens;
  while (tokens > 1 && t / tokens < 2 * kComputeUnits) --tokens;
  const uint32_t wgs = (t + tokens - 1) / tokens * parts;
  if (tokens > 1)
    hipLaunchKernelGGL((rope_append_kernel<kBf16, kInter, true>), dim3(wgs), dim3(kThreads), tokens * lds, stream, p, parts,
                       per, tokens, FastDiv::of(items));
  else
    hipLaunchKernelGGL((rope_append_kernel<kBf16, kInter, false>), dim3(wgs), dim3(kThreads), lds, stream, p, parts, per,
                       tokens, FastDiv::of(items));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope_append(const RopeAppend& p, hipStream_t stream) {
  if (p.bf16) return p.interleaved ? launch<true, true>(p, stream) : launch<true, false>(p, stream);
  return p.interleaved ? launch<false, true>(p, stream) : launch<false, false>(p, stream);
}

}  // namespace kaio
