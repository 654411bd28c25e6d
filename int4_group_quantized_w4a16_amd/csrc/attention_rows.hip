// Attention over the paged cache, by rows: one wave per row and head, for head
// sizes that the matrix-instruction forms do not have.
//
//   o = sum_c p_c v_c / sum_c p_c,  p_c = exp(scale * q.k_c - m),  m = max
//
// over the visible positions c of the row at position pos: 0 <= c <= pos, the
// page there, and with a window c > pos - window or c < sinks.  A row that sees
// nothing is zero.  Lane j scores key 64 b + j of block b; the running maximum
// and sum go with the blocks, so each key is read once per row and head.
//
// A simple kernel, bound by its loads' latency: each lane walks its key by
// 2-byte loads, and the wave V key by key.  64 sequences of 125 to 8000 keys,
// bf16: 32 heads over 8 of 80 or 96 columns 6.2 ms, 16 over 4 of 256 13.4 ms
// (0.1 TB/s); 512 causal tokens, 32 heads over 8 of 96: 344 us.

#include "launch.hpp"
#include "paged.hpp"

namespace kaio {
namespace {

constexpr int kMaxDim = 256;

template <bool kBf16>
__global__ void __launch_bounds__(64) paged_attention_rows_kernel(PagedAttention p) {
  __shared__ float qs[kMaxDim];
  __shared__ float ps[64];
  __shared__ int32_t slots[64];
  const PagedKV& kv = p.kv;
  const uint32_t lane = threadIdx.x, d = kv.head_dim;
  const uint32_t t = blockIdx.x / p.q_heads, h = blockIdx.x % p.q_heads;
  const uint32_t kh = p.group.div(h);
  uint32_t seq;
  int32_t pos;
  find_row(kv, t, lane, seq, pos);
  for (uint32_t e = lane; e < d; e += 64) qs[e] = to_f32<kBf16>(p.q[((size_t)t * p.q_heads + h) * d + e]);
  __syncthreads();
  float m = -INFINITY, l = 0.f, o[kMaxDim / 64] = {};
  const int64_t lo = p.window ? (int64_t)pos - p.window : -1;   // c > lo, or c < sinks
  const int64_t end = pos < (int64_t)kv.cap ? pos : (int64_t)kv.cap - 1;   // nothing is past the table
  for (int64_t c0 = 0; c0 <= end; c0 += 64) {
    if (p.window && c0 + 63 <= lo && c0 >= p.sinks) {          // between the sinks and the window
      c0 = (lo + 1) / 64 * 64 - 64;
      continue;
    }
    const int64_t c = c0 + lane;
    const bool sees = c <= pos && (c > lo || c < p.sinks);
    const int32_t slot = sees ? slot_of(kv, seq, (int32_t)c) : -1;
    float s = -INFINITY;
    if (slot >= 0) {
      const uint16_t* kr = kv.k + ((size_t)slot * kv.kv_heads + kh) * d;
      float dot = 0.f;
      for (uint32_t e = 0; e < d; ++e) dot += qs[e] * to_f32<kBf16>(kr[e]);
      s = dot * p.scale;
    }
    float top = s;
    for (int x = 32; x; x >>= 1) top = fmaxf(top, __shfl_xor(top, x));
    const float m1 = fmaxf(m, top), base = m1 == -INFINITY ? 0.f : m1;
    const float w = slot >= 0 ? expf(s - base) : 0.f, old = expf(m - base);
    float sum = w;
    for (int x = 32; x; x >>= 1) sum += __shfl_xor(sum, x);
    l = l * old + sum;
    m = m1;
    ps[lane] = w;
    slots[lane] = slot;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMaxDim / 64; ++i) o[i] *= old;
    for (int j = 0; j < 64; ++j) {
      if (slots[j] < 0) continue;
      const uint16_t* vr = kv.v + ((size_t)slots[j] * kv.kv_heads + kh) * d;
#pragma unroll
      for (int i = 0; i < kMaxDim / 64; ++i)
        if (lane + 64 * i < d) o[i] += ps[j] * to_f32<kBf16>(vr[lane + 64 * i]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < kMaxDim / 64; ++i)
    if (lane + 64 * i < d)
      p.out[((size_t)t * p.q_heads + h) * d + lane + 64 * i] = from_f32<kBf16>(l == 0.f ? 0.f : o[i] / l);
}

}  // namespace

hipError_t launch_attention_rows(const PagedAttention& p, hipStream_t stream) {
  const dim3 grid(p.kv.tokens * p.q_heads);
  if (p.bf16)
    hipLaunchKernelGGL((paged_attention_rows_kernel<true>), grid, dim3(64), 0, stream, p);
  else
    hipLaunchKernelGGL((paged_attention_rows_kernel<false>), grid, dim3(64), 0, stream, p);
  return hipGetLastError();
}

}  // namespace kaio
