// Rows rounded to 8 bits, each with a scale of its own (rounding.hpp).
//
// Bound: HBM, 3 bytes per element.  A row is read once and held in registers
// between its maximum and its rounding (up to 32768 elements; past that it is
// read again, mostly from the caches), by a wave where that holds it in one turn,
// else by a workgroup.
//
// Measured: 16384 x 4096 39.3 us (5.1 TB/s, what a copy reaches), 16384 x 8192
// 74.3 us (5.4 TB/s), 1 to 64 x 4096 2.2 to 2.5 us (a launch).  Rows of 256 / 512 /
// 1024 elements, 32768 of them: by waves 14.3 / 16.1 / 22.3 us, by workgroups 27.7 /
// 28.6 / 31.1.  1024 rows of 32768 held 25.0 us, read twice 30.7.  Stores are plain
// ones: nontemporal, 2 to 15% less here, they make the product that reads the
// rounded rows wait for them (61 x 11004 x 4096 14.1 -> 14.8 us in all).

#include "common.hpp"
#include "launch.hpp"
#include "rounding.hpp"

namespace kaio {
namespace {

constexpr int kThreads = 256;

// kRow threads share a row (64: a wave; kThreads: the workgroup) and hold kHeld
// pieces of 16 elements each; kHeld 0: any number, read twice.
template <bool kBf16, int kRow, int kHeld>
__global__ void __launch_bounds__(kThreads)
quantize_rows_kernel(const uint16_t* __restrict__ x, uint8_t* __restrict__ q, float* __restrict__ scale, uint32_t m, uint32_t k) {
  const uint32_t row = blockIdx.x * (kThreads / kRow) + threadIdx.x / kRow, at = threadIdx.x % kRow, pieces = k / 16;
  if (kRow == 64 && row >= m) return;
  const uint4* const src = reinterpret_cast<const uint4*>(x + (size_t)row * k);
  uint4* const dst = reinterpret_cast<uint4*>(q + (size_t)row * k);
  uint4 v[kHeld ? kHeld : 1][2];
  uint32_t most = 0;
  if constexpr (kHeld != 0) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const uint32_t p = at + i * kRow;
      v[i][0] = v[i][1] = uint4{0, 0, 0, 0};
      if (p < pieces) {
        v[i][0] = src[2 * p];
        v[i][1] = src[2 * p + 1];
      }
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i) most = max_bits(max_bits(most, v[i][0]), v[i][1]);
  } else {
    for (uint32_t p = at; p < pieces; p += kRow) most = max_bits(max_bits(most, src[2 * p]), src[2 * p + 1]);
  }
#pragma unroll
  for (int s = 32; s; s >>= 1) most = max_bits(most, (uint32_t)__shfl_xor((int)most, s));
  if constexpr (kRow > 64) {
    __shared__ uint32_t waves[kRow / 64];
    if (at % 64 == 0) waves[at / 64] = most;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kRow / 64; ++w) most = max_bits(most, waves[w]);
  }
  most = (most >> 16) > (most & 0xFFFFu) ? most >> 16 : most & 0xFFFFu;
  const Rounding r = Rounding::of<kBf16>(most);
  if (at == 0) scale[row] = Rounding::scale<kBf16>(most);
  if constexpr (kHeld != 0) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const uint32_t p = at + i * kRow;
      if (p < pieces) dst[p] = r.sixteen<kBf16>(v[i][0], v[i][1]);
    }
  } else {
    for (uint32_t p = at; p < pieces; p += kRow) dst[p] = r.sixteen<kBf16>(src[2 * p], src[2 * p + 1]);
  }
}

template <bool kBf16>
hipError_t launch(const uint16_t* x, uint8_t* q, float* scale, uint32_t m, uint32_t k, hipStream_t stream) {
  const uint32_t pieces = k / 16;
#define KAIO_ROWS(ROW, HELD)                                                                                        \
  hipLaunchKernelGGL((quantize_rows_kernel<kBf16, ROW, HELD>), dim3((m + kThreads / ROW - 1) / (kThreads / ROW)), \
                     dim3(kThreads), 0, stream, x, q, scale, m, k)
  if (pieces <= 64) KAIO_ROWS(64, 1);
  else if (pieces <= kThreads) KAIO_ROWS(kThreads, 1);
  else if (pieces <= 2 * kThreads) KAIO_ROWS(kThreads, 2);
  else if (pieces <= 4 * kThreads) KAIO_ROWS(kThreads, 4);
  else if (pieces <= 8 * kThreads) KAIO_ROWS(kThreads, 8);
  else KAIO_ROWS(kThreads, 0);
#undef KAIO_ROWS
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_rows(const uint16_t* x, bool bf16, uint8_t* q, float* scale, uint32_t m, uint32_t k,
                                hipStream_t stream) {
  return bf16 ? launch<true>(x, q, scale, m, k, stream) : launch<false>(x, q, scale, m, k, stream);
}

}  // namespace kaio
