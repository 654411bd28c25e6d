// Product in 8-bit integers with a scale for each token and each channel:
//
//   y[i, j] = act( xs[i] ws[j] sum_k xq[i, k] wq[j, k] + b[j] ) + r[i, j]
//
// The sum is exact in i32 (k < 2^17), so the order of its parts does not show.
// Both operands are read as they lie, [index][k]: a lane of a 16x16x64 MFMA
// takes 16 consecutive k of one row.  The channels are the MFMA's rows and the
// tokens its columns, so that a lane ends with consecutive channels of a token.
//
// Tiles (linear8_tile_kernel), many tokens.  Both operands go to LDS by direct
// 16-byte loads, 64 k a step, in a ring of kRing steps; per step a wave issues
// its MFMAs on fragments in registers, reads the next step's fragments between
// them and sends for the step kRing ahead, into the place that this step's
// fragments came from; one barrier per step.
//
// Strips (linear8_strip_kernel), few tokens: the weights are the work and go
// from memory to registers once; a workgroup's waves share out k and add up in
// LDS.

#include "attention_common.hpp"
#include "common.hpp"
#include "epilogue.hpp"
#include "launch.hpp"
#include "paged.hpp"

#include <type_traits>

namespace kaio {
namespace {

typedef int intx4 __attribute__((ext_vector_type(4)));

// Eight consecutive channels of one token, from their integer sums.
template <bool kBf16>
struct Channels8 {
  float ws[8], bias[8];
  // 8 x 16 bits from `src`, of which the first `n` are there
  static __device__ __forceinline__ void fetch(const uint16_t* src, uint32_t n, float (&out)[8]) {
    uint16_t v[8] = {};
    if (n >= 8) {
      __builtin_memcpy(v, __builtin_assume_aligned(src, 2), 16);
    } else {
#pragma unroll
      for (uint32_t e = 0; e < 7; ++e)
        if (e < n) v[e] = src[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = to_f32<kBf16>(v[e]);
  }
  // channels col .. col + 7, col a multiple of 8, of which the first `n` are there
  __device__ __forceinline__ void load(const Linear8& p, uint32_t col, uint32_t n) {
    if (n >= 8) {
      const float4 a = *reinterpret_cast<const float4*>(p.ws + col), b = *reinterpret_cast<const float4*>(p.ws + col + 4);
      ws[0] = a.x, ws[1] = a.y, ws[2] = a.z, ws[3] = a.w, ws[4] = b.x, ws[5] = b.y, ws[6] = b.z, ws[7] = b.w;
    } else {
#pragma unroll
      for (uint32_t e = 0; e < 8; ++e) ws[e] = e < n ? p.ws[col + e] : 0.f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) bias[e] = 0.f;
    if (p.bias) fetch(p.bias + col, n, bias);
  }
  __device__ __forceinline__ void store(const Linear8& p, const int (&acc)[8], float xs, size_t at, uint32_t n) const {
    float y[8], r[8] = {};
    if (p.residual) fetch(p.residual + at, n, r);
    // the channel's scale first: what is out of f32's range after the token's is so in the result
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf((float)acc[e] * ws[e], xs, bias[e]);
    activations<8>(y, p.act);
    uint16_t out[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = from_f32<kBf16>(y[e] + r[e]);
    uint16_t* const dst = p.y + at;
    if (n >= 8) {
      __builtin_memcpy(__builtin_assume_aligned(dst, 2), out, 16);
    } else {
#pragma unroll
      for (uint32_t e = 0; e < 7; ++e)
        if (e < n) dst[e] = out[e];
    }
  }
};

// ---- tiles ------------------------------------------------------------------

// The MFMA with its accumulator in place: from the builtin the compiler makes copies of accumulators at loop edges.  It
// does not see the hazards of these: `settle` waits before results are read, and after registers are cleared.
__device__ __forceinline__ void mfma_inplace(intx4& acc, const intx4& a, const intx4& b) {
  asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}
template <int TM, int TN>
__device__ __forceinline__ void settle(intx4 (&acc)[TM][TN]) {
  asm volatile("s_nop 15\n\ts_nop 15\n\ts_nop 15" : "+a"(acc[0][0]));
#pragma unroll
  for (int r = 0; r < TM; ++r)
#pragma unroll
    for (int c = 0; c < TN; ++c) asm volatile("" : "+a"(acc[r][c]));
}

// Direct load to LDS of 16 bytes per lane: from rsrc's base + soff + the lane's offset to lds + 16 * lane.  (See dma in
// attention_common.hpp for the form and its wait states.)
__device__ __forceinline__ void load_lds(u32x4 rsrc, uint32_t off, uint32_t soff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(off), "s"(rsrc), "s"(soff) : "m0");
}

// Places of 16-byte chunks in a step's rows of 64 bytes: chunk c of row r in slot 4 r + (c ^ spread(r)).  A fragment read
// is served 8 lanes at a time over 128 bytes of banks, two rows of one parity then apart by their spread: both by
// consecutive rows (tokens) and by rows 0-3 and 8-11 of 16 (channels).
__device__ __forceinline__ uint32_t spread(uint32_t r) { return ((r >> 1) & 3) ^ (((r >> 3) & 1) * 3); }

// BC channels by BT tokens by NWC x NWT waves; kRagged: k % 64 != 0 (a chunk past k is then read as zeros, by an offset
// outside of the descriptor's range).
template <bool kRagged, int BC, int BT, int NWC, int NWT, int kRing>
__global__ void __launch_bounds__(64 * NWC * NWT, 1) linear8_tile_kernel(Linear8 p, uint32_t ctiles, uint32_t ttiles) {
  constexpr int NW = NWC * NWT, WC = BC / NWC, WT = BT / NWT, TM = WC / 16, TN = WT / 16;
  constexpr int kLoads = (BC + BT) * 4 / (64 * NW);
  constexpr uint32_t kStep = (BC + BT) * 64;   // bytes of a step
  static_assert(TM % 2 == 0 && (BC + BT) * 4 % (64 * NW) == 0 && BC % 16 == 0, "tile");
  extern __shared__ char lds[];
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t kq = lane >> 4, l16 = lane & 15, wc = wave / NWT, wt = wave % NWT;

  // Tiles in bands of 4 tiles of tokens, channel by channel: what runs at a time on an XCD shares rows of both operands.
  const uint32_t id = xcd_remap(blockIdx.x, gridDim.x), band = id / (4 * ctiles), in = id - band * 4 * ctiles;
  const uint32_t high = ttiles - 4 * band < 4 ? ttiles - 4 * band : 4;
  const uint32_t m0 = (4 * band + in % high) * BT, n0 = in / high * BC;

  const uint32_t K = p.k, steps = (K + 63) / 64;
  constexpr uint32_t kRange = 0x7FFFFFF0u, kOutside = 0x80000000u;
  u32x4 rsrc[2];
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const uint64_t b = reinterpret_cast<uint64_t>(o ? p.x + (size_t)m0 * K : p.w + (size_t)n0 * K);
    rsrc[o] = u32x4{(uint32_t)b, (uint32_t)(b >> 32) & 0xFFFFu, kRange, 0x00020000u};
  }
  uint32_t off[kLoads], chunk[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const uint32_t s = (i * NW + wave) * 64 + lane, r = s >> 2;
    chunk[i] = ((s & 3) ^ spread(r)) * 16;
    const uint32_t left = r < BC ? p.n - n0 : p.m - m0, at = r < BC ? r : r - BC;   // rows past the end repeat the last
    off[i] = (at < left ? at : left - 1) * K + chunk[i];
  }
  const uint32_t ring = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;
  // load i of step s into place s % kRing; nothing is read past the last step (zeros arrive), but every load counts
  auto send = [&](uint32_t s, int i) {
    const bool w = (i * NW + wave) * 16 < BC;   // 64 chunks are 16 rows of one operand
    u32x4 r = w ? rsrc[0] : rsrc[1];
    r[2] = s < steps ? kRange : 0;
    uint32_t o = off[i];
    if (kRagged) o = s * 64 + chunk[i] < K ? o : kOutside;
    load_lds(r, o, s * 64, ring + (s % kRing) * kStep + (i * NW + wave) * 1024);
  };

  intx4 acc[TM][TN];
#pragma unroll
  for (int r = 0; r < TM; ++r)
#pragma unroll
    for (int c = 0; c < TN; ++c) acc[r][c] = intx4{0, 0, 0, 0};
  settle(acc);

  // Row i of the MFMA's channel tiles 2q and 2q + 1 is channel 32 q + 8 (i / 4) + i % 4 and the one 4 on: the lane that
  // gets rows 4 kq .. + 3 of both has eight consecutive channels.
  const uint32_t crow = wc * WC + 8 * (l16 >> 2) + (l16 & 3), trow = BC + wt * WT + l16;
  const uint32_t cat0 = crow * 64 + (kq ^ spread(crow)) * 16, cat1 = (crow + 4) * 64 + (kq ^ spread(crow + 4)) * 16;
  const uint32_t tat = trow * 64 + (kq ^ spread(trow)) * 16;
  struct Frags {
    intx4 a[TM], b[TN];
  };
  auto read_a = [&](Frags& f, const char* at, int r) {
    f.a[r] = *reinterpret_cast<const intx4*>(at + (r & 1 ? cat1 : cat0) + (r >> 1) * 2048);
  };
  auto read_b = [&](Frags& f, const char* at, int c) { f.b[c] = *reinterpret_cast<const intx4*>(at + tat + c * 1024); };

  // step s on f, with the next step's fragments to n between its rows
  auto step = [&](uint32_t s, const Frags& f, Frags& n) {
    const char* const next = lds + ((s + 1) % kRing) * kStep;
    constexpr int kWork = kLoads + TN + TM, kPer = (kWork + TM - 1) / TM;
#pragma unroll
    for (int r = 0; r < TM; ++r) {
#pragma unroll
      for (int c = 0; c < TN; ++c) mfma_inplace(acc[r][c], f.a[r], f.b[c]);
#pragma unroll
      for (int j = r * kPer; j < (r + 1) * kPer && j < kWork; ++j) {
        // loads and reads in turn
        if (j < 2 * kLoads && j % 2 == 0) send(s + kRing, j / 2);
        else {
          const int x = j < 2 * kLoads ? j / 2 : j - kLoads;
          if (x < TN) read_b(n, next, x);
          else read_a(n, next, x - TN);
        }
      }
    }
    wait_vm_barrier<(kRing - 2) * kLoads>();
  };

  Frags f0, f1;
#pragma unroll
  for (int s = 0; s < kRing; ++s)
#pragma unroll
    for (int i = 0; i < kLoads; ++i) send(s, i);
  wait_vm_barrier<(kRing - 1) * kLoads>();
#pragma unroll
  for (int r = 0; r < TM; ++r) read_a(f0, lds, r);
#pragma unroll
  for (int c = 0; c < TN; ++c) read_b(f0, lds, c);
  wait_vm_barrier<(kRing - 2) * kLoads>();   // every wave has its fragments: the place is free
  for (uint32_t s = 0; s < steps; s += 2) {  // (a step past the last multiplies zeros)
    step(s, f0, f1);
    step(s + 1, f1, f0);
  }
  wait_vm<0>();
  settle(acc);

  auto finish = [&](auto bf16) {
    constexpr bool kBf16 = decltype(bf16)::value;
    float xs[TN];
#pragma unroll
    for (int c = 0; c < TN; ++c) {
      const uint32_t row = m0 + wt * WT + 16 * c + l16;
      xs[c] = p.xs[row < p.m ? row : p.m - 1];
    }
#pragma unroll
    for (int q = 0; q < TM / 2; ++q) {
      const uint32_t col = n0 + wc * WC + 32 * q + 8 * kq;
      if (col >= p.n) continue;
      Channels8<kBf16> ch;
      ch.load(p, col, p.n - col);
#pragma unroll
      for (int c = 0; c < TN; ++c) {
        const uint32_t row = m0 + wt * WT + 16 * c + l16;
        if (row >= p.m) continue;
        const intx4 lo = acc[2 * q][c], hi = acc[2 * q + 1][c];
        const int sums[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        ch.store(p, sums, xs[c], (size_t)row * p.n + col, p.n - col);
      }
    }
  };
  if (p.bf16) finish(std::true_type{});
  else finish(std::false_type{});
}

// ---- strips -----------------------------------------------------------------

// 16 CT channels and up to 16 TT tokens; k in pieces of 128 (two MFMAs) that the waves take in turn, kAhead of them
// on the way.
template <int CT, int TT, int WAVES, int kAhead>
__global__ void __launch_bounds__(64 * WAVES) linear8_strip_kernel(Linear8 p) {
  constexpr int kRow = 16 * CT + 4;   // ints between tokens: a wave's 16-byte writes then spread over the banks
  __shared__ int part[WAVES][16 * TT][kRow];
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), kq = lane >> 4, l16 = lane & 15;
  const uint32_t n0 = blockIdx.x * 16 * CT, K = p.k;
  const int8_t *w[CT], *x[TT];
#pragma unroll
  for (int i = 0; i < CT; ++i) w[i] = p.w + (size_t)(n0 + 16 * i + l16 < p.n ? n0 + 16 * i + l16 : p.n - 1) * K;
#pragma unroll
  for (int i = 0; i < TT; ++i) x[i] = p.x + (size_t)(16 * i + l16 < p.m ? 16 * i + l16 : p.m - 1) * K;
  struct Piece {
    intx4 w[CT][2], x[TT][2];
  } piece[kAhead];
  const uint32_t pieces = (K + 127) / 128;
  auto load = [&](Piece& v, uint32_t at) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t k = at * 128 + kq * 32 + h * 16;
      const bool in = k < K;
      const uint32_t c = in ? k : 0;
#pragma unroll
      for (int i = 0; i < TT; ++i) {   // past the end of the row: zeros for x, anything for w
        v.x[i][h] = *reinterpret_cast<const intx4*>(x[i] + c);
        if (!in) v.x[i][h] = intx4{0, 0, 0, 0};
      }
#pragma unroll
      for (int i = 0; i < CT; ++i) v.w[i][h] = *reinterpret_cast<const intx4*>(w[i] + c);
    }
  };
#pragma unroll
  for (int a = 0; a < kAhead; ++a)
    if (wave + a * WAVES < pieces) load(piece[a], wave + a * WAVES);
  intx4 acc[CT][TT] = {};
  for (uint32_t at = wave; at < pieces; at += kAhead * WAVES) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (at + a * WAVES >= pieces) break;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < CT; ++i)
#pragma unroll
          for (int j = 0; j < TT; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(piece[a].w[i][h], piece[a].x[j][h], acc[i][j], 0, 0, 0);
      if (at + (kAhead + a) * WAVES < pieces) load(piece[a], at + (kAhead + a) * WAVES);
    }
  }
#pragma unroll
  for (int i = 0; i < CT; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) *reinterpret_cast<intx4*>(&part[wave][16 * j + l16][16 * i + 4 * kq]) = acc[i][j];
  __syncthreads();
  auto finish = [&](auto bf16) {
    constexpr bool kBf16 = decltype(bf16)::value;
    for (uint32_t o = tid; o < p.m * 16 * CT; o += 64 * WAVES) {
      const uint32_t row = o / (16 * CT), c = o % (16 * CT), col = n0 + c;
      if (col >= p.n) continue;
      int sum = 0;
#pragma unroll
      for (int v = 0; v < WAVES; ++v) sum += part[v][row][c];
      const size_t at = (size_t)row * p.n + col;
      float y[1] = {__builtin_fmaf((float)sum * p.ws[col], p.xs[row], p.bias ? to_f32<kBf16>(p.bias[col]) : 0.f)};
      activations<1>(y, p.act);
      if (p.residual) y[0] += to_f32<kBf16>(p.residual[at]);
      p.y[at] = from_f32<kBf16>(y[0]);
    }
  };
  if (p.bf16) finish(std::true_type{});
  else finish(std::false_type{});
}

// k == 0: the product is zero, the epilogue remains
__global__ void __launch_bounds__(256) linear8_empty_kernel(Linear8 p) {
  const uint64_t pieces = (p.n + 7) / 8, total = p.m * pieces;
  const int zero[8] = {};
  for (uint64_t e = (uint64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (uint64_t)gridDim.x * 256) {
    const uint32_t row = (uint32_t)(e / pieces), col = (uint32_t)(e % pieces) * 8;
    auto finish = [&](auto bf16) {
      Channels8<decltype(bf16)::value> ch;
      ch.load(p, col, p.n - col);
      ch.store(p, zero, p.xs[row], (size_t)row * p.n + col, p.n - col);
    };
    if (p.bf16) finish(std::true_type{});
    else finish(std::false_type{});
  }
}

template <bool kRagged, int BC, int BT, int NWC, int NWT, int kRing>
hipError_t launch_tile_form(const Linear8& p, hipStream_t stream) {
  const uint32_t ctiles = (p.n + BC - 1) / BC, ttiles = (p.m + BT - 1) / BT;
  constexpr size_t lds = (size_t)(BC + BT) * 64 * kRing;
  auto* kern = &linear8_tile_kernel<kRagged, BC, BT, NWC, NWT, kRing>;
  static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL(kern, dim3(ctiles * ttiles), dim3(64 * NWC * NWT), lds, stream, p, ctiles, ttiles);
  return hipGetLastError();
}
template <int BC, int BT, int NWC, int NWT, int kRing>
hipError_t launch_tile(const Linear8& p, hipStream_t stream) {
  return p.k % 64 == 0 ? launch_tile_form<false, BC, BT, NWC, NWT, kRing>(p, stream)
                       : launch_tile_form<true, BC, BT, NWC, NWT, kRing>(p, stream);
}
template <int CT, int TT, int WAVES, int kAhead>
hipError_t launch_strip(const Linear8& p, hipStream_t stream) {
  hipLaunchKernelGGL((linear8_strip_kernel<CT, TT, WAVES, kAhead>), dim3((p.n + 16 * CT - 1) / (16 * CT)), dim3(64 * WAVES), 0,
                     stream, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_w8a8(const Linear8& p, hipStream_t stream) {
  if (p.k == 0) {
    const uint64_t wgs = ((uint64_t)p.m * ((p.n + 7) / 8) + 255) / 256;
    hipLaunchKernelGGL(linear8_empty_kernel, dim3((uint32_t)(wgs < 4096 ? wgs : 4096)), dim3(256), 0, stream, p);
    return hipGetLastError();
  }
  if (p.m <= 16) return launch_strip<1, 1, 8, 4>(p, stream);
  if (p.m <= 32) return launch_strip<1, 2, 8, 2>(p, stream);
  if (p.m <= 64) return launch_strip<2, 4, 8, 2>(p, stream);
  if ((uint64_t)p.m * p.n <= 512 * 4096) return launch_tile<64, 128, 2, 2, 4>(p, stream);
  return launch_tile<256, 256, 2, 4, 4>(p, stream);
}

}  // namespace kaio
