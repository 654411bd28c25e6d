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
// LDS.  Up to 8 tokens are rounded there too (linear8_rounds).
//
// Bound: up to some 100 tokens by the weights' way from HBM, 1 byte each; where
// there are a few thousand rows on both sides by the matrix cores, and at 8192 x
// 12288 by the power that the card allows them (2.4 to 2.5e15 operations/s in
// long runs; MFMAs alone without loads reach 3.0 to 3.4e15).  In between a
// compute unit waits for its own blocks.  Measured (16-bit x, rounding included;
// m x n x k; weights from HBM, in brackets where the 256 MB cache before it keeps
// them): 1 x 4096 x 4096 6.7 us (6.2), 1 x 4096 x 8192 10.1, 1 x 11004 x 4096 15.6,
// 61 x 11004 x 4096 19.6 (14.1), 64 x 512 x 8192 12.5, 509 x 4096 x 4096 26 (22 to
// 23.4), of which rounding 5, 2048 x 4096 x 8192 (77 to 81), of which rounding 10
// (tiles 2.0e15 operations/s), 8192 x 12288 x 4096 (319 to 346, by box).
//
// Results leave by nontemporal stores (plain ones: 413 instead of 381 us for the
// last of these, in an earlier form), so that they push no operands out of the L2.

#include "attention_common.hpp"
#include "common.hpp"
#include "epilogue.hpp"
#include "launch.hpp"
#include "paged.hpp"
#include "rounding.hpp"

#include <type_traits>

namespace kaio {
namespace {

typedef int intx4 __attribute__((ext_vector_type(4)));
typedef uint16_t ushort8_t __attribute__((ext_vector_type(8), aligned(2)));   // eight results, wherever a row begins

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
  // of scales and biases (or null), 16-byte aligned, the first `n`
  __device__ __forceinline__ void load(const float* s, const uint16_t* b, uint32_t n) {
    if (n >= 8) {
      const floatx4 lo = *reinterpret_cast<const floatx4*>(s), hi = *reinterpret_cast<const floatx4*>(s + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) ws[e] = e < 4 ? lo[e & 3] : hi[e & 3];
    } else {
#pragma unroll
      for (uint32_t e = 0; e < 8; ++e) ws[e] = e < n ? s[e] : 0.f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) bias[e] = 0.f;
    if (b) fetch(b, n, bias);
  }
  __device__ __forceinline__ void store(const Linear8& p, const int (&acc)[8], float xs, size_t at, uint32_t n) const {
    float y[8], r[8] = {};
    if (p.residual) fetch(p.residual + at, n, r);
    // the channel's scale first: what is out of f32's range after the token's is so in the result
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf((float)acc[e] * ws[e], xs, bias[e]);
    activations<8>(y, p.act);
    ushort8_t out;
#pragma unroll
    for (int e = 0; e < 8; ++e) out[e] = from_f32<kBf16>(y[e] + r[e]);
    uint16_t* const dst = p.y + at;
    if (n >= 8) {
      // past the caches: written back by them, a tile's results held up the next one's operands (8192 x 12288 x 4096 413 ->
      // 381 us)
      __builtin_nontemporal_store(out, reinterpret_cast<ushort8_t*>(dst));
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

// Raw buffer of `bytes`: what lies past them is read as zeros.
__device__ __forceinline__ u32x4 buffer(const void* a, uint32_t bytes) {
  const uint64_t b = reinterpret_cast<uint64_t>(a);
  return u32x4{(uint32_t)b, (uint32_t)(b >> 32) & 0xFFFFu, bytes, 0x00020000u};
}
// Direct load to LDS of 16 bytes per lane: from rsrc's base + soff + the lane's offset to lds + 16 * lane.  (See dma in
// attention_common.hpp for the form and its wait states.)
__device__ __forceinline__ void load_lds(u32x4 rsrc, uint32_t off, uint32_t soff, uint32_t lds) {
  asm("" : "+s"(soff));   // in a register: a literal is no operand there
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(off), "s"(rsrc), "s"(soff) : "m0");
}

// Places of 16-byte chunks in a block's rows of 128 bytes: chunk c of row r in slot 8 r + (c ^ spread(r)).  A fragment read
// is served 8 lanes at a time over 128 bytes of banks: both 8 consecutive rows (tokens) and rows 0-3 and 8-11 of 16
// (channels) then lie apart.
__device__ __forceinline__ uint32_t spread(uint32_t r) { return (r & 7) ^ (((r >> 3) & 1) * 4); }

// A tile's scales and biases in LDS.
template <int BC, int BT>
struct TileScales {
  static constexpr uint32_t kWs = 0, kXs = 4 * BC, kBias = 4 * (BC + BT), kBytes = 6 * BC + 4 * BT;
};

// BC channels by BT tokens by KS sets of NWC x NWT waves; kRagged: k % 128 != 0 (a chunk past k is then read as zeros, by an
// offset outside of the descriptor's range).
//
// Blocks are 128 k of the tile's rows, whole cache lines (by 64 k, half a line at a time, lines came twice: 1.3 times the
// time).  They arrive in a ring of kRing steps.
//
// KS 1: a wave takes both halves of a block in turn, the second half's fragments read under the first half's MFMAs, the
// next block's first under the second's; the one barrier in between says that this block is read and the next one there.
// A workgroup takes tiles one after the other without a pause in its loads: the last blocks of a tile send for the first
// ones of the next, which arrive while the tile is finished.
//
// Where tiles are small, a block is short against what it waits for, and KS sets of waves share out k: each takes one
// half of KS / 2 blocks, and their sums are added in LDS.  Those take one tile per workgroup.
template <bool kRagged, int BC, int BT, int NWC, int NWT, int KS, int kRing>
__global__ void __launch_bounds__(64 * NWC * NWT * KS, 1) linear8_tile_kernel(Linear8 p, uint32_t ctiles, uint32_t ttiles) {
  constexpr int NW = NWC * NWT, WC = BC / NWC, WT = BT / NWT, TM = WC / 16, TN = WT / 16;
  constexpr int kPairs = KS > 1 ? KS / 2 : 1, kSenders = KS > 1 ? 2 * NW : NW;   // blocks of a step, waves that send for one
  constexpr int kLoadsW = BC * 8 / (64 * kSenders), kLoads = kLoadsW + BT * 8 / (64 * kSenders);   // of a wave, per step
  constexpr uint32_t kBlock = (BC + BT) * 128, kStep = kPairs * kBlock;   // bytes
  static_assert(TM % 2 == 0 && BC * 8 % (64 * kSenders) == 0 && BT * 8 % (64 * kSenders) == 0 && BC <= 256 && BT <= 256 &&
                    NW * KS >= 4 && (KS == 1 || KS % 2 == 0) && kRing >= 2, "tile");
  static_assert(KS == 1 || (KS - 1) * BC * BT * 4 <= kRing * kStep, "the sums of the other sets fit in the ring");
  using Scales = TileScales<BC, BT>;
  extern __shared__ __attribute__((aligned(16))) char lds[];   // the ring, then the scales of two tiles
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave_id = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t set = KS == 1 ? 0 : wave_id / NW, wave = KS == 1 ? wave_id : wave_id % NW;
  const uint32_t pair = set / 2, sender = KS == 1 ? wave : set % 2 * NW + wave;
  const uint32_t kq = lane >> 4, l16 = lane & 15, wc = wave / NWT, wt = wave % NWT;
  const uint32_t K = p.k, blocks = (K + 127) / 128;
  // steps of a tile; with sets an even number (past the end zeros are added)
  const uint32_t steps = KS == 1 ? blocks : (blocks + 2 * kPairs - 1) / (2 * kPairs) * 2;
  const uint32_t tiles = ctiles * ttiles;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;

  // Tiles in bands of 4 tiles of tokens, channel by channel: what runs at a time on an XCD shares rows of both operands.
  auto place = [&](uint32_t v, uint32_t& m0, uint32_t& n0) {
    const uint32_t id = xcd_remap(v, tiles), band = id / (4 * ctiles), in = id - band * 4 * ctiles;
    const uint32_t high = ttiles - 4 * band < 4 ? ttiles - 4 * band : 4;
    m0 = (4 * band + in % high) * BT;
    n0 = in / high * BC;
  };

  // What is sent for: step `at` of a tile.
  constexpr uint32_t kRange = 0x7FFFFFF0u, kOutside = 0x80000000u;
  uint32_t load_tile = blockIdx.x, at = 0;
  const int8_t *base_w = p.w, *base_x = p.x;
  uint32_t range = 0;
  uint32_t off[kLoads], chunk[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const uint32_t s = ((i - (i < kLoadsW ? 0 : kLoadsW)) * kSenders + sender) * 64 + lane;
    chunk[i] = ((s & 7) ^ spread(s >> 3)) * 16;
  }
  auto aim = [&] {   // at the first step of load_tile; past the last tile at nothing
    at = 0;
    if (load_tile >= tiles) {
      range = 0;
      return;
    }
    uint32_t m0, n0;
    place(load_tile, m0, n0);
    range = kRange;
    base_w = p.w + (size_t)n0 * K;
    base_x = p.x + (size_t)m0 * K;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const bool w = i < kLoadsW;
      const uint32_t row = (((i - (w ? 0 : kLoadsW)) * kSenders + sender) * 64 + lane) >> 3;
      const uint32_t left = w ? p.n - n0 : p.m - m0;   // rows past the end repeat the last
      off[i] = (row < left ? row : left - 1) * K + chunk[i];
    }
  };
  // load i of that step into `to`, nothing past the tile's sum: zeros arrive, but every load counts
  auto send = [&](uint32_t to, int i) {
    uint32_t o = off[i];
    const uint32_t k = (at * kPairs + pair) * 128;
    if (kRagged) o = k + chunk[i] < K ? o : kOutside;
    const u32x4 r = buffer(i < kLoadsW ? base_w : base_x, kRagged || k < K ? range : 0);
    load_lds(r, o, k, to + (i < kLoadsW ? i * kSenders + sender : BC / 8 + (i - kLoadsW) * kSenders + sender) * 1024);
  };
  auto sent = [&] {   // the whole step
    if (++at == steps) {
      load_tile += gridDim.x;
      aim();
    }
  };

  // Row i of the MFMA's channel tiles 2q and 2q + 1 is channel 32 q + 8 (i / 4) + i % 4 and the one 4 on: the lane that
  // gets rows 4 kq .. + 3 of both has eight consecutive channels.  Offsets in the first half of a block; those of the
  // second differ in bit 6.
  const uint32_t crow = wc * WC + 8 * (l16 >> 2) + (l16 & 3), trow = BC + wt * WT + l16;
  const uint32_t cat0 = crow * 128 + (kq ^ spread(crow)) * 16, cat1 = (crow + 4) * 128 + (kq ^ spread(crow + 4)) * 16;
  const uint32_t tat = trow * 128 + (kq ^ spread(trow)) * 16;
  struct Frags {
    intx4 a[TM], b[TN];
  };
  auto read_one = [&](Frags& f, const char* from, uint32_t half, int x) {   // x: first the tokens' fragments
    if (x < TN) f.b[x] = *reinterpret_cast<const intx4*>(from + (tat ^ half * 64) + x * 2048);
    else f.a[x - TN] = *reinterpret_cast<const intx4*>(from + (((x - TN) & 1 ? cat1 : cat0) ^ half * 64) + ((x - TN) >> 1) * 4096);
  };
  auto read = [&](Frags& f, const char* from, uint32_t half) {
#pragma unroll
    for (int x = 0; x < TN + TM; ++x) read_one(f, from, half, x);
  };

  intx4 acc[TM][TN];
  auto clear = [&] {
#pragma unroll
    for (int r = 0; r < TM; ++r)
#pragma unroll
      for (int c = 0; c < TN; ++c) acc[r][c] = intx4{0, 0, 0, 0};
    settle(acc);
  };
  // MFMAs on f; between their rows the reads of n and, with kSend, the loads of a step into `to`, in turn
  auto multiply = [&](auto kSend, const Frags& f, Frags& n, const char* from, uint32_t half, uint32_t to) {
    constexpr int kS = decltype(kSend)::value ? kLoads : 0, kWork = kS + TN + TM, kPer = (kWork + TM - 1) / TM;
    constexpr int kTurns = kS < TN + TM ? kS : TN + TM;
#pragma unroll
    for (int r = 0; r < TM; ++r) {
#pragma unroll
      for (int c = 0; c < TN; ++c) mfma_inplace(acc[r][c], f.a[r], f.b[c]);
#pragma unroll
      for (int j = r * kPer; j < (r + 1) * kPer && j < kWork; ++j) {
        if (j < 2 * kTurns) {
          if (j % 2 == 0) send(to, j / 2);
          else read_one(n, from, half, j / 2);
        } else if (kS > TN + TM) {
          send(to, j - kTurns);
        } else {
          read_one(n, from, half, j - kTurns);
        }
      }
    }
    if (decltype(kSend)::value) sent();
  };
  using Yes = std::true_type;
  using No = std::false_type;
  // everything sent for but the last kLeft steps is there, for every wave, and what was read is; landed: all of it is known
  // to be there
  auto meet = [&](auto kLeft, bool landed) {
    if (landed) {
      wait_lds<0>();
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    } else {
      wait_vm_barrier<decltype(kLeft)::value * kLoads>();
    }
  };
  constexpr auto kAllButOne = std::integral_constant<int, kRing - 1>{};
  constexpr auto kAllButTwo = std::integral_constant<int, kRing - 2>{};
  uint32_t here = 0;   // the step's place in the ring
  auto next = [&] { return here + kStep == kRing * kStep ? 0 : here + kStep; };
  const char* const mine = lds + pair * kBlock;
  const uint32_t ring = lds0 + pair * kBlock, half = set % 2;

  // scales and bias of a tile, one load by each of three waves (zeros past the ends of the arrays)
  auto send_scales = [&](uint32_t to, uint32_t m0, uint32_t n0) {
    if (wave_id == 0 && lane * 4 < BC) load_lds(buffer(p.ws, 4 * p.n), n0 * 4 + lane * 16, 0, to + Scales::kWs);
    if (wave_id == 1 && lane * 4 < BT) load_lds(buffer(p.xs, 4 * p.m), m0 * 4 + lane * 16, 0, to + Scales::kXs);
    if (wave_id == 2 && p.bias && lane * 8 < BC) load_lds(buffer(p.bias, 2 * p.n), n0 * 2 + lane * 16, 0, to + Scales::kBias);
  };
  auto finish = [&](auto bf16, uint32_t m0, uint32_t n0, const char* scales) {
    constexpr bool kBf16 = decltype(bf16)::value;
    float xs[TN];
#pragma unroll
    for (int c = 0; c < TN; ++c) xs[c] = reinterpret_cast<const float*>(scales + Scales::kXs)[wt * WT + 16 * c + l16];
#pragma unroll
    for (int q = 0; q < TM / 2; ++q) {
      const uint32_t in = wc * WC + 32 * q + 8 * kq, col = n0 + in;
      if (col >= p.n) continue;
      Channels8<kBf16> ch;
      if (col + 8 <= p.n)
        ch.load(reinterpret_cast<const float*>(scales + Scales::kWs) + in,
                p.bias ? reinterpret_cast<const uint16_t*>(scales + Scales::kBias) + in : nullptr, 8);
      else   // (a load by dwords leaves out the last of an odd number of biases)
        ch.load(p.ws + col, p.bias ? p.bias + col : nullptr, p.n - col);
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

  Frags f0, f1;
  clear();
  aim();
#pragma unroll
  for (int s = 0; s < kRing; ++s) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) send(ring + s * kStep, i);
    sent();
  }
  meet(kAllButOne, false);
  read(f0, mine, half);
  if (KS > 1) meet(kAllButTwo, false);   // every wave has its fragments: the place is free, and the next step there
  uint32_t flip = 0;
  for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x, flip ^= 1) {
    uint32_t m0, n0;
    place(tile, m0, n0);
    // (the other place than the tile before, which a slower wave may still be finishing)
    send_scales(lds0 + kRing * kStep + flip * Scales::kBytes, m0, n0);
    if constexpr (KS == 1) {
      // After a tile every load of the ring has landed: its first steps wait for none, and so not for the tile's stores.
      const uint32_t landed = tile == blockIdx.x ? 0 : kRing - 1;
      for (uint32_t s = 0; s < steps; ++s) {
        multiply(No{}, f0, f1, lds + here, 1, 0);
        meet(kAllButTwo, s < landed);
        const uint32_t to = lds0 + here;
        here = next();
        multiply(Yes{}, f1, f0, lds + here, 0, to);
      }
    } else {
      for (uint32_t s = 0; s < steps; s += 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t to = ring + here;
          here = next();
          multiply(Yes{}, h ? f1 : f0, h ? f0 : f1, mine + here, half, to);
          meet(kAllButTwo, false);
        }
      }
    }
    wait_vm<0>();   // the ring's loads and the scales
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    settle(acc);
    if constexpr (KS > 1) {
      // [set - 1][tile r, c][wave][lane] of four sums
      intx4* const sums = reinterpret_cast<intx4*>(lds) + wave * 64 + lane;
      if (set) {
#pragma unroll
        for (int r = 0; r < TM; ++r)
#pragma unroll
          for (int c = 0; c < TN; ++c) sums[(((set - 1) * TM + r) * TN + c) * NW * 64] = acc[r][c];
      }
      __syncthreads();
      if (set) return;
#pragma unroll
      for (int r = 0; r < TM; ++r)
#pragma unroll
        for (int c = 0; c < TN; ++c)
#pragma unroll
          for (int o = 0; o < KS - 1; ++o) acc[r][c] += sums[((o * TM + r) * TN + c) * NW * 64];
    }
    const char* const scales = lds + kRing * kStep + flip * Scales::kBytes;
    if (p.bf16) finish(std::true_type{}, m0, n0, scales);
    else finish(std::false_type{}, m0, n0, scales);
    if constexpr (KS > 1) return;
    clear();
    read(f0, mine + here, 0);   // again: the tile's end has use for the registers
  }
  wait_vm<0>();
}

// ---- strips -----------------------------------------------------------------

// What the waves of a workgroup wrote to LDS is there; loads in flight stay there.
__device__ __forceinline__ void meet_lds() {
  wait_lds<0>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// The rounded rows of up to 8 tokens in LDS, rows of p.k bytes and zeros to the next multiple of 128, `stride` apart, with
// their scales.  Made from 16-bit rows by the whole workgroup, kHeld pieces of 16 elements per thread at a time.
template <bool kBf16, int kThreads, int kHeld>
struct RoundedRows {
  uint4 v[kHeld][2];
  uint32_t per_row, total;   // pieces
  __device__ __forceinline__ void load(const Linear8& p) {
    per_row = p.k / 16;
    total = p.m * per_row;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const uint32_t at = threadIdx.x + i * kThreads;
      v[i][0] = v[i][1] = uint4{0, 0, 0, 0};
      if (at < total) {
        v[i][0] = reinterpret_cast<const uint4*>(p.x16)[2 * at];
        v[i][1] = reinterpret_cast<const uint4*>(p.x16)[2 * at + 1];
      }
    }
  }
  __device__ __forceinline__ void store(const Linear8& p, char* rows, uint32_t stride, uint32_t* most, float* scale) {
    const uint32_t tid = threadIdx.x;
    if (tid < 16) most[tid] = 0;
    meet_lds();
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const uint32_t at = tid + i * kThreads, row = at / per_row;
      uint32_t a = max_bits(max_bits(0u, v[i][0]), v[i][1]);
      a = (a >> 16) > (a & 0xFFFFu) ? a >> 16 : a & 0xFFFFu;
      if (__all(row == (uint32_t)__builtin_amdgcn_readfirstlane(row))) {   // a wave inside one row: one maximum of it
#pragma unroll
        for (int s = 32; s; s >>= 1) {
          const uint32_t o = (uint32_t)__shfl_xor((int)a, s);
          a = a > o ? a : o;
        }
        if (tid % 64 == 0 && at < total) atomicMax(&most[row], a);
      } else if (at < total) {
        atomicMax(&most[row], a);
      }
    }
    meet_lds();
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const uint32_t at = tid + i * kThreads, row = at / per_row;
      if (at < total)
        *reinterpret_cast<uint4*>(rows + row * stride + (at - row * per_row) * 16) =
            Rounding::of<kBf16>(most[row]).template sixteen<kBf16>(v[i][0], v[i][1]);
    }
    const uint32_t tail = (8 - per_row % 8) % 8;
    if (tid < p.m * tail) *reinterpret_cast<uint4*>(rows + tid / tail * stride + (per_row + tid % tail) * 16) = uint4{0, 0, 0, 0};
    if (tid < p.m) scale[tid] = Rounding::scale<kBf16>(most[tid]);
    meet_lds();
  }
};

// 16 channels and up to 16 tokens; k in pieces of 128 (two MFMAs) that the waves take in turn, kAhead of them on the way.
// Rounds (p.x16): 16-bit tokens are rounded here, by every workgroup, while the first weights are on the way.
template <bool kRounds, bool kBf16, int WAVES, int kAhead>
__global__ void __launch_bounds__(64 * WAVES) linear8_strip_kernel(Linear8 p) {
  __shared__ int part[WAVES][16][20];   // (20: a wave's 16-byte writes spread over the banks)
  __shared__ uint32_t most[16];
  __shared__ float scale[16];
  extern __shared__ __attribute__((aligned(16))) char rows[];
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), kq = lane >> 4, l16 = lane & 15;
  const uint32_t n0 = blockIdx.x * 16, K = p.k, pieces = (K + 127) / 128, stride = pieces * 128 + 16;
  const uint32_t channel = n0 + l16 < p.n ? n0 + l16 : p.n - 1, token = l16 < p.m ? l16 : p.m - 1;   // past the end: the last
  const int8_t* const w = p.w + (size_t)channel * K;
  const int8_t* const x = kRounds ? nullptr : p.x + (size_t)token * K;
  RoundedRows<kBf16, 64 * WAVES, kLinear8Round / 16 / (64 * WAVES)> rounded;
  if constexpr (kRounds) rounded.load(p);
  struct Piece {
    intx4 w[2], x[2];
  } piece[kAhead];
  auto load = [&](Piece& v, uint32_t at) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t k = at * 128 + kq * 32 + h * 16;
      const bool in = k < K;
      if constexpr (!kRounds) {   // past the end of the row: zeros for x, anything for w
        v.x[h] = *reinterpret_cast<const intx4*>(x + (in ? k : 0));
        if (!in) v.x[h] = intx4{0, 0, 0, 0};
      }
      v.w[h] = *reinterpret_cast<const intx4*>(w + (in ? k : 0));
    }
  };
#pragma unroll
  for (int a = 0; a < kAhead; ++a)
    if (wave + a * WAVES < pieces) load(piece[a], wave + a * WAVES);
  if constexpr (kRounds) rounded.store(p, rows, stride, most, scale);
  intx4 acc = {};
  for (uint32_t at = wave; at < pieces; at += kAhead * WAVES) {
#pragma unroll
    for (int a = 0; a < kAhead; ++a) {
      if (at + a * WAVES >= pieces) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (kRounds)
          piece[a].x[h] = *reinterpret_cast<const intx4*>(rows + token * stride + (at + a * WAVES) * 128 + kq * 32 + h * 16);
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(piece[a].w[h], piece[a].x[h], acc, 0, 0, 0);
      }
      if (at + (kAhead + a) * WAVES < pieces) load(piece[a], at + (kAhead + a) * WAVES);
    }
  }
  *reinterpret_cast<intx4*>(&part[wave][l16][4 * kq]) = acc;
  __syncthreads();
  for (uint32_t o = tid; o < p.m * 16; o += 64 * WAVES) {
    const uint32_t row = o / 16, c = o % 16, col = n0 + c;
    if (col >= p.n) continue;
    int sum = 0;
#pragma unroll
    for (int v = 0; v < WAVES; ++v) sum += part[v][row][c];
    const size_t at = (size_t)row * p.n + col;
    const float xs = kRounds ? scale[row] : p.xs[row];
    float y[1] = {__builtin_fmaf((float)sum * p.ws[col], xs, p.bias ? to_f32<kBf16>(p.bias[col]) : 0.f)};
    activations<1>(y, p.act);
    if (p.residual) y[0] += to_f32<kBf16>(p.residual[at]);
    p.y[at] = from_f32<kBf16>(y[0]);
  }
}

// k == 0: the product is zero, the epilogue remains
__global__ void __launch_bounds__(256) linear8_empty_kernel(Linear8 p) {
  const uint64_t pieces = (p.n + 7) / 8, total = p.m * pieces;
  const int zero[8] = {};
  for (uint64_t e = (uint64_t)blockIdx.x * 256 + threadIdx.x; e < total; e += (uint64_t)gridDim.x * 256) {
    const uint32_t row = (uint32_t)(e / pieces), col = (uint32_t)(e % pieces) * 8;
    auto finish = [&](auto bf16) {
      Channels8<decltype(bf16)::value> ch;
      ch.load(p.ws + col, p.bias ? p.bias + col : nullptr, p.n - col);
      ch.store(p, zero, p.xs ? p.xs[row] : 0.f, (size_t)row * p.n + col, p.n - col);
    };
    if (p.bf16) finish(std::true_type{});
    else finish(std::false_type{});
  }
}

template <bool kRagged, int BC, int BT, int NWC, int NWT, int KS, int kRing>
hipError_t launch_tile_form(const Linear8& p, hipStream_t stream) {
  const uint32_t ctiles = (p.n + BC - 1) / BC, ttiles = (p.m + BT - 1) / BT;
  constexpr size_t lds = (size_t)(BC + BT) * 128 * (KS > 1 ? KS / 2 : 1) * kRing + 2 * TileScales<BC, BT>::kBytes;
  // as many workgroups as the compute units hold at a time
  const uint64_t tiles = (uint64_t)ctiles * ttiles, most = KS > 1 ? tiles : (160u << 10) / lds * kComputeUnits;
  auto* kern = &linear8_tile_kernel<kRagged, BC, BT, NWC, NWT, KS, kRing>;
  static LdsOf of;
  if (hipError_t e = of.allow(reinterpret_cast<const void*>(kern), (int)lds)) return e;
  hipLaunchKernelGGL(kern, dim3((uint32_t)(tiles < most ? tiles : most)), dim3(64 * NWC * NWT * KS), lds, stream, p, ctiles, ttiles);
  return hipGetLastError();
}
template <int BC, int BT, int NWC, int NWT, int KS, int kRing>
hipError_t launch_tile(const Linear8& p, hipStream_t stream) {
  return p.k % 128 == 0 ? launch_tile_form<false, BC, BT, NWC, NWT, KS, kRing>(p, stream)
                       : launch_tile_form<true, BC, BT, NWC, NWT, KS, kRing>(p, stream);
}
template <bool kRounds, int WAVES, int kAhead>
hipError_t launch_strip(const Linear8& p, hipStream_t stream) {
  const size_t lds = kRounds ? (size_t)p.m * ((p.k + 127) / 128 * 128 + 16) : 0;
  constexpr int most = (int)(kLinear8Round + 8 * (128 + 16));
  auto go = [&](auto* kern, LdsOf& of) {
    if (hipError_t e = of.allow(reinterpret_cast<const void*>(kern), most)) return e;
    hipLaunchKernelGGL(kern, dim3((p.n + 15) / 16), dim3(64 * WAVES), lds, stream, p);
    return hipGetLastError();
  };
  static LdsOf bf16, f16;
  return p.bf16 ? go(&linear8_strip_kernel<kRounds, true, WAVES, kAhead>, bf16) : go(&linear8_strip_kernel<kRounds, false, WAVES, kAhead>, f16);
}

hipError_t launch_form(const Linear8& p, Linear8Form f, hipStream_t stream) {
  switch (f) {
    case kStrip16: return p.x16 ? launch_strip<true, 16, 2>(p, stream) : launch_strip<false, 16, 2>(p, stream);
    case kStrip4: return launch_strip<false, 4, 8>(p, stream);
    case kTile32x32: return launch_tile<32, 32, 1, 1, 4, 4>(p, stream);
    case kTile32x64: return launch_tile<32, 64, 1, 2, 4, 4>(p, stream);
    case kTile64x32: return launch_tile<64, 32, 1, 1, 4, 4>(p, stream);
    case kTile64x64: return launch_tile<64, 64, 2, 2, 2, 4>(p, stream);
    case kTile64x128: return launch_tile<64, 128, 1, 4, 2, 4>(p, stream);
    case kTile128x128: return launch_tile<128, 128, 2, 4, 1, 4>(p, stream);
    case kTile128x256: return launch_tile<128, 256, 2, 4, 1, 3>(p, stream);
    case kTile256x256: return launch_tile<256, 256, 2, 4, 1, 2>(p, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_linear_w8a8(const Linear8& p, hipStream_t stream) {
  if (p.k == 0) {
    const uint64_t wgs = ((uint64_t)p.m * ((p.n + 7) / 8) + 255) / 256;
    hipLaunchKernelGGL(linear8_empty_kernel, dim3((uint32_t)(wgs < 4096 ? wgs : 4096)), dim3(256), 0, stream, p);
    return hipGetLastError();
  }
  return launch_form(p, linear8_form(p.m, p.n), stream);
}

}  // namespace kaio
