// W4A16 fused tri-output QKV projection -- split-K kernel for small m (m <= 64).
//
// Operation: kaio-candle 0.2.0, src/qkv_project_int4.rs (module doc and the
// doc comment of qkv_project_int4); same contract as the tile kernel.
//
// gfx950 design
// -------------
// At small m the 4-bit weights are almost all of the bytes: every weight must
// stream from HBM once, spread over the whole chip, so the reduction axis is
// split across the waves of a workgroup (the tile kernel's column tiles would
// leave most CUs idle).  The arithmetic intensity (~31 flop/byte at m = 8) is
// above the f32 VALU ridge, so the products still run on MFMA: x is the A
// operand in RT row tiles of 16 (rows past m repeat row m-1), the weights the
// B operand.
// * Workgroup = WAVES waves on a strip of 16*VEC columns of ONE output.  Lane
//   (kb, c) loads one VEC-word vector = the words of columns VEC*c .. VEC*c+VEC-1
//   at packed row kb of a 32-k step: each word is the B operand of VEC x RT
//   MFMAs (one per row tile), whose column c stands for output column
//   VEC*c + t.  A wave-wide load covers 4 packed rows x 64*VEC contiguous bytes.
// * Every workgroup reads the same small x.  Each wave loads its groups' x
//   rows as 256-byte row segments (4 rows per load) into a wave-private LDS
//   slice and reads its A fragments back from there; fragment-shaped loads
//   (16 rows, 64 bytes each, per load) cost ~1.5 us more per call at
//   m = 8, n = k = 4096.
// * Split-K across the waves (wave w takes groups [wG/W, (w+1)G/W)); each
//   wave streams its groups GCHUNK at a time through two register buffers,
//   the next chunk's loads in flight while the current chunk computes, or,
//   from 40 to 64 groups at m <= 8, issues all of its groups' loads at once
//   with x in LDS by direct loads.  No load sits under a branch (see the main
//   loop); a partial last strip loads clamped columns (see the body).
// * INT4 unpack once per word whatever RT is: with one row tile, in
//   nibble-interleaved k order (9 VALU ops per word) with the x fragments
//   permuted to the same order in registers; with two or more, in k order
//   (10 ops per word, values q * 2^-9, the factor returned through the scale)
//   with no permutation.
// * Per group: 4 chained MFMAs per (column set, row tile) into a fresh
//   partial, then acc += partial * scale in f32 (every product exact, as in
//   the tile kernel).
// * The wave partial sums meet in LDS and are added in a fixed order, so
//   results are deterministic; then f32 -> f16 (RNE) and row stores.
// Configurations (row tiles per wave x row blocks, columns per strip, waves)
// are chosen per m so that the register file holds two chunks plus the
// accumulators without spilling and the reduction buffer stays at 64 KiB
// (plus 68 KiB of x slices): m <= 16: 1 x 1, 64, 16 (8 x rows kept when
// m <= 8); m <= 32: 2 x 1, 64, 8; m <= 64: 2 x 2, 64, 8.  Larger m (and INT4
// from m = 33 when the group count divides by 4) runs the tile kernel, which
// unpacks each word once per tile of 64, 96 or 128 rows.

#include "w4a16_split_k.hpp"

namespace kaio {
namespace {

template <int BITS, int RT, int RSPLIT, int VEC, int WAVES, bool kFull, int XR, bool kTrim = false, int NG = 0>
__global__ void __launch_bounds__(WAVES * 64, 1)
qkv_decode_kernel(QkvProblem p, uint32_t nstrips) {
  w4a16_split_k<BITS, RT, RSPLIT, VEC, WAVES, kFull, XR, kTrim, NG>(p, nstrips);
}

// kOnlyFull: the caller guarantees n % BN == 0 (only the full-strip kernel is built)
template <int BITS, int RT, int RSPLIT, int VEC, int WAVES, int XR = 16 * RT, bool kOnlyFull = false>
hipError_t launch_split_k(const QkvProblem& p, hipStream_t stream) {
  constexpr uint32_t BN = 16 * VEC;
  const uint32_t nstrips = (p.n + BN - 1) / BN;
  const dim3 grid(3 * nstrips), block(WAVES * kWave);
  // every wave with exactly two chunks (k = 4096 at 16 waves): the straight-line path only
  constexpr uint32_t KSPLIT = WAVES / RSPLIT;
  const bool straight = p.k / kGroup == 2 * GCHUNK * KSPLIT;
  if constexpr (WAVES == 16) {
    if ((kOnlyFull || p.n % BN == 0) && !straight) {
      hipLaunchKernelGGL((qkv_decode_kernel<BITS, RT, RSPLIT, VEC, WAVES, true, XR, true>), grid, block, 0, stream,
                         p, nstrips);
      return hipGetLastError();
    }
    if constexpr (!kOnlyFull) {
      if (p.n % 4 == 0 && !straight) {
        hipLaunchKernelGGL((qkv_decode_kernel<BITS, RT, RSPLIT, VEC, WAVES, false, XR, true>), grid, block, 0,
                           stream, p, nstrips);
        return hipGetLastError();
      }
    }
  }
  if (kOnlyFull || p.n % BN == 0)
    hipLaunchKernelGGL((qkv_decode_kernel<BITS, RT, RSPLIT, VEC, WAVES, true, XR>), grid, block, 0, stream, p,
                       nstrips);
  else if constexpr (!kOnlyFull)
    hipLaunchKernelGGL((qkv_decode_kernel<BITS, RT, RSPLIT, VEC, WAVES, false, XR>), grid, block, 0, stream, p,
                       nstrips);
  return hipGetLastError();
}

// m <= 8, n % 4 == 0, 16 waves owning 3 or 4 groups each: all of a wave's
// groups in flight, x through direct LDS loads
template <int NG>
hipError_t launch_all_groups(const QkvProblem& p, hipStream_t stream) {
  const uint32_t nstrips = (p.n + 63) / 64;
  if (p.n % 64 == 0)
    hipLaunchKernelGGL((qkv_decode_kernel<4, 1, 1, 4, 16, true, 8, false, NG>), dim3(3 * nstrips),
                       dim3(16 * kWave), 0, stream, p, nstrips);
  else
    hipLaunchKernelGGL((qkv_decode_kernel<4, 1, 1, 4, 16, false, 8, false, NG>), dim3(3 * nstrips),
                       dim3(16 * kWave), 0, stream, p, nstrips);
  return hipGetLastError();
}

template <int BITS>
hipError_t launch_decode_bits(const QkvProblem& p, hipStream_t stream) {
  if constexpr (BITS == 4) {
    // It pays once the 16 waves own 2.5 groups or more on average (m = 8,
    // n = 4096: k = 5120 11.9 -> 11.1 us, 6144 12.7 -> 11.6, 8192 15.1 ->
    // 14.7); from 33 to 39 groups most waves own two and it gains nothing.
    const uint32_t groups = p.k / kGroup;
    if (p.m <= 8 && p.n % 4 == 0 && groups >= 40 && groups <= 64)
      return groups <= 48 ? launch_all_groups<3>(p, stream) : launch_all_groups<4>(p, stream);
  }
  // INT8 words are twice the registers per group: 16-wave workgroups fit
  // (128 VGPRs, buffer loads) only with full strips at m <= 8; otherwise INT8
  // keeps the 8-wave register budget (each wave then streams four groups).
  // m = 8, n = k = 4096: 12.66 us at 8 waves, 11.57 at 16.
  if (BITS == 8 && p.m <= 8 && p.n % 64 == 0) return launch_split_k<BITS, 1, 1, 4, 16, 8, true>(p, stream);
  constexpr int kSmallWaves = BITS == 8 ? 8 : 16;
  if (p.m <= 8) return launch_split_k<BITS, 1, 1, 4, kSmallWaves, 8>(p, stream);
  if (p.m <= 16) return launch_split_k<BITS, 1, 1, 4, kSmallWaves>(p, stream);
  if (p.m <= 32) return launch_split_k<BITS, 2, 1, 4, 8>(p, stream);
  return launch_split_k<BITS, KAIO_SK4_RT, 4 / KAIO_SK4_RT, KAIO_SK4_VEC, KAIO_SK4_WAVES>(p, stream);
}

}  // namespace

hipError_t launch_qkv_decode(const QkvProblem& p, hipStream_t stream) {
  static_assert(kDecodeMaxM <= 64, "the widest configuration covers 64 rows");
  static_assert(decode_bn(16) == 64 && decode_bn(32) == 64 && decode_bn(64) == 16 * KAIO_SK4_VEC,
                "strip widths must match the host-side grid computation");
  return p.bits == 8 ? launch_decode_bits<8>(p, stream) : launch_decode_bits<4>(p, stream);
}

}  // namespace kaio
