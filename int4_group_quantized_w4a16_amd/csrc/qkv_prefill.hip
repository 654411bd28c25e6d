// W4A16 fused tri-output QKV projection -- MFMA tile kernel (m > 64; INT4 from
// m > 32 when the group count divides by 4).
//
// Operation: kaio-candle 0.2.0, src/qkv_project_int4.rs (module doc and the
// doc comment of qkv_project_int4): one launch computes Q, K and V f16[M,N]
// from a shared f16 x[M,K], three packed-INT4 u32[K/8,N] weights and three
// f16[K/128,N] group scales, accumulating in f32.
//
// gfx950 design
// -------------
// * Workgroup = WAVES waves, tile = BM (128, 96 or 64 for small grids) rows
//   of x by 16*WAVES columns of EACH output.  Wave w owns columns
//   [16w, 16w+16) of all three outputs and all BM rows, so the waves share
//   one x tile in LDS and never unpack the same weight twice.  Small grids
//   of 4-wave tiles run two (or four) such sets of waves per workgroup, each
//   over its share of the groups with its own ring, their sums added in LDS
//   at the end; the smallest grids compute one output per workgroup.
// * Everything a group of 128 k needs is staged into LDS rings with direct
//   global->LDS loads (no registers, no VALU): x and the packed weights one
//   group ahead, the scales 32 (or 8) groups at a time.  Each address is a
//   wave-uniform base in SGPRs plus a 32-bit lane offset.  One barrier per
//   group; the only waits on the vector-memory counter are explicit.
// * x: chunk kc of row r lands in slot r*16 + (kc ^ (r & 15)), which makes
//   the MFMA A-operand reads bank-conflict free.  A fragments are read two
//   row tiles ahead of the MFMAs that use them.
// * Weights: one u32 holds the eight consecutive k of one column that a lane
//   feeds to one v_mfma_f32_16x16x32_f16 as its B operand.  Each wave fetches
//   the 16 packed rows x 16 columns it multiplies (one 16-byte load per lane
//   and output when n % 8 == 0), reads its words back and unpacks them to
//   exact f16 values q * 2^-9 in registers (10 VALU ops per word) -- during
//   the last two row tiles of the previous group, so that the unpack
//   overlaps MFMAs; the epilogue takes the factor 2^-9 back, exactly.
// * Scales are applied per group in f32: the four MFMAs of a group
//   accumulate a fresh partial sum of x*q*2^-9 (exact small integers, scaled
//   by a power of two, times f16 activations), then
//   acc += partial * scale (the f16 scale converted inside the FMA;
//   the accumulators hold 2^-9 times the result until the epilogue's
//   exact multiply by 512).  Rounding q*scale to f16
//   before the MFMA would cost up to 2^-12 relative per product, too much
//   for the f16 output; the partial/scale split keeps every product exact.
// * Epilogue: f32 -> f16 (RNE), transposed through LDS one output at a time
//   (unpadded rows, columns swizzled per 4-row group), 16-byte row stores.

#include "w4a16_tile.hpp"

namespace kaio {
namespace {

template <int BITS, int WAVES, int XDIST, bool kAligned, int BM, int KS, int NQ>
__global__ void __launch_bounds__(KS * WAVES * 64, 1)
qkv_prefill_kernel(QkvProblem p, uint32_t mtiles) {
  w4a16_tile<BITS, WAVES, XDIST, kAligned, BM, KS, NQ>(p, mtiles);
}

template <int BITS, int WAVES, int XDIST, bool kAligned, int BM, int KS, int NQ>
hipError_t launch_variant(const QkvProblem& p, hipStream_t stream) {
  constexpr int BN = 16 * WAVES;
  const uint32_t mtiles = (p.m + BM - 1) / BM;
  const uint32_t ntiles = (p.n + BN - 1) / BN;
  const size_t lds = (size_t)KS * SetRing<BITS, WAVES, XDIST, BM, KS, NQ>::kSize * 16;
  const dim3 grid(mtiles * ntiles * (NQ == 1 ? 3 : 1)), block(KS * WAVES * 64);
  auto* kern = &qkv_prefill_kernel<BITS, WAVES, XDIST, kAligned, BM, KS, NQ>;
  static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL(kern, grid, block, lds, stream, p, mtiles);
  return hipGetLastError();
}

template <int BITS, int WAVES, int BM, int KS, int NQ = 3>
hipError_t launch_aligned_or_not(const QkvProblem& p, hipStream_t stream) {
  // 16-byte output rows and f16-pair scale loads need n % 8 == 0
  return p.n % 8 == 0 ? launch_variant<BITS, WAVES, KAIO_PREFILL_XDIST, true, BM, KS, NQ>(p, stream)
                      : launch_variant<BITS, WAVES, KAIO_PREFILL_XDIST, false, BM, KS, NQ>(p, stream);
}

constexpr uint32_t form_code(PrefillForm f) { return ((f.waves * 1000 + f.bm) * 10 + f.sets) * 10 + f.outs; }

// the form tile_form() picks for this problem
template <int BITS>
hipError_t launch_prefill_bits(const QkvProblem& p, hipStream_t stream) {
  switch (form_code(tile_form(p.m, p.n, p.k, BITS))) {
    case form_code({8, 128, 1, 3}): return launch_aligned_or_not<BITS, 8, 128, 1>(p, stream);
    case form_code({8, 96, 1, 3}): return launch_aligned_or_not<BITS, 8, 96, 1>(p, stream);
    case form_code({4, 128, 2, 3}):
      if constexpr (BITS == 4) return launch_aligned_or_not<BITS, 4, 128, 2>(p, stream);
      break;
    case form_code({4, 96, 2, 3}): return launch_aligned_or_not<BITS, 4, 96, 2>(p, stream);
    case form_code({4, 64, 2, 3}): return launch_aligned_or_not<BITS, 4, 64, 2>(p, stream);
    case form_code({4, 128, 1, 3}): return launch_aligned_or_not<BITS, 4, 128, 1>(p, stream);
    case form_code({4, 96, 1, 3}): return launch_aligned_or_not<BITS, 4, 96, 1>(p, stream);
    case form_code({4, 64, 1, 3}): return launch_aligned_or_not<BITS, 4, 64, 1>(p, stream);
    case form_code({4, 128, 2, 1}): return launch_aligned_or_not<BITS, 4, 128, 2, 1>(p, stream);
    case form_code({4, 96, 2, 1}): return launch_aligned_or_not<BITS, 4, 96, 2, 1>(p, stream);
    case form_code({4, 128, 1, 1}): return launch_aligned_or_not<BITS, 4, 128, 1, 1>(p, stream);
    case form_code({4, 96, 1, 1}): return launch_aligned_or_not<BITS, 4, 96, 1, 1>(p, stream);
    case form_code({4, 64, 4, 1}):
      if constexpr (BITS == 4) return launch_aligned_or_not<BITS, 4, 64, 4, 1>(p, stream);
      break;
    default: break;
  }
  return hipErrorInvalidValue;   // a form without a kernel (tile_form never picks one)
}

}  // namespace

hipError_t launch_qkv_prefill(const QkvProblem& p, hipStream_t stream) {
  return p.bits == 8 ? launch_prefill_bits<8>(p, stream) : launch_prefill_bits<4>(p, stream);
}

}  // namespace kaio
