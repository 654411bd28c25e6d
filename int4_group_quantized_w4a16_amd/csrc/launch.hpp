// Internal launchers (host side).  The C ABI in kaio_abi.cpp validates every
// argument before calling these; the launchers assume valid, non-empty problems.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "../../include/kaio.h"
#include "paged.hpp"

namespace kaio {

constexpr int kMaxDevices = 64;

// What a kernel that takes more than 64 KiB of LDS needs once on each device before it is launched there (one static object
// per kernel).
class LdsOf {
  std::atomic<uint64_t> done_{0};   // devices, as bits

 public:
  hipError_t allow(const void* kern, int bytes) {
    int device = 0;
    if (hipError_t e = hipGetDevice(&device)) return e;
    const uint64_t bit = 1ull << (device & (kMaxDevices - 1));
    if (done_.load(std::memory_order_acquire) & bit) return hipSuccess;
    const hipError_t e = hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == hipSuccess) done_.fetch_or(bit, std::memory_order_release);
    return e;
  }
};

struct QkvProblem {
  const uint16_t* x;        // f16 [m, k]
  const uint32_t* w[3];     // u32 [k*bits/32, n]: INT4 (bits 4) or INT8 (bits 8) values packed along k
  const uint16_t* s[3];     // f16 [k/128, n]
  uint16_t* out[3];         // f16 [m, n]
  uint32_t m, n, k;
  uint32_t bits;            // 4 (W4A16) or 8 (W8A16)
};

// Tile geometry, shared with the host-side grid-size checks.
constexpr uint64_t kComputeUnits = 256;  // MI355X
// Forms of the tile kernel: waves per set (each wave owns 16 columns of every
// output it computes), rows per tile, sets of waves per workgroup (2: the
// groups are split in halves over two sets, which needs an even group count)
// and outputs per workgroup (3: Q, K and V; 1: one of them, three times the
// workgroups).  Every form holds one workgroup per compute unit.  pass_cost: the time of one
// full pass of the form over the compute units, relative to 8 waves x 128
// rows (1000), measured at n = k = 4096 (16x16x32 f16 MFMA, 8 waves of 128
// rows: ~85 us per pass).  Small tiles cost more per output (the unpack is
// amortised over fewer rows), so the choice trades tile efficiency against
// how well the grid fills whole passes.
struct PrefillForm {
  uint32_t waves, bm, sets, outs;
};
struct PrefillFormCost {
  PrefillForm f;
  uint32_t pass_cost;
};
constexpr PrefillFormCost kPrefillForms[] = {
    {{8, 128, 1, 3}, 1000}, {{8, 96, 1, 3}, 780}, {{4, 128, 2, 3}, 555}, {{4, 96, 2, 3}, 450},
    {{4, 64, 2, 3}, 355},   {{4, 128, 1, 3}, 640}, {{4, 96, 1, 3}, 520}, {{4, 64, 1, 3}, 400}};
// s sets need a group count divisible by s; two three-output INT8 rings of
// 128-row tiles do not fit in LDS
constexpr bool prefill_form_ok(PrefillForm f, uint32_t k, uint32_t bits) {
  return f.sets == 1 || ((k / 128) % f.sets == 0 && (bits == 4 || f.bm <= 96 || f.outs == 1));
}
constexpr uint64_t prefill_wgs(PrefillForm f, uint32_t m, uint32_t n) {
  return (uint64_t)((m + f.bm - 1) / f.bm) * ((n + 16 * f.waves - 1) / (16 * f.waves)) * (f.outs == 1 ? 3 : 1);
}
// predicted time: whole passes at the full cost, a partial last pass at
// 0.7 + 0.3 x its share of the compute units (fewer workgroups contend less)
constexpr uint64_t prefill_cost(const PrefillFormCost& c, uint32_t m, uint32_t n) {
  const uint64_t wgs = prefill_wgs(c.f, m, n);
  const uint64_t full = wgs / kComputeUnits, rem = wgs % kComputeUnits;
  return c.pass_cost * (1000 * full + (rem ? 700 + 300 * rem / kComputeUnits : 0));
}
// the form with the least predicted time (the first of equals)
constexpr PrefillForm prefill_form(uint32_t m, uint32_t n, uint32_t k, uint32_t bits) {
  PrefillForm best = kPrefillForms[0].f;
  uint64_t best_cost = ~0ull;
  for (const PrefillFormCost& c : kPrefillForms) {
    if (!prefill_form_ok(c.f, k, bits)) continue;
    const uint64_t t = prefill_cost(c, m, n);
    if (t < best_cost) {
      best_cost = t;
      best = c.f;
    }
  }
  return best;
}
constexpr uint32_t kMaxN = 1u << 26;   // keeps 32-bit per-lane byte offsets in range (16 rows x N x 4 B)
constexpr uint32_t kMaxK = 1u << 24;
#ifndef KAIO_SK_MAXM
#define KAIO_SK_MAXM 64
#endif
constexpr uint32_t kDecodeMaxM = KAIO_SK_MAXM;   // the split-K kernel covers m <= this
// INT4 at 32 < m <= 64 with a group count divisible by 4 runs the tile kernel
// instead: one output per workgroup, 4 waves x 16 columns, 64-row tiles, four
// sets of waves (16 waves, four per SIMD) each over a quarter of the groups
// in a tight ring (148 KiB of LDS for the four; INT8's would not fit).  The
// four sets' independent load streams hide the latency that one group of
// lead leaves exposed.  Same-box graph replay over rotated weights, N = K =
// 4096, us (split-K -> four sets): m = 40 16.3 -> 15.3, 48 16.7 -> 15.5, 64
// 17.4 -> 15.7 (bit-identical: both split K into the same four parts); at
// m <= 32 it was slower (m = 32 11.8 -> 15.4), and at m > 64, where 64-row
// tiles double the grid, too (m = 80 20.2 -> 27.9).
constexpr bool qkv_split_k(uint32_t m, uint32_t k, uint32_t bits) {
  return m <= kDecodeMaxM && !(m > 32 && bits == 4 && (k / 128) % 4 == 0);
}
// Above kDecodeMaxM and up to kOneOutMaxM rows the tile kernel runs with one output per
// workgroup: 4 waves x 16 columns, 96-row tiles up to 96 rows and 128-row
// tiles beyond, the groups split over two sets of waves when their count is
// even.  At n = k = 4096 that is 192 workgroups where the three-output forms
// have 64; each weight word is unpacked once per tile instead of once per 32
// rows as in the split-K kernel.  Graph replay over rotated weight sets
// (us, split-K -> this form): m = 72 26.5 -> 20.3, 96 26.9 -> 20.9, 112
// 27.0 -> 22.6, 128 27.3 -> 23.3; at m <= 64 it was slower (m = 64 17.5 ->
// 18.3), and so were three-output 64-row tiles (30.3-30.8) and one-output
// 64-row tiles (32.5-32.9).  Its groups are short (32 MFMAs per wave), so
// the weights' memory latency, covered only one group ahead, bounds it.
constexpr uint32_t kOneOutMaxM = 128;
// the form of the tile kernel where qkv_split_k is false
constexpr PrefillForm tile_form(uint32_t m, uint32_t n, uint32_t k, uint32_t bits) {
  if (m <= kDecodeMaxM) return PrefillForm{4, 64, 4, 1};
  if (m <= kOneOutMaxM) return PrefillForm{4, m <= 96 ? 96u : 128u, (k / 128) % 2 == 0 ? 2u : 1u, 1};
  return prefill_form(m, n, k, bits);
}
// split-K configuration for 32 < m <= 64: row tiles per wave (the other
// rows go to other waves), words per lane load, waves per workgroup
#ifndef KAIO_SK4_RT
#define KAIO_SK4_RT 2
#endif
#ifndef KAIO_SK4_VEC
#define KAIO_SK4_VEC 4
#endif
#ifndef KAIO_SK4_WAVES
#define KAIO_SK4_WAVES 8
#endif
// columns of one output per split-K workgroup, by row count
constexpr uint32_t decode_bn(uint32_t m) { return m <= 32 ? 64u : 16u * KAIO_SK4_VEC; }
constexpr uint32_t kGemmBM = 256;
constexpr uint32_t kGemmBN = 256;
constexpr uint64_t kMaxWorkgroups = (1ull << 24) - 1;  // 1-D grid limit at 256 threads

hipError_t launch_qkv_prefill(const QkvProblem& p, hipStream_t stream);
hipError_t launch_qkv_decode(const QkvProblem& p, hipStream_t stream);
hipError_t launch_fill_zero(void* dst, size_t bytes, hipStream_t stream);
// grad16 is caller-provided scratch for f16(grad), m * n halves.
hipError_t launch_gemm_f16f32_bwd(const uint16_t* a, const uint16_t* b, const float* grad, uint16_t* grad_a,
                                  uint16_t* grad_b, uint16_t* grad16, uint32_t m, uint32_t n, uint32_t k,
                                  hipStream_t stream);
// The same with f16(grad) in the library's static per-device buffer of
// kGemmBwdScratchBytes (m * n * 2 must fit); nothing is allocated.
constexpr uint64_t kGemmBwdScratchBytes = 64ull << 20;
hipError_t launch_gemm_f16f32_bwd_noalloc(const uint16_t* a, const uint16_t* b, const float* grad,
                                          uint16_t* grad_a, uint16_t* grad_b, uint32_t m, uint32_t n,
                                          uint32_t k, hipStream_t stream);
hipError_t launch_gemm_f16f32(const uint16_t* a, const uint16_t* b, float* c,
                              uint32_t m, uint32_t n, uint32_t k, hipStream_t stream);
// y = act(x . (int4(W) * S) + bias) + residual; bias and residual may be null.
struct LinearProblem {
  const uint16_t* x;          // f16 [m, k]
  const uint32_t* w;          // u32 [k / 8, n]
  const uint16_t* s;          // f16 [k / 128, n]
  const uint16_t* bias;       // f16 [n]
  const uint16_t* residual;   // f16 [m, n]
  uint16_t* y;                // f16 [m, n]
  uint32_t m, n, k;
  int act;                    // kaio_activation
};
// Forms of the linear product.  Strips (the split-K kernel): 16 * vec columns
// per workgroup and up to `rows` rows.  Tiles: `waves` waves per set, `rows`
// rows, `sets` sets of waves that share out the groups, and `blocks` blocks of
// 16 * waves columns per workgroup.
struct LinearForm {
  uint32_t vec, waves, rows, sets, blocks;   // vec 0: a tile
  constexpr uint32_t code() const { return (((vec * 32 + waves) * 256 + rows) * 8 + sets) * 8 + blocks; }
};
// Strips.  n = 4096 / 11008, k = 4096, us with weights streamed from HBM, by
// columns per strip (16, 32, 64): m = 8 6.4 5.9 7.0 / 14.3 10.4 8.1, m = 16
// 7.4 6.9 8.0 / 19.1 13.1 9.6, m = 32 9.8 10.0 12.3 / - 18.7 13.5, m = 64 11.8
// 13.2 17.6 / - 31.4 21.5: the widest strip that still gives one workgroup to
// every compute unit, and 32 columns at least up to m = 16.
constexpr LinearForm linear_strips(uint32_t m, uint32_t n) {
  const uint32_t rows = m <= 8 ? 8 : m <= 16 ? 16 : m <= 32 ? 32 : 64;
  if (n > 8192) return LinearForm{4, m <= 16 ? 16u : 8u, rows, 1, 1};
  const bool narrow = n % 2 != 0 || (m > 16 && n <= 4096);
  return LinearForm{narrow ? 1u : 2u, m <= 16 ? 16u : 8u, rows, 1, 1};
}
// Tiles: as prefill_cost, `cost` is the time of a full pass at k = 4096 (0.1
// us, epilogue with bias, silu and residual) over slots = 256 x the
// workgroups a compute unit holds at once; a partial pass takes base + (1 -
// base) x its share.  The set counts divide the groups.
struct LinearFormCost {
  LinearForm f;
  uint32_t slots, cost, base;
};
constexpr LinearFormCost kLinearForms[] = {
    {{0, 4, 64, 4, 1}, 256, 153, 850},  {{0, 4, 64, 2, 1}, 256, 162, 850},  {{0, 4, 96, 2, 1}, 256, 201, 850},
    {{0, 4, 64, 2, 2}, 256, 233, 850},  {{0, 4, 96, 2, 2}, 256, 293, 800},
    {{0, 4, 128, 2, 2}, 256, 356, 800}, {{0, 8, 96, 1, 2}, 256, 503, 750},  {{0, 8, 128, 1, 2}, 256, 635, 750},
    {{0, 8, 128, 1, 3}, 256, 860, 750}, {{0, 4, 64, 1, 1}, 768, 376, 450},  {{0, 4, 64, 1, 2}, 512, 433, 450},
    {{0, 4, 96, 1, 1}, 512, 368, 500}};
constexpr uint64_t linear_tiles(LinearForm f, uint64_t m, uint64_t n) {
  const uint64_t bn = 16 * f.waves * f.blocks;
  return (m + f.rows - 1) / f.rows * ((n + bn - 1) / bn);
}
constexpr LinearForm linear_form(uint32_t m, uint32_t n, uint32_t k) {
  const uint32_t groups = k / 128;
  // up to 32 rows strips always; to 64 where they are faster than the four-set tile or there is none
  if (m <= 32 || (m <= 64 && (n <= 4096 || (n <= 8192 && groups % 4 != 0)))) return linear_strips(m, n);
  LinearForm best = kLinearForms[0].f;
  uint64_t best_cost = ~0ull;
  for (const LinearFormCost& c : kLinearForms) {
    if (groups % c.f.sets != 0) continue;
    const uint64_t wgs = linear_tiles(c.f, m, n), full = wgs / c.slots, rem = wgs % c.slots;
    const uint64_t t = c.cost * (1000 * full + (rem ? c.base + (1000 - c.base) * rem / c.slots : 0));
    if (t < best_cost) {
      best_cost = t;
      best = c.f;
    }
  }
  return best;
}
// a bound on the workgroups of a call in any form (16 columns x 64 rows are the smallest tile)
constexpr uint64_t linear_wgs(uint64_t m, uint64_t n) { return (m + 63) / 64 * ((n + 15) / 16); }
hipError_t launch_linear_w4a16(const LinearProblem& p, hipStream_t stream);

// Rows of 16-bit numbers rounded to int8, each with its scale.
hipError_t launch_quantize_rows(const uint16_t* x, bool bf16, uint8_t* q, float* scale, uint32_t m, uint32_t k,
                                hipStream_t stream);

// y = act(xs ws (x . w^T) + bias) + residual in 8-bit integers; bias and residual may be null.
struct Linear8 {
  const uint16_t* x16;        // 16-bit [m, k] to be rounded by the kernel (linear8_rounds), else null, and then
  const int8_t* x;            // [m, k]
  const float* xs;            // [m]
  const int8_t* w;            // [n, k]
  const float* ws;            // [n]
  const uint16_t* bias;       // [n], 16-bit as y
  const uint16_t* residual;   // [m, n]
  uint16_t* y;                // [m, n]
  uint32_t m, n, k;
  int act;                    // kaio_activation
  bool bf16;
};
constexpr uint32_t kLinear8MaxK = (1u << 17) - 16;   // |sum| <= 2^14 k stays below 2^31
// bytes of m rounded rows of k, then of their scales
constexpr uint64_t linear8_rows_bytes(uint64_t m, uint64_t k) { return m * k; }
constexpr uint64_t linear8_workspace(uint64_t m, uint64_t k) { return linear8_rows_bytes(m, k) + (4 * m + 15) / 16 * 16; }
// Forms of the 8-bit product: strips of 16 channels by their waves (up to 16 tokens), tiles of channels x tokens.
enum Linear8Form { kStrip16, kStrip4, kTile32x32, kTile32x64, kTile64x32, kTile64x64, kTile64x128, kTile128x128, kTile128x256, kTile256x256 };
// Of a tile form the time (0.1 us at k = 4096, n = 4096, weights from HBM) of one workgroup on every compute unit, and of
// two at once where they fit (0: they do not).  Other k are not measured, and the choice does not look at k.  A form's tiles fill the compute units layer by layer, and a layer takes its
// time however many tiles it has: us at n = 4096 by m = 64 / 96 / 128 / 256 / 384 / 509 / 1024 / 2048: 32x32 8.2 11.3 11.3, 32x64 10.4
// 9.7 10.4 18.5, 64x64 12.6 12.2 12.6 12.8 18.2 18.9, 64x128 - - - 16.4 16.4 16.5 29.4, 128x128 - - - 20.8 20.8 20.8 21.1
// 39.9, 128x256 - - - - - - 29.2 33.8, 256x256 - - - - - - - 50.6 (57 of six at 8192 x 12288, 128x256 67.6 there).
struct Linear8Cost {
  Linear8Form f;
  uint32_t channels, tokens, one, two;
};
constexpr Linear8Cost kLinear8Forms[] = {
    {kTile32x32, 32, 32, 82, 113},    {kTile32x64, 32, 64, 104, 0},     {kTile64x32, 64, 32, 110, 0},   {kTile64x64, 64, 64, 126, 187},
    {kTile64x128, 64, 128, 164, 0}, {kTile128x128, 128, 128, 211, 0}, {kTile128x256, 128, 256, 338, 0}, {kTile256x256, 256, 256, 570, 0}};
constexpr uint64_t linear8_cost(const Linear8Cost& c, uint64_t m, uint64_t n) {
  const uint64_t tiles = (m + c.tokens - 1) / c.tokens * ((n + c.channels - 1) / c.channels);
  const uint64_t layers = (tiles + kComputeUnits - 1) / kComputeUnits;
  return c.two ? layers / 2 * c.two + layers % 2 * c.one : layers * c.one;
}
constexpr Linear8Form linear8_form(uint32_t m, uint32_t n) {
  // Strips, us with weights from HBM, 16 waves / 4: 16 x 4096 x 4096 6.9 / 7.6, 1 x 11004 x 4096 12.5 / 12.0, 16 tokens there
  // 15.8 / 14.9; the smallest tile takes 8.2 and 15.5.
  if (m <= 16) return n > 8192 ? kStrip4 : kStrip16;
  Linear8Form best = kTile256x256;
  uint64_t best_cost = ~0ull;
  for (const Linear8Cost& c : kLinear8Forms) {
    const uint64_t t = linear8_cost(c, m, n);
    if (t < best_cost) {
      best_cost = t;
      best = c.f;
    }
  }
  return best;
}
// Whether a call rounds its 16-bit x in the product's own workgroups, every one all of it, instead of by a launch of its own:
// us of calls one after the other, weights from HBM, inside / apart, at m = 1, 4, 8: n 2048, k 2048 4.9 / 8.6, 5.2 / 8.8, 5.5 / 8.9;
// n 4096, k 4096 6.7 / 10.4, 7.4 / 10.7, 8.8 / 10.6; n 4096, k 8192 10.1 / 13.3, 11.8 / 13.8.  The limit of one workgroup for
// each compute unit is that of an earlier form, which was slower past it (11004 channels 24.4 / 14.7); of this one 8192
// channels, k 4096, take 9.0 / 13.7, 10.1 / 14.1, 12.0 / 14.1.
constexpr uint32_t kLinear8Round = 1u << 15;   // elements of x that they take
constexpr bool linear8_rounds(uint32_t m, uint32_t n, uint32_t k) {
  return m <= 8 && n <= 16 * kComputeUnits && (uint64_t)m * k <= kLinear8Round;
}
static_assert(linear8_form(8, 16 * kComputeUnits) == kStrip16, "the form that rounds");
// a bound on the workgroups of a call in any form
constexpr uint64_t linear8_wgs(uint64_t m, uint64_t n) { return (m + 31) / 32 * ((n + 15) / 16); }
hipError_t launch_linear_w8a8(const Linear8& p, hipStream_t stream);

// Mixture of experts.  Tokens are taken in blocks of kMoeBlock, each of which has its own active experts.
constexpr uint32_t kMoeBlock = 64, kMoeMaxExperts = 512, kMoeMaxTop = 16, kMoeMaxTokens = 1u << 17;
constexpr uint32_t kMoeStrip = 32;   // columns of the products' workgroups
struct MoeRoute {             // an active expert: its rows of h in the block
  uint32_t expert, first, count;
};
struct MoePair {              // a row of h: the token (of the block), and the expert's share of its result
  uint32_t token;
  float share;
};
struct Moe {
  const uint16_t *x, *router, *residual;        // [tokens, hidden], [experts, hidden], [tokens, hidden] or null
  const uint32_t *w_gate, *w_up, *w_down;       // [experts, hidden / 8, inner] (2), [experts, inner / 8, hidden]
  const uint16_t *s_gate, *s_up, *s_down;       // scales, a row per 128 of k
  uint16_t* y;
  uint32_t tokens, experts, hidden, inner, top_k;
  int act;
  bool normalize;
  uint32_t slots, splits;     // most active experts of a block; parts of the down product
  // workspace
  double* scores;             // [tokens, experts]
  MoeRoute* route;            // [blocks, slots]
  MoePair* pair;              // [tokens * top_k]
  uint32_t *active, *arrived; // [blocks], [blocks, hidden / kMoeStrip]
  uint16_t* h;                // [tokens * top_k, 2, inner]: high and low numbers
  uint8_t* bin;               // [tokens * top_k, inner / kMoeStrip]: their exponents
  uint32_t* odd;              // [blocks]: whether there are unusual ones
  float* partial;             // [splits, tokens, hidden] where splits > 1
};
struct MoePlan {
  uint64_t blocks, slots, splits;
  uint64_t route, pair, active, arrived, h, bin, odd, partial, bytes;   // offsets in the workspace (scores come first)
};
constexpr MoePlan moe_plan(uint64_t tokens, uint64_t experts, uint64_t hidden, uint64_t inner, uint64_t top_k) {
  MoePlan a{};
  a.blocks = (tokens + kMoeBlock - 1) / kMoeBlock;
  const uint64_t pairs = (tokens < kMoeBlock ? tokens : kMoeBlock) * top_k;
  a.slots = pairs < experts ? pairs : experts;
  // two workgroups of the down product per compute unit, of two units for each wave at least
  const uint64_t strips = hidden / kMoeStrip * a.blocks, units = a.slots * (inner / 128);
  const uint64_t fill = (2 * kComputeUnits + strips - 1) / strips, most = units / 16 ? units / 16 : 1;
  a.splits = fill < most ? fill : most;
  uint64_t at = 0;
  const auto take = [&at](uint64_t bytes) {
    const uint64_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  take(tokens * experts * 8);
  a.route = take(a.blocks * a.slots * sizeof(MoeRoute));
  a.pair = take(tokens * top_k * sizeof(MoePair));
  a.active = take(a.blocks * 4);
  a.arrived = take(a.blocks * (hidden / kMoeStrip) * 4);
  a.h = take(tokens * top_k * inner * 4);
  a.bin = take(tokens * top_k * (inner / kMoeStrip));
  a.odd = take(a.blocks * 4);
  a.partial = take(a.splits > 1 ? a.splits * tokens * hidden * 4 : 0);
  a.bytes = at;
  return a;
}
hipError_t launch_moe_w4a16(const Moe& p, hipStream_t stream);

constexpr uint32_t kMaxAxes = 8;
struct RopeAppend {
  PagedKV kv;
  const uint16_t *q, *k_new, *v_new;   // [tokens, heads, head_dim]
  uint16_t* q_out;
  const int32_t* positions;            // [axes, tokens]
  const double* inv_freq;              // [half]
  uint32_t first_pair[kMaxAxes];       // first pair of each axis
  uint32_t axes, half, q_heads;
  FastDiv per_head;                    // items per head of the vector form (head_dim / 16)
  bool bf16, interleaved;
};
hipError_t launch_rope_append(const RopeAppend& p, hipStream_t stream);

struct PagedAttention {
  PagedKV kv;
  const uint16_t* q;                   // [tokens, q_heads, head_dim]
  uint16_t* out;
  void* workspace;
  uint32_t q_heads, max_new;
  FastDiv group;                       // q heads per K/V head
  float scale;
  uint32_t window, sinks;              // window 0: none
  bool bf16;
};
// How a call runs: head_dim 64 and 128 on matrix instructions, few rows per
// sequence in the stream form, more in the tile form; other head_dims by rows.
constexpr uint32_t kTileRows = 128, kTileKeys = 64, kTileMinUnits = 2;
constexpr uint32_t kStreamRows = 16, kStreamKeys = 128, kStreamMinUnits = 1;
constexpr uint32_t kSchedTiles = 512;     // tiles (per K/V head) and sequences the split form's schedule holds
struct AttentionPlan {
  bool rows, stream, split;
  uint32_t tiles;           // bound on the tiles of one K/V head
  uint32_t workgroups;
  uint64_t workspace;       // bytes
};
// Whether few enough blocks leave nothing to gain from splitting tiles: one workgroup takes a tile from end to end, with
// no schedule to derive and nothing to join.  blocks: a bound on a tile's; share: tiles over workgroups resident at
// once.  A tile's block takes `alone` us with one workgroup on a compute unit, a split call `base` us more than a direct
// one and `full` us per block and resident workgroup (the mean tile of a prompt has half of the last one's blocks).  us,
// split / direct: 1024 tokens of 32 heads over 8, causal, 49 / 28; 4096 tokens 231 / 156; 1024 over 1024 58 / 46; 33 over
// 2000 25 / 45; 300 over 1000 36 / 34 (split all the same, by the rule); decode over 8 x 250 keys 12.8 / 8.5, 64 x 500
// 22.9 / 18.0, 16 x 900 15.2 / 21.4.  Past `most` blocks lengths that differ could leave too much to single workgroups.
// The limit holds for one sequence too, whose tiles differ only by their place in it: 4160 / 6144 / 8000 tokens, split,
// take 230 / 453 / 664 us, 4096 and 8192 (by the number of tiles), direct, 160 and 555.
// If it holds for a number of blocks, it holds for fewer.
constexpr bool attention_direct(bool stream, uint32_t head_dim, double blocks, double share, double mean) {
  const double alone = stream ? 2.0 : head_dim == 128 ? 1.24 : 0.85, full = stream ? 2.0 : head_dim == 128 ? 2.5 : 1.7;
  const double base = stream ? 7.0 : 14.0, most = stream ? 4.0 : 64.0;
  return blocks <= most && blocks * (alone - full * share * mean) <= base;
}
// window 0 and sinks 0 give a workspace that is enough with any.
constexpr AttentionPlan attention_plan(uint32_t kv_heads, uint32_t q_heads, uint32_t head_dim, uint32_t seqs,
                                       uint64_t cap, uint32_t tokens, uint32_t max_new, uint32_t window, uint32_t sinks) {
  AttentionPlan a{};
  a.rows = head_dim != 64 && head_dim != 128;
  if (a.rows) return a;
  const uint64_t g = q_heads / kv_heads;
  a.stream = max_new * g <= kStreamRows;
  const uint64_t rows = a.stream ? kStreamRows : kTileRows, keys = a.stream ? kStreamKeys : kTileKeys;
  // every sequence's last tile may be short
  const uint64_t tiles = tokens * g / rows + seqs;
  a.tiles = tiles ? (uint32_t)tiles : 1;
  // workgroups resident at once (three of the tile form's at 64 columns would fit: 80.4 us against 77.3 for 2049
  // windowed rows of 16 heads, as more workgroups mean more pieces)
  const uint64_t slots = 2 * kComputeUnits;
  uint64_t blocks = (cap + keys - 1) / keys;
  double mean = cap > max_new ? 1.0 - 0.5 * max_new / (double)cap : 0.5;
  if (window) {   // the sinks' blocks, and those of the window before each row of a tile
    const uint64_t seen = (sinks + keys - 1) / keys + (window + rows / g + keys - 1) / keys + 1;
    if (seen < blocks) {
      blocks = seen;
      mean = 1.0;
    }
  }
  const bool direct = attention_direct(a.stream, head_dim, (double)blocks, (double)a.tiles * kv_heads / slots, mean);
  a.split = !direct && tiles <= kSchedTiles && a.tiles * kv_heads < 4 * slots && (cap / keys + 2) * a.tiles * kv_heads < (1ull << 31);
  a.workgroups = (uint32_t)(a.split ? slots : a.tiles * kv_heads);
  a.workspace = a.split ? slots * (32 + 2 * rows * (head_dim + 2) * 4) : 0;
  return a;
}
hipError_t launch_attention_tile(const PagedAttention& p, const AttentionPlan& plan, hipStream_t stream);
hipError_t launch_attention_stream(const PagedAttention& p, const AttentionPlan& plan, hipStream_t stream);
hipError_t launch_attention_join(const PagedAttention& p, const AttentionPlan& plan, hipStream_t stream);
hipError_t launch_attention_rows(const PagedAttention& p, hipStream_t stream);

hipError_t launch_dequant_group_bwd(kaio_dtype dtype, int64_t outer, int64_t axis,
                                    int64_t group, const void* dy, const void* scale,
                                    void* dq, hipStream_t stream);

}  // namespace kaio
