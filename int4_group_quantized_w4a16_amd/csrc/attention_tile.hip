// Attention over the paged cache, tile form: many rows (prompts, chunks).
//
// gfx950 design
// -------------
// * Workgroup = 4 waves, 128 packed rows (token * group + head) of one
//   (sequence, K/V head); wave w owns rows 32w .. 32w+31 and keeps their Q
//   fragments, running maximum, sum and output in registers.  Keys pass in
//   tiles of 32 (blocks of two) through a ring of four LDS buffers shared by
//   the waves (16 KiB each at 128 columns), so two workgroups share a CU.
// * Software pipeline: while the vector unit turns tile t's scores into
//   weights, the matrix unit makes tile t+1's scores; while it then multiplies
//   tile t's weights with V, the vector unit finds tile t+1's maxima.  The
//   exponentials (16 cycles each for 64 lanes) take about as long as the
//   MFMAs, so neither can wait for the other: one 64-key block at a time
//   without this overlap ran 8192 causal keys, 32 heads of 128 columns, in
//   764 us.
// * Scores are computed transposed, S^T = K.Q^T (32x32x16 MFMA, K the A
//   operand): a lane then holds, for ITS row, 16 keys of each 32, and their
//   weights in exactly the order in which it feeds them to the second product
//   O^T = V^T.P^T as B operand, with k index (h, j) standing for key
//   8 (j / 4) + 4 h + j % 4 of 16.  Weights never leave the lane; V^T comes
//   from transposed LDS reads of four keys each in the same order.
// * The cache rows of a tile go straight to LDS (direct loads) three tiles
//   ahead; one barrier per tile.  Lane j of each wave looks up the slot of key
//   j of a block, a block ahead of that.  A load covers 4 (64 columns: 8)
//   keys.  Where they share a page (page_size a multiple of that) and the cache
//   is below 4 GiB per tensor, it takes the slot as a 32-bit scalar offset from
//   the head's base; otherwise there is a load, with a 64-bit base, per key
//   (1535 rows over 4000 to 12000 keys, as below: 351 us in a cache of 5 GiB,
//   342 with pages of 6, 246 so).
// * LDS rows are unpadded (a direct load writes lane-contiguous chunks), so
//   bank conflicts are avoided by where each 16-byte chunk is put: K chunk c
//   of row r at c ^ (r % 16), V at its 64-byte window xor r % 4 (64 columns:
//   the same over pairs of rows, which share a 256-byte line of banks).
// * Softmax in f32 with base-2 exponents: p = 2^(c s - m), c = scale * log2 e
//   folded into one FMA; m lags (kLag).  Weights are rounded to the 16-bit
//   type for the second product; their sum, in f32, is taken of the rounded
//   ones (two to a dot instruction), so that the weights used add up to one.
// * A wave goes first (s_setprio) while it makes weights and scores, where it
//   has both arithmetic and MFMAs to issue; its neighbour on the SIMD is then
//   mostly in its second product, which needs few issue slots (8192 causal
//   keys: 612 us without, 592 with).
// * Masks are applied only in blocks that some row does not wholly see, by
//   selects on scores, from the set of keys that the lane's row sees as the
//   bits of a word (comparing key by key: 75.8 us for the windowed case below,
//   69.1 so).  In those blocks a pass over V in LDS zeroes slots that are not
//   there and non-finite values (weight 0 times infinity is not 0); the latter
//   are added to the rows that see them afterwards, as they are.  Such blocks
//   run in a loop of their own, so that the common one is small and keeps its
//   accumulators in place.
// * Measured: 8192 causal keys, 32 heads of 128 columns, f16: 571 to 616 us by
//   card, 578 = 952 TFLOP/s.  1535 rows of three sequences over 4000 to 12000
//   cached keys, 32 heads over 8: 244 us with the join (13), 828.  2049 rows of
//   16 heads of 64 columns in a window of 4096: 66 us with the join (8), 525.
//   1024 causal tokens, 32 heads over 8: 28 to 30 us.  MFMA and vector unit
//   busy: 54% and 51% of the first case's cycles, 53% and 48%, 30% and 52%; the
//   waves wait 38%, 37%, 30% of their cycles to issue and 20%, 22%, 26% for
//   loads and barriers.  Of the first
//   case's time 421 us remain without the softmax and 388 without the MFMAs
//   (half of the cycles are the MFMAs' own): what bounds it is how far the two
//   waves of a SIMD overlap.  Slower: 64 rows per wave with one wave per SIMD
//   (836 us), eight waves in a workgroup, the halves kept half a step apart by
//   barriers (744) or not (629), K fragments read a step ahead (+1%), V of
//   edge tiles cleaned a tile ahead without a barrier of its own (+2%).

#include <type_traits>

#include "attention_common.hpp"

namespace kaio {
namespace {

constexpr uint32_t R = kTileRows, B = kTileKeys;
static_assert(R == 128 && B == 64, "four waves of 32 rows, blocks of two 32-key tiles");

template <int D>
struct Lds {
  static constexpr int kRow = D * 2;         // bytes
  static constexpr int kV = 32 * kRow;       // offset of V in a tile's buffer
  static constexpr int kSize = 2 * kV;
};

// kGrouped: keys that a load covers share a page, so one slot, a scalar offset, serves them all (and the offsets of
// the cache fit in 32 bits).  Otherwise a load per key.
template <bool kBf16, int D, bool kGrouped>
__global__ void __launch_bounds__(256, 2) attention_tile_kernel(PagedAttention p, bool split, uint32_t tiles_bound) {
  using L = Lds<D>;
  constexpr int KS = D / 16;            // k steps of the first product
  constexpr int DT = D / 32;            // 32-column tiles of the output
  constexpr int CPR = D / 8;            // 16-byte chunks per row
  constexpr int RPW = 64 / CPR;         // rows per direct load of a wave
  constexpr int NL = 32 / RPW / 4;      // direct loads per wave, tile and tensor
  // one object: reads of one that direct loads write do not wait for direct loads to another
  struct Shared {
    char ring[4][L::kSize];
    uint32_t ids[4][4][64];             // per wave: page ids of four blocks' keys
    uint32_t flags[4];                  // per wave: V of the tile holds non-finite values
  };
  __shared__ __attribute__((aligned(256))) Shared sh;
  auto& ring = sh.ring;
  auto& ids = sh.ids;
  auto& flags = sh.flags;
  extern __shared__ char dyn[];
  Line& line = *reinterpret_cast<Line*>(dyn);   // split form only

  const PagedKV& kv = p.kv;
  const uint32_t tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t g = p.group.d;
  const size_t row_bytes = (size_t)kv.kv_heads * D * 2;   // a cache slot
  const bool negate = p.scale < 0.f;
  const float c = fmaxf(fabsf(p.scale) * 1.44269504088896341f, 1.17549435e-38f);
  constexpr uint32_t ks = !kGrouped ? 0 : D == 128 ? 2 : 3;   // keys per slot looked up: 1 << ks
  constexpr uint32_t kPer = 1u << ks;                         // blocks per window of 64 slots
  static_assert(!kGrouped || kPer == RPW, "keys per load");
  constexpr int kLoads = 2 * NL * (kGrouped ? 1 : RPW);       // of a wave per tile

  Walk<R, B, kTileMinUnits> walk(p, line, split, tiles_bound, lane);
  while (walk.next()) {
    const Tile& t = walk.t;
    const uint32_t b0 = walk.b0, b1 = walk.b1, head = walk.head, seq = walk.seq_index;
    const bool complete = walk.complete;

    // ---- this lane's row ----
    const uint32_t r = wave * 32 + l32 < t.rows ? wave * 32 + l32 : t.rows - 1;
    const uint32_t pr = t.row0 + r, tok = p.group.div(pr);
    const size_t qrow = ((size_t)(t.q0 + (int32_t)tok) * p.q_heads + head * g + (pr - tok * g)) * D;
    const int32_t pos = t.q0 + (int32_t)tok + t.shift;
    const int32_t floor = window_floor(p, pos);
    const int32_t sinks = p.window ? (int32_t)(p.sinks < 0x7FFFFFFFu ? p.sinks : 0x7FFFFFFFu) : 0;
    const int32_t tfloor1 = window_floor(p, t.p1);

    short8_t q[KS];
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      q[k] = *reinterpret_cast<const short8_t*>(p.q + qrow + k * 16 + h * 8);
      if (negate) q[k] ^= (short)0x8000;
    }
    floatx16 o[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[i][e] = 0.f;
    float m = -INFINITY, l = 0.f;

    const uint32_t nblk = t.count ? b1 - b0 : 0;    // a tile that sees nothing has no blocks
    auto key0_of = [&](uint32_t i) {                // first key of the piece's block i
      const uint32_t b = b0 + i;
      return (int32_t)((b < t.ns ? b : t.wb0 + (b - t.ns)) * B);
    };
    // Slots, one per 1 << ks keys: window w is blocks w << ks .., lane j its j-th group of keys.  In two steps: the
    // page ids go to LDS by a direct load (a register load here would make the compiler wait for everything in
    // flight where it is used), and are read a window later.
    const char* const table = reinterpret_cast<const char*>(kv.table + (size_t)seq * kv.width);
    auto group_key = [&](uint32_t w) {              // first key of this lane's group; its block
      const uint32_t blk = (w << ks) + (lane >> (6 - ks));
      return (uint32_t)key0_of(blk) + ((lane & ((64u >> ks) - 1)) << ks);
    };
    auto request = [&](uint32_t w) {                // returns the group's place in its page
      const uint32_t k = group_key(w), kc = k < kv.cap ? k : kv.cap - 1, pg = kv.page.div(kc);
      dma4(table, pg * 4, ids[wave][w & 3]);
      return kc - pg * kv.page.d;
    };
    auto slots = [&](uint32_t w, uint32_t place) {
      const uint32_t id = ids[wave][w & 3][lane];
      return (w << ks) + (lane >> (6 - ks)) < nblk && (int32_t)group_key(w) < t.hi && id < kv.pages
                 ? (int32_t)(id * kv.page.d + place) : -1;
    };
    // lane of slots() that has key j of block i (j a multiple of 1 << ks, or anything in its group)
    auto slot_lane = [&](uint32_t i, uint32_t j) { return ((i % kPer) << (6 - ks)) + (j >> ks); };
    // The wave's share of a tile's rows to ring buffer b: load n covers rows (4 n + wave) RPW .. of keys 32 half ..
    // of block i, whose slots these are.  Always the same number of loads (the waits count them): absent slots read
    // slot 0, which is there.
    const uint32_t lrow = lane / CPR, lch = lane % CPR;
    auto kswz = [](uint32_t row) { return D == 128 ? (row & 15) : ((row >> 1) & 7); };            // of a 16-byte chunk
    auto vswz = [](uint32_t row) { return (D == 128 ? (row & 3) : ((row >> 1) & 1)) * 4; };
    const char* const khead = reinterpret_cast<const char*>(kv.k) + (size_t)head * D * 2;
    const char* const vhead = reinterpret_cast<const char*>(kv.v) + (size_t)head * D * 2;
    const u32x4 krsrc = raw_rsrc(khead), vrsrc = raw_rsrc(vhead);
    uint32_t koff[NL], voff[NL];
#pragma unroll
    for (int n = 0; n < NL; ++n) {
      const uint32_t row = (4 * n + wave) * RPW + lrow, off = kGrouped ? lrow * (uint32_t)row_bytes : 0;
      koff[n] = off + (lch ^ kswz(row)) * 16;
      voff[n] = off + (lch ^ vswz(row)) * 16;
    }
    auto fetch = [&](uint32_t b, int32_t there, uint32_t i, int half) {   // there: slots, 0 for absent ones
#pragma unroll
      for (int n = 0; n < NL; ++n) {
        const uint32_t row0 = (4 * n + wave) * RPW;
        char* const kl = ring[b] + row0 * L::kRow;
        if constexpr (kGrouped) {
          const uint32_t s0 = __builtin_amdgcn_readlane(there, (int)slot_lane(i, half * 32 + row0));
          dma16_pair<L::kV>(krsrc, koff[n], vrsrc, voff[n], s0, (uint32_t)row_bytes, kl);
        } else {
#pragma unroll 1
          for (uint32_t j = 0; j < (uint32_t)RPW; ++j) {
            const uint32_t s0 = __builtin_amdgcn_readlane(there, (int)(half * 32 + row0 + j));
            const size_t at = (size_t)s0 * row_bytes;
            if (lrow == j) {
              dma16(khead + at, koff[n], kl);
              dma16(vhead + at, voff[n], kl + L::kV);
            }
          }
        }
      }
    };
    // zeroes V of absent slots and non-finite values of the tile in buffer b; are there any of the latter?
    auto fix_v = [&](uint32_t b, uint32_t live) {
      bool special = false;
      char* const vl = ring[b] + L::kV;
#pragma unroll
      for (int n = 0; n < NL; ++n) {
        const uint32_t at = (n * 256 + tid) * 16, row = at / L::kRow;
        u32x4 v = *reinterpret_cast<const u32x4*>(vl + at);
        const bool there = (live >> row) & 1;
        bool change = !there;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool sp = any_special<kBf16>(v[e]);
          special |= there && sp;
          change |= sp;
          v[e] = there ? finite_only<kBf16>(v[e]) : 0u;
        }
        if (change) *reinterpret_cast<u32x4*>(vl + at) = v;
      }
      flags[wave] = __ballot(special) != 0;
      wait_vm_barrier<63>();   // LDS only
      return (flags[0] | flags[1] | flags[2] | flags[3]) != 0;
    };
    // some row of the tile does not see some key of the block that starts at key0
    auto edge_of = [&](int32_t key0) {
      return key0 + (int32_t)B - 1 > t.p0 || (p.window && key0 <= tfloor1 && key0 + (int32_t)B > sinks);
    };

    // The lane's places in the ring: K fragments by k step, V by column tile, of the block's first buffer (0 or 2); the
    // second is an immediate away, and going to the next block's flips one bit.
    constexpr uint32_t kFlip = 2 * L::kSize;
    static_assert((kFlip & (kFlip - 1)) == 0, "two buffers are a power of two");
    const char* const lds = ring[0];
    uint32_t kat[KS], vat[DT];
    const uint32_t kx = (h ^ kswz(l32)) * 16;
#pragma unroll
    for (int k = 0; k < KS; ++k) kat[k] = l32 * L::kRow + (kx ^ (k * 32));
    short8_t kf[2][4];
    auto read_k = [&](int second, int j) {     // k steps 4 j .. 4 j + 3 of the block's first or second tile
#pragma unroll
      for (int x = 0; x < 4; ++x) kf[j][x] = *reinterpret_cast<const short8_t*>(lds + kat[4 * j + x] + second * L::kSize);
    };
    // V^T fragments of a k step (16 keys), columns 32 d ..: its keys 4 h + (0..3), and 8 further on
    const uint32_t vrow = 4 * h + ((lane & 15) >> 2);
    const uint32_t vx = ((lane & 16) * 2 + (lane & 3) * 8) ^ (vswz(vrow) * 16);
#pragma unroll
    for (int d = 0; d < DT; ++d) vat[d] = L::kV + vrow * L::kRow + (vx ^ (d * 64));
    short8_t vf[2][DT];
    auto read_v = [&](int second, int step_k) {
#pragma unroll
      for (int d = 0; d < DT; ++d) {
        const char* const a = lds + vat[d] + second * L::kSize + step_k * 16 * L::kRow;
        vf[step_k][d] = join(read_tr(a), read_tr(a + 8 * L::kRow));
      }
    };
    floatx16 s[2];                       // scores: element e is key 8 (e / 4) + 4 h + e % 4 of the tile
    auto scores = [&](floatx16& sc, int j) {
#pragma unroll
      for (int x = 0; x < 4; ++x) sc = mfma32<kBf16>(kf[j][x], q[4 * j + x], sc);
    };
    auto max_of = [&](const floatx16& sc) {   // of this lane's half of the row, unscaled
      float top = sc[0];
#pragma unroll
      for (int e = 1; e < 16; ++e) top = fmaxf(top, sc[e]);
      return top;
    };

    int32_t sl0 = -1, sl1 = -1, sl2 = -1;    // slots of this window's keys and of the next two's
    int32_t slf = 0;                         // slots of the window that is fetched from, 0 for absent ones
    uint32_t place = 0;                      // of window w + 2 at the start of window w
    float top = 0.f;
    float limit = -INFINITY, base = 0.f;     // m + kLag, and kLift - m (0 while nothing is seen)
    if (nblk) {
      const uint32_t p0 = request(0), p1 = request(1);
      place = request(2);
      wait_vm<0>();   // the ids are the wave's own
      sl0 = slots(0, p0);
      sl1 = slots(1, p1);
      slf = max(sl0, 0);
      fetch(0, slf, 0, 0);
      fetch(1, slf, 0, 1);
      if constexpr (kPer == 1) slf = max(sl1, 0);
      fetch(2, slf, 1, 0);
      wait_vm_barrier<2 * kLoads>();
#pragma unroll
      for (int e = 0; e < 16; ++e) s[0][e] = 0.f;
#pragma unroll
      for (int j = 0; j < KS / 4; ++j) {
        read_k(0, j);
        scores(s[0], j);
      }
      top = max_of(s[0]);
    }

    // Tile 2 i + half of the piece; its scores and their maxima are there.  kEdge: some row does
    // not see some key of the block (of the tile's rows: the choice is the workgroup's).
    auto step = [&](auto edge_tag, auto half_tag, uint32_t i) {
      constexpr bool kEdge = decltype(edge_tag)::value;
      constexpr int kHalf = decltype(half_tag)::value;
      const uint32_t b = 2 * (i & 1) + kHalf;
      floatx16& sc = s[kHalf];
      floatx16& sn = s[1 - kHalf];
      wait_vm_barrier<kLoads>();         // the next tile is in place, the one before this no longer read
      if (kHalf == 0 && i % kPer == 0) {
        sl2 = slots(i / kPer + 2, place);
        place = request(i / kPer + 3);
      }
      const uint32_t in = i + 1 + kHalf;     // its first half is fetched now (kHalf 1), or its second
      if constexpr (kHalf == 1) {
        if (in % kPer == 0) slf = max(kPer == 1 ? sl2 : sl1, 0);
      }
      fetch((b + 3) & 3, slf, in, 1 - kHalf);
      if constexpr (kHalf == 1) {        // the next tile's K is in the next block's buffers
#pragma unroll
        for (int k = 0; k < KS; ++k) kat[k] ^= kFlip;
      }
      read_k(1 - kHalf, 0);
      bool special = false;
      uint32_t there = 0, sees = 0;
      if constexpr (kEdge) {
        const int32_t tile0 = key0_of(i) + 32 * kHalf;
        const int32_t mine = __shfl(sl0, (int)slot_lane(i, 32 * kHalf + l32));
        there = (uint32_t)__ballot(mine >= 0 && tile0 + (int32_t)l32 < t.hi);
        special = fix_v(b, there);
        // the keys of the tile that this lane's row sees, bit by bit: there, c <= pos, and c > floor or c < sinks
        auto first = [](int32_t n) { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1; };   // n ones
        sees = there & first(pos - tile0 + 1) & (~first(floor - tile0 + 1) | first(sinks - tile0));
        const uint32_t bits = sees >> (4 * h);
#pragma unroll
        for (int e = 0; e < 16; ++e)
          sc[e] = (int32_t)(bits << (31 - (8 * (e / 4) + e % 4))) < 0 ? sc[e] : -INFINITY;
        top = max_of(sc);
      }
      if (__any(top * c > limit)) {      // the row's maximum, over both halves, only where it matters
        const float m1 = fmaxf(m, max_halves(top) * c);
        const float old = m1 == -INFINITY ? 1.f : exp2_fast(m - m1);
        l *= old;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int e = 0; e < 16; ++e) o[d][e] *= old;
        m = m1;
        limit = m + kLag;
        base = m == -INFINITY ? 0.f : kLift<kBf16> - m;
      }
      short8_t w[2];
      auto weigh = [&](int step_k) {     // weights of a k step
        u32x4 pk;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float a = exp2_fast(__builtin_fmaf(sc[8 * step_k + e], c, base));
          const float b = exp2_fast(__builtin_fmaf(sc[8 * step_k + e + 1], c, base));
          pk[e / 2] = pack2<kBf16>(a, b);
          l = add2<kBf16>(pk[e / 2], l);
        }
        w[step_k] = __builtin_bit_cast(short8_t, pk);
      };
      // Left alone, the compiler reads each fragment just before its MFMA and waits out the LDS latency every
      // time; the scheduling barriers keep the reads one group of MFMAs ahead.
      if constexpr (KS > 4) read_k(1 - kHalf, 1);
      else read_v(kHalf, 0);
#pragma unroll
      for (int e = 0; e < 16; ++e) sn[e] = 0.f;
      // (One wait per group, by count, instead of one per fragment.)
      __builtin_amdgcn_sched_barrier(0);
      wait_lds<(KS > 4 ? 4 : 2 * DT)>();
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(1);
      scores(sn, 0);
      weigh(0);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (KS > 4) {
        read_v(kHalf, 0);
        __builtin_amdgcn_sched_barrier(0);
        wait_lds<2 * DT>();
        __builtin_amdgcn_sched_barrier(0);
        scores(sn, 1);
        weigh(1);
        __builtin_amdgcn_sched_barrier(0);
      }
      read_v(kHalf, 1);
      __builtin_amdgcn_sched_barrier(0);
      wait_lds<2 * DT>();
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(0);
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] = mfma32<kBf16>(vf[0][d], w[0], o[d]);
      if constexpr (KS <= 4) weigh(1);
      __builtin_amdgcn_sched_barrier(0);
      wait_lds<0>();
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] = mfma32<kBf16>(vf[1][d], w[1], o[d]);
      top = max_of(sn);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (kEdge) {
        if (special) {
          // the non-finite values of the tile, from the cache, to the rows that see their key: as they are, since no
          // weight changes them, also one that 16 bits round to zero
#pragma unroll 1
          for (int j = 0; j < 32; ++j) {
            if (!((there >> j) & 1)) continue;
            const int32_t sj = __builtin_amdgcn_readlane(sl0, (int)slot_lane(i, 32 * kHalf + j)) + (j & ((1 << ks) - 1));
            const bool mine = (sees >> j) & 1;
            const uint16_t* const row = reinterpret_cast<const uint16_t*>(vhead + (size_t)sj * row_bytes) + 4 * h;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const u32x2 v = *reinterpret_cast<const u32x2*>(row + d * 32 + k * 8);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  const float vv = to_f32<kBf16>((uint16_t)(v[y >> 1] >> (16 * (y & 1))));
                  o[d][4 * k + y] += mine && !(fabsf(vv) < INFINITY) ? vv : 0.f;
                }
                __builtin_amdgcn_sched_barrier(0);   // few registers at a time
              }
          }
          wait_vm<0>();   // or the compiler waits for these loads in the common loop
        }
      }
    };
    auto block = [&](auto edge_tag, uint32_t i) {
      step(edge_tag, std::integral_constant<int, 0>{}, i);
      step(edge_tag, std::integral_constant<int, 1>{}, i);
#pragma unroll
      for (int d = 0; d < DT; ++d) vat[d] ^= kFlip;
      if ((i + 1) % kPer == 0) {
        sl0 = sl1;
        sl1 = sl2;
      }
    };
    // every row sees every key of block i, and all are there
    auto clean = [&](uint32_t i) {
      constexpr uint32_t bits = 64 >> ks;
      const uint64_t absent = __ballot(sl0 < 0) >> (i % kPer * bits);
      return !edge_of(key0_of(i)) && (absent & (~0ull >> (64 - bits))) == 0;
    };
    for (uint32_t i = 0; i < nblk;) {
      for (; i < nblk && !clean(i); ++i) block(std::true_type{}, i);
      for (; i < nblk && clean(i); ++i) block(std::false_type{}, i);
    }
    wait_vm_barrier<0>();   // the loads past the end have landed before the ring is used again

    // ---- the piece's result ----
    l = add_halves(l);
    const bool mine = wave * 32 + l32 < t.rows;
    if (complete) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          // columns 32 d + 8 j + 4 h + (0..3) and 8 further on; exchanging halves gives each lane 8 in a row
          uint32_t a0 = pack2<kBf16>(o[d][4 * j] * inv, o[d][4 * j + 1] * inv);
          uint32_t a1 = pack2<kBf16>(o[d][4 * j + 2] * inv, o[d][4 * j + 3] * inv);
          uint32_t c0 = pack2<kBf16>(o[d][4 * j + 4] * inv, o[d][4 * j + 5] * inv);
          uint32_t c1 = pack2<kBf16>(o[d][4 * j + 6] * inv, o[d][4 * j + 7] * inv);
          const auto x0 = __builtin_amdgcn_permlane32_swap(a0, c0, false, false);
          const auto x1 = __builtin_amdgcn_permlane32_swap(a1, c1, false, false);
          if (mine)
            *reinterpret_cast<u32x4*>(p.out + qrow + 32 * d + 8 * (j + (int)h)) =
                u32x4{(uint32_t)x0[0], (uint32_t)x1[0], (uint32_t)x0[1], (uint32_t)x1[1]};
        }
    } else {
      float* const part = partial_of<R, D>(p, gridDim.x, 2 * walk.wg + (b0 == 0));
      if (mine) {
        float* const at = part + fragment_of<D>(r, 4 * h);
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<floatx4*>(at + (4 * d + j) * 256) =
                floatx4{o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]};
        if (h == 0) {
          part[R * D + r] = m;
          part[R * D + R + r] = l;
        }
      }
    }
  }
  walk.leave_note();
  uint32_t own_a, own_b;
  walk.owned(own_a, own_b);
  zero_unowned(p, blockIdx.x, gridDim.x, own_a, own_b);
}

}  // namespace

hipError_t launch_attention_tile(const PagedAttention& p, const AttentionPlan& plan, hipStream_t stream) {
  const size_t lds = plan.split ? sizeof(Line) : 0;
  const uint64_t cache = (uint64_t)p.kv.pages * p.kv.page.d * p.kv.kv_heads * p.kv.head_dim * 2;
  const bool grouped = p.kv.page.d % (p.kv.head_dim == 128 ? 4 : 8) == 0 && cache <= 0xFFFFFFFFull;
#define KAIO_TILE(BF, DIM)                                                                                      \
  if (grouped)                                                                                                  \
    hipLaunchKernelGGL((attention_tile_kernel<BF, DIM, true>), dim3(plan.workgroups), dim3(256), lds, stream,   \
                       p, plan.split, plan.tiles);                                                              \
  else                                                                                                          \
    hipLaunchKernelGGL((attention_tile_kernel<BF, DIM, false>), dim3(plan.workgroups), dim3(256), lds, stream,  \
                       p, plan.split, plan.tiles)
  if (p.kv.head_dim == 128) {
    if (p.bf16) { KAIO_TILE(true, 128); } else { KAIO_TILE(false, 128); }
  } else {
    if (p.bf16) { KAIO_TILE(true, 64); } else { KAIO_TILE(false, 64); }
  }
#undef KAIO_TILE
  return hipGetLastError();
}

}  // namespace kaio
