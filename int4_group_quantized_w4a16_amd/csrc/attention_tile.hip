// Attention over the paged cache, tile form: many rows (prompts, chunks).
//
// gfx950 design
// -------------
// * Workgroup = 4 waves, 128 packed rows (token * group + head) of one
//   (sequence, K/V head); wave w owns rows 32w .. 32w+31 and keeps their Q
//   fragments, running maximum, sum and output in registers.  Keys pass in
//   blocks of 64 through two LDS buffers shared by the waves (33 KiB each at
//   128 columns), so two workgroups share a CU and one's softmax runs under
//   the other's matrix instructions.
// * Scores are computed transposed, S^T = K.Q^T (32x32x16 MFMA, K the A
//   operand): a lane then holds, for ITS row, 16 keys of each 32, and their
//   weights in exactly the order in which it feeds them to the second product
//   O^T = V^T.P^T as B operand, with k index (h, j) standing for key
//   8 (j / 4) + 4 h + j % 4 of 16.  Weights never leave the lane; V^T comes
//   from transposed LDS reads of four keys each in the same order.
// * The cache rows of the next block go straight to LDS (direct loads) while
//   the current one is computed on; one barrier per block.  Lane j of each
//   wave looks up the slot of key j one block ahead of that.  A load covers 4
//   (64 columns: 8) keys; where they share a page (page_size a multiple of
//   that) it takes a wave-uniform 64-bit base and one lane offset, otherwise
//   one load per key.
// * LDS rows are unpadded (a direct load writes lane-contiguous chunks), so
//   bank conflicts are avoided by where each 16-byte chunk is put: K chunk c
//   of row r at c ^ (r % 16), V at its 64-byte window xor r % 4 (64 columns:
//   the same over pairs of rows, which share a 256-byte line of banks).
// * Softmax in f32 with base-2 exponents: p = 2^(c s - m), c = scale * log2 e
//   folded into one FMA; m lags (kLag).  Weights are rounded to the 16-bit
//   type for the second product, the sum is taken of the unrounded ones.
// * Masks are applied only in blocks that some row does not wholly see, by
//   selects on scores.  In those blocks a pass over V in LDS zeroes slots that
//   are not there and non-finite values (weight 0 times infinity is not 0);
//   the latter are added to the rows that see them afterwards, one by one.
//   Such blocks run in a loop of their own, so that the common one is small
//   and keeps its accumulators in place.

#include <type_traits>

#include "attention_common.hpp"

namespace kaio {
namespace {

constexpr uint32_t R = kTileRows, B = kTileKeys;
static_assert(R == 128 && B == 64, "four waves of 32 rows, blocks of two 32-key score tiles");

template <int D>
struct Lds {
  static constexpr int kRow = D * 2;         // bytes
  static constexpr int kV = B * kRow;        // offset of V in a buffer
  static constexpr int kSize = 2 * kV;
};

template <bool kBf16, int D>
__global__ void __launch_bounds__(256, 2) attention_tile_kernel(PagedAttention p, bool split, uint32_t tiles_bound) {
  using L = Lds<D>;
  constexpr int KS = D / 16;            // k steps of the first product
  constexpr int DT = D / 32;            // 32-column tiles of the output
  constexpr int CPR = D / 8;            // 16-byte chunks per row
  constexpr int RPW = 64 / CPR;         // rows per direct load of a wave
  constexpr int NL = B / RPW / 4;       // direct loads per wave, block and tensor
  __shared__ __attribute__((aligned(256))) char buf[2][L::kSize];
  __shared__ uint32_t flags[2][4];      // per buffer and wave: V holds non-finite values
  extern __shared__ char dyn[];
  Line& line = *reinterpret_cast<Line*>(dyn);   // split form only

  const PagedKV& kv = p.kv;
  const uint32_t tid = threadIdx.x, lane = tid & 63, l32 = lane & 31, h = lane >> 5;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t g = p.group.d;
  const size_t row_elems = (size_t)kv.kv_heads * D;       // a cache slot
  const bool negate = p.scale < 0.f;
  const float c = fmaxf(fabsf(p.scale) * 1.44269504088896341f, 1.17549435e-38f);

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
    // rows are in order of their positions: the wave's first and last
    const int32_t wpos0 = __builtin_amdgcn_readlane(pos, 0), wpos1 = __builtin_amdgcn_readlane(pos, 31);
    const int32_t wfloor1 = __builtin_amdgcn_readlane(floor, 31);
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
    // slot of key `lane` of block i
    auto slots = [&](uint32_t i) {
      const int32_t k = key0_of(i) + (int32_t)lane;
      return i < nblk && k < t.hi ? slot_of(kv, seq, k) : -1;
    };
    // The wave's share of the block's rows to LDS: load n covers rows (4 n + wave) RPW ..
    const uint32_t lrow = lane / CPR, lch = lane % CPR;
    const bool shared_page = kv.page.d % RPW == 0;
    auto kswz = [](uint32_t row) { return D == 128 ? (row & 15) : ((row >> 1) & 7); };            // of a 16-byte chunk
    auto vswz = [](uint32_t row) { return (D == 128 ? (row & 3) : ((row >> 1) & 1)) * 4; };
    auto fetch = [&](uint32_t buffer, int32_t slot) {
#pragma unroll
      for (int n = 0; n < NL; ++n) {
        const uint32_t row0 = (4 * n + wave) * RPW, row = row0 + lrow;
        char* const kl = buf[buffer] + row0 * L::kRow;
        const uint32_t koff = (lch ^ kswz(row)) * 16, voff = (lch ^ vswz(row)) * 16;
        if (shared_page) {
          // keys past t.hi or of an absent page share their first key's fate or lie in its page: valid memory
          const int32_t s0 = __builtin_amdgcn_readlane(slot, (int)row0);
          const size_t at = ((size_t)(s0 < 0 ? 0 : s0) * row_elems + head * D) * 2;
          const uint32_t lane_off = lrow * (uint32_t)(row_elems * 2);
          dma16(reinterpret_cast<const char*>(kv.k) + at, lane_off + koff, kl);
          dma16(reinterpret_cast<const char*>(kv.v) + at, lane_off + voff, kl + L::kV);
        } else {
#pragma unroll 1
          for (uint32_t j = 0; j < (uint32_t)RPW; ++j) {
            const int32_t s0 = __builtin_amdgcn_readlane(slot, (int)(row0 + j));
            const size_t at = ((size_t)(s0 < 0 ? 0 : s0) * row_elems + head * D) * 2;
            if (lrow == j) {
              dma16(reinterpret_cast<const char*>(kv.k) + at, koff, kl);
              dma16(reinterpret_cast<const char*>(kv.v) + at, voff, kl + L::kV);
            }
          }
        }
      }
    };
    // zeroes V of absent slots and non-finite values; notes whether there are any of the latter
    auto fix_v = [&](uint32_t buffer, uint64_t live) {
      bool special = false;
      char* const vl = buf[buffer] + L::kV;
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
      flags[buffer][wave] = __ballot(special) != 0;
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      return (flags[buffer][0] | flags[buffer][1] | flags[buffer][2] | flags[buffer][3]) != 0;
    };
    // some row of the tile does not see some key of the block that starts at key0
    auto edge_of = [&](int32_t key0) {
      return key0 + (int32_t)B - 1 > t.p0 || (p.window && key0 <= tfloor1 && key0 + (int32_t)B > sinks);
    };

    int32_t slot = slots(0), slot_next = slots(1);
    uint64_t live = __ballot(slot >= 0);
    if (live) fetch(0, slot);
    wait_vm_barrier<0>();

    // One block.  kEdge: some row does not see some key (of the tile's rows: the choice is the workgroup's).
    auto block = [&](auto edge_tag, uint32_t i) {
      constexpr bool kEdge = decltype(edge_tag)::value;
      const int32_t key0 = key0_of(i);
      const char* const kb = buf[i & 1];
      const char* const vb = kb + L::kV;
      const uint64_t live_next = __ballot(slot_next >= 0);
      if (live_next) fetch((i + 1) & 1, slot_next);
      const int32_t slot_after = slots(i + 2);
      bool special = false;
      if constexpr (kEdge) special = fix_v(i & 1, live);

      // does any of the wave's rows see any of the block's keys?
      if (!kEdge || (live && key0 <= wpos1)) {
        // Left alone, the compiler reads each fragment just before its MFMA and waits out the LDS latency every
        // time; the scheduling barriers keep the reads one group of MFMAs ahead.
        floatx16 s[2];
        const uint32_t kbase = l32 * L::kRow, kx = (h ^ kswz(l32)) * 16;
        short8_t kf[2][4];
        auto read_k = [&](int g) {       // k steps 2 g and 2 g + 1 of both score tiles
#pragma unroll
          for (int x = 0; x < 4; ++x)
            kf[g & 1][x] = *reinterpret_cast<const short8_t*>(kb + (x & 1) * 32 * L::kRow +
                                                              (kbase + (kx ^ ((2 * g + (x >> 1)) * 32))));
        };
#pragma unroll
        for (int st = 0; st < 2; ++st)
#pragma unroll
          for (int e = 0; e < 16; ++e) s[st][e] = 0.f;
        read_k(0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int g = 0; g < KS / 2; ++g) {
          if (g + 1 < KS / 2) read_k(g + 1);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int x = 0; x < 4; ++x) s[x & 1] = mfma32<kBf16>(kf[g & 1][x], q[2 * g + (x >> 1)], s[x & 1]);
          __builtin_amdgcn_sched_barrier(0);
        }
        // element e of tile st is key 32 st + 8 (e / 4) + 4 h + e % 4
        if constexpr (kEdge) {
          const uint32_t lo32 = (uint32_t)(live >> (4 * h)), hi32 = (uint32_t)(live >> (32 + 4 * h));
#pragma unroll
          for (int st = 0; st < 2; ++st)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int off = 8 * (e / 4) + e % 4;
              const int32_t key = key0 + 32 * st + off + 4 * (int32_t)h;
              const bool sees = key <= pos && (key > floor || key < sinks) && (((st ? hi32 : lo32) >> off) & 1);
              s[st][e] = sees ? s[st][e] : -INFINITY;
            }
        }
        float top = s[0][0];
#pragma unroll
        for (int e = 1; e < 32; ++e) top = fmaxf(top, s[e >> 4][e & 15]);
        top = max_halves(top) * c;
        if (__any(top > m + kLag)) {
          const float m1 = fmaxf(m, top);
          const float old = m1 == -INFINITY ? 1.f : exp2_fast(m - m1);
          l *= old;
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[d][e] *= old;
          m = m1;
        }
        const float base = m == -INFINITY ? 0.f : -m;
        // V^T fragment of k step ks, columns 32 d ..: keys 16 ks + 4 h + (0..3), and 8 further on
        const uint32_t vrow = 4 * h + ((lane & 15) >> 2);
        const uint32_t vx = ((lane & 16) * 2 + (lane & 3) * 8) ^ (vswz(vrow) * 16);
        short8_t vf[2][DT];
        auto read_v = [&](int ks) {
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            const char* const a = vb + ks * 16 * L::kRow + (vrow * L::kRow + (vx ^ (d * 64)));
            vf[ks & 1][d] = join(read_tr(a), read_tr(a + 8 * L::kRow));
          }
        };
        short8_t w[4];
        auto weigh = [&](int ks) {       // weights of k step ks: elements 8 (ks % 2) .. + 7 of tile ks / 2
          u32x4 pk;
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float a = exp2_fast(__builtin_fmaf(s[ks >> 1][8 * (ks & 1) + e], c, base));
            const float b = exp2_fast(__builtin_fmaf(s[ks >> 1][8 * (ks & 1) + e + 1], c, base));
            l += a;
            l += b;
            pk[e / 2] = pack2<kBf16>(a, b);
          }
          w[ks] = __builtin_bit_cast(short8_t, pk);
        };
        // each step's weights are made under the previous step's MFMAs
        read_v(0);
        weigh(0);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          if (ks < 3) read_v(ks + 1);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int d = 0; d < DT; ++d) o[d] = mfma32<kBf16>(vf[ks & 1][d], w[ks], o[d]);
          if (ks < 3) weigh(ks + 1);
          __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (kEdge) {
          if (special) {
            // the non-finite values of the block, from the cache, to the rows that see their key
            typedef uint32_t u32x16 __attribute__((ext_vector_type(16)));
            const u32x16 wv = __builtin_bit_cast(u32x16, w);
#pragma unroll 1
            for (int j = 0; j < (int)B; ++j) {      // key j: an element of half (j / 4) % 2
              const int32_t sj = __builtin_amdgcn_readlane(slot, j);
              const int in32 = j & 31, half = (in32 >> 2) & 1, e = 4 * (in32 >> 3) + (in32 & 3);
              const uint32_t pair = wv[8 * (j >> 5) + (e >> 1)];
              const uint32_t pw = __shfl(e & 1 ? pair >> 16 : pair & 0xFFFFu, (int)l32 + 32 * half);
              const float x = to_f32<kBf16>((uint16_t)pw);
              if (sj < 0) continue;
              const uint16_t* const row = kv.v + (size_t)sj * row_elems + head * D + 4 * h;
#pragma unroll
              for (int d = 0; d < DT; ++d)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const u32x2 v = *reinterpret_cast<const u32x2*>(row + d * 32 + k * 8);
#pragma unroll
                  for (int y = 0; y < 4; ++y) {
                    const float vf = to_f32<kBf16>((uint16_t)(v[y >> 1] >> (16 * (y & 1))));
                    o[d][4 * k + y] += x != 0.f && !(fabsf(vf) < INFINITY) ? x * vf : 0.f;
                  }
                }
            }
          }
        }
      }
      slot = slot_next;
      slot_next = slot_after;
      live = live_next;
      wait_vm_barrier<0>();   // the next block is in place, this one no longer read
    };
    for (uint32_t i = 0; i < nblk;) {
      for (; i < nblk && (edge_of(key0_of(i)) || ~live); ++i) block(std::true_type{}, i);
      for (; i < nblk && !(edge_of(key0_of(i)) || ~live); ++i) block(std::false_type{}, i);
    }

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
        float* const row = part + (size_t)r * D + 4 * h;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<floatx4*>(row + 32 * d + 8 * j) =
                floatx4{o[d][4 * j], o[d][4 * j + 1], o[d][4 * j + 2], o[d][4 * j + 3]};
        if (h == 0) {
          part[R * D + r] = m;
          part[R * D + R + r] = l;
        }
      }
    }
  }
  walk.leave_note();
  zero_unowned(p, blockIdx.x, gridDim.x);
}

}  // namespace

hipError_t launch_attention_tile(const PagedAttention& p, const AttentionPlan& plan, hipStream_t stream) {
  const size_t lds = plan.split ? sizeof(Line) : 0;
#define KAIO_TILE(BF, DIM)                                                                                   \
  hipLaunchKernelGGL((attention_tile_kernel<BF, DIM>), dim3(plan.workgroups), dim3(256), lds, stream, p,     \
                     plan.split, plan.tiles)
  if (p.kv.head_dim == 128) {
    if (p.bf16) KAIO_TILE(true, 128);
    else KAIO_TILE(false, 128);
  } else {
    if (p.bf16) KAIO_TILE(true, 64);
    else KAIO_TILE(false, 64);
  }
#undef KAIO_TILE
  return hipGetLastError();
}

}  // namespace kaio
