// Attention over the paged cache, stream form: few rows per sequence (decode).
//
// Bound by memory: every K and V row of a K/V head is read once for the whole
// group of query heads (and few new tokens) that share it, up to 16 packed
// rows per tile.
// * Workgroup = 4 waves on one tile; its 128-key blocks are cut into 32 keys
//   per wave, and each wave runs by itself: its own running maximum, sum and
//   output, its own LDS slice, no barrier inside the loop.  The waves' results
//   meet in LDS at the end of the piece.  The line of blocks is shared out
//   evenly over the workgroups (attention_schedule.hpp), two per CU.
// * S^T = K.Q^T with 16x16x32 MFMAs, two score tiles of 16 keys: lane (kb,
//   l16) holds row l16's keys 4 kb + (0..3) of each, which are, in this order,
//   its B operand of O^T = V^T.P^T over the 32 keys; V^T by transposed LDS
//   reads.
// * Softmax as in the tile form: f32 scores, maxima and sums, weights rounded
//   to the 16-bit type for the second product (f32 weights would take it out of
//   the 16-bit MFMAs), and their sum taken of the rounded ones, so that the
//   weights used add up to one.
// * Each wave's next 16 KiB of K and V are in flight in registers while the
//   current ones are computed on: 128 KiB per CU, four times what the memory
//   latency needs.  Both as non-temporal loads: a cache is read once per step.
// * Measured with the join: 64 sequences of 125 to 8000 keys, 8 K/V heads of
//   128 columns under 32, bf16: 182 us, 5.9 TB/s.  One sequence of 131000 keys:
//   98 us, 5.5 TB/s.  Four of 225 to 900 keys, 32 heads, where launches and
//   the latency of table, then keys, count: 18 us.  Eight of 110 to 258 keys,
//   in the direct form: 8.4 us.  The first at 64 columns: 104 us, 5.1 TB/s.

#include "attention_common.hpp"

namespace kaio {
namespace {

constexpr uint32_t R = kStreamRows, B = kStreamKeys;
constexpr int kKeys = 32;                    // keys per wave and block
static_assert(R == 16 && B == 4 * kKeys, "four waves of 32 keys, 16 rows");

template <int D>
struct Lds {
  static constexpr int kKRow = D * 2 + 16;   // 16 bytes more than a multiple of the banks: rows lie apart
  static constexpr int kVRow = D * 2;
  static constexpr int kK = kKeys * kVRow;   // V first (its swizzle wants aligned rows)
  static constexpr int kSize = kK + kKeys * kKRow;
  static_assert(kSize % 256 == 0 && kKeys * kKRow >= (int)R * D * 4, "the wave's output fits over K");
};

template <bool kBf16, int D>
__global__ void __launch_bounds__(256, 2) attention_stream_kernel(PagedAttention p, bool split, uint32_t tiles_bound) {
  using L = Lds<D>;
  constexpr int KS = D / 32;            // k steps of the first product
  constexpr int DT = D / 16;            // 16-column tiles of the output
  constexpr int CPR = D / 8;            // 16-byte chunks per row
  constexpr int RPL = 64 / CPR;         // rows per load of the wave
  constexpr int NL = kKeys / RPL;       // loads
  __shared__ __attribute__((aligned(256))) char buf[4][L::kSize];
  __shared__ float stat[2][4][R];       // maximum and sum of each wave's rows
  extern __shared__ char dyn[];
  Line& line = *reinterpret_cast<Line*>(dyn);   // split form only

  const PagedKV& kv = p.kv;
  const uint32_t tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, kb = lane >> 4;
  const uint32_t wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t g = p.group.d;
  const size_t row_elems = (size_t)kv.kv_heads * D;
  const bool negate = p.scale < 0.f;
  const float c = fmaxf(fabsf(p.scale) * 1.44269504088896341f, 1.17549435e-38f);

  Walk<R, B, kStreamMinUnits> walk(p, line, split, tiles_bound, lane);
  bool first_piece = true;
  while (walk.next()) {
    const Tile& t = walk.t;
    const uint32_t b0 = walk.b0, b1 = walk.b1, head = walk.head, seq = walk.seq_index;
    const bool complete = walk.complete;

    const uint32_t r = l16 < t.rows ? l16 : t.rows - 1;
    const uint32_t pr = t.row0 + r, tok = p.group.div(pr);
    const size_t qrow = ((size_t)(t.q0 + (int32_t)tok) * p.q_heads + head * g + (pr - tok * g)) * D;
    const int32_t pos = t.q0 + (int32_t)tok + t.shift;
    const int32_t floor = window_floor(p, pos), tfloor1 = window_floor(p, t.p1);
    const int32_t sinks = p.window ? (int32_t)(p.sinks < 0x7FFFFFFFu ? p.sinks : 0x7FFFFFFFu) : 0;

    short8_t q[KS];
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      q[k] = *reinterpret_cast<const short8_t*>(p.q + qrow + k * 32 + kb * 8);
      if (negate) q[k] ^= (short)0x8000;
    }
    floatx4 o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d) o[d] = floatx4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;

    const uint32_t nblk = t.count ? b1 - b0 : 0;
    auto key0_of = [&](uint32_t i) {                // first of this wave's keys in the piece's block i
      const uint32_t b = b0 + i;
      return (int32_t)((b < t.ns ? b : t.wb0 + (b - t.ns)) * B + wave * kKeys);
    };
    auto slots = [&](uint32_t i) {                  // slot of key lane % 32 of block i
      const int32_t k = key0_of(i) + (int32_t)(lane & 31);
      return i < nblk && k < t.hi ? slot_of(kv, seq, k) : -1;
    };
    u32x4 kr[NL], vr[NL];
    const uint32_t lrow = lane / CPR, lch = lane % CPR;
    auto fetch = [&](int32_t slot) {
      size_t at[NL];
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int32_t s = __shfl(slot, (int)(i * RPL + lrow));
        at[i] = (size_t)(s < 0 ? 0 : s) * row_elems + head * D + lch * 8;
      }
#pragma unroll
      for (int i = 0; i < NL; ++i) kr[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(kv.k + at[i]));
#pragma unroll
      for (int i = 0; i < NL; ++i) vr[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(kv.v + at[i]));
    };
    char* const mine = buf[wave];
    // V rows: 32-byte windows xor the row (128 columns: 8 rows over the banks; 64: two rows side by side)
    auto vswz = [](uint32_t row) { return (D == 128 ? (row & 7) : ((row >> 1) & 3)) * 32; };
    bool special = false;
    auto store = [&](int32_t slot, uint32_t live, bool edge) {
      if (~live) {
#pragma unroll
        for (int i = 0; i < NL; ++i)
          if (__shfl(slot, (int)(i * RPL + lrow)) < 0) vr[i] = u32x4{0, 0, 0, 0};
      }
      if (edge) {
        bool any = false;
#pragma unroll
        for (int i = 0; i < NL; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) any |= any_special<kBf16>(vr[i][e]);
        special = __any(any);
      }
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const uint32_t row = i * RPL + lrow;
        *reinterpret_cast<u32x4*>(mine + L::kK + row * L::kKRow + lch * 16) = kr[i];
        *reinterpret_cast<u32x4*>(mine + row * L::kVRow + ((lch * 16) ^ vswz(row))) = vr[i];
      }
    };
    auto edge_of = [&](int32_t key0) {
      return key0 + kKeys - 1 > t.p0 || (p.window && key0 <= tfloor1 && key0 + kKeys > sinks);
    };

    int32_t slot = slots(0), slot_next = slots(1);
    uint32_t live = (uint32_t)__ballot(slot >= 0);
    if (live) fetch(slot);
    if (!first_piece) __syncthreads();   // the previous piece's results are no longer read

    for (uint32_t i = 0; i < nblk; ++i) {
      const int32_t key0 = key0_of(i);
      const bool edge = edge_of(key0);
      special = false;
      // one wave's LDS accesses run in order: these writes follow its reads of the previous block
      asm volatile("" ::: "memory");
      if (live) store(slot, live, edge);
      asm volatile("" ::: "memory");
      const uint32_t live_next = (uint32_t)__ballot(slot_next >= 0);
      if (live_next) fetch(slot_next);
      const int32_t slot_after = slots(i + 2);
      if (live) {
        floatx4 s[2];
        const char* const kl = mine + L::kK + l16 * L::kKRow + kb * 16;
#pragma unroll
        for (int st = 0; st < 2; ++st) {
          s[st] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < KS; ++k)
            s[st] = mfma16<kBf16>(*reinterpret_cast<const short8_t*>(kl + st * 16 * L::kKRow + k * 64), q[k], s[st]);
        }
        // element e of tile st is key 16 st + 4 kb + e
        if (edge || ~live) {
          const uint32_t bits = live >> (4 * kb);
#pragma unroll
          for (int st = 0; st < 2; ++st)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int32_t key = key0 + 16 * st + 4 * (int32_t)kb + e;
              const bool sees = key <= pos && (key > floor || key < sinks) && ((bits >> (16 * st + e)) & 1);
              s[st][e] = sees ? s[st][e] : -INFINITY;
            }
        }
        float top = s[0][0];
#pragma unroll
        for (int e = 1; e < 8; ++e) top = fmaxf(top, s[e >> 2][e & 3]);
        top = max_rows16(top) * c;
        if (__any(top > m + kLag)) {
          const float m1 = fmaxf(m, top);
          const float old = m1 == -INFINITY ? 1.f : exp2_fast(m - m1);
          l *= old;
#pragma unroll
          for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][e] *= old;
          m = m1;
        }
        const float base = m == -INFINITY ? 0.f : kLift<kBf16> - m;
        u32x4 pk;
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const float a = exp2_fast(__builtin_fmaf(s[e >> 2][e & 3], c, base));
          const float b = exp2_fast(__builtin_fmaf(s[e >> 2][(e & 3) + 1], c, base));
          pk[e / 2] = pack2<kBf16>(a, b);
          l = add2<kBf16>(pk[e / 2], l);
        }
        const short8_t w = __builtin_bit_cast(short8_t, pk);
        const uint32_t vrow = 4 * kb + (l16 >> 2);
        auto vfrag = [&](int d) {
          const char* const a = mine + vrow * L::kVRow + ((d * 32 + (l16 & 3) * 8) ^ vswz(vrow));
          return join(read_tr(a), read_tr(a + 16 * L::kVRow));   // 16 rows on: the same swizzle
        };
        if (!special) {
#pragma unroll
          for (int d = 0; d < DT; ++d) o[d] = mfma16<kBf16>(vfrag(d), w, o[d]);
        } else {   // non-finite values apart, as counts of those that a row sees: weight 0 times infinity is not 0
          constexpr short one = kBf16 ? 0x3F80 : 0x3C00;
          short8_t sees;
#pragma unroll
          for (int e = 0; e < 8; ++e) sees[e] = s[e >> 2][e & 3] == -INFINITY ? (short)0 : one;
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            const Special<kBf16> v(vfrag(d));
            const floatx4 z = {0.f, 0.f, 0.f, 0.f};
            o[d] = mfma16<kBf16>(v.fin, w, o[d]);
            const floatx4 nan = mfma16<kBf16>(v.nan, sees, z), inf = mfma16<kBf16>(v.pos, sees, z),
                          neg = mfma16<kBf16>(v.neg, sees, z);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[d][e] = with_special(o[d][e], nan[e], inf[e], neg[e]);
          }
        }
      }
      slot = slot_next;
      slot_next = slot_after;
      live = live_next;
    }

    // ---- the waves' results together ----
    l = add_rows16(l);
    asm volatile("" ::: "memory");
    float* const own = reinterpret_cast<float*>(mine + L::kK);   // [R][D] over K; lane (kb, l16): row l16, columns 16 d + 4 kb ..
#pragma unroll
    for (int d = 0; d < DT; ++d) *reinterpret_cast<floatx4*>(own + l16 * D + ((16 * d + 4 * kb) ^ ((l16 & 7) * 4))) = o[d];
    if (kb == 0) {
      stat[0][wave][l16] = m;
      stat[1][wave][l16] = l;
    }
    __syncthreads();
    constexpr int PT = R * D / 256;          // elements per thread: 8 or 4, all of one row
    const uint32_t row = tid / (D / PT), col = tid % (D / PT) * PT;
    if (row < t.rows) {
      float top = stat[0][0][row];
#pragma unroll
      for (int w = 1; w < 4; ++w) top = fmaxf(top, stat[0][w][row]);
      const float base = top == -INFINITY ? 0.f : top;
      float sum = 0.f, acc[PT];
#pragma unroll
      for (int e = 0; e < PT; ++e) acc[e] = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = exp2_fast(stat[0][w][row] - base);
        sum += f * stat[1][w][row];
        const float* const src = reinterpret_cast<const float*>(buf[w] + L::kK) + row * D;
#pragma unroll
        for (int e = 0; e < PT; e += 4) {
          const floatx4 v = *reinterpret_cast<const floatx4*>(src + ((col + e) ^ ((row & 7) * 4)));
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[e + j] += f * v[j];
        }
      }
      if (complete) {
        const uint32_t opr = t.row0 + row, otok = p.group.div(opr);
        uint16_t* const dst =
            p.out + ((size_t)(t.q0 + (int32_t)otok) * p.q_heads + head * g + (opr - otok * g)) * D + col;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        uint32_t packed[PT / 2];
#pragma unroll
        for (int e = 0; e < PT; e += 2) packed[e / 2] = pack2<kBf16>(acc[e] * inv, acc[e + 1] * inv);
        __builtin_memcpy(__builtin_assume_aligned(dst, PT * 2), packed, PT * 2);
      } else {
        float* const part = partial_of<R, D>(p, gridDim.x, 2 * walk.wg + (b0 == 0));
#pragma unroll
        for (int e = 0; e < PT; e += 4)
          *reinterpret_cast<floatx4*>(part + row * D + col + e) = floatx4{acc[e], acc[e + 1], acc[e + 2], acc[e + 3]};
        if (col == 0) {
          part[R * D + row] = top;
          part[R * D + R + row] = sum;
        }
      }
    }
    first_piece = false;
  }
  walk.leave_note();
  uint32_t own_a, own_b;
  walk.owned(own_a, own_b);
  zero_unowned(p, blockIdx.x, gridDim.x, own_a, own_b);
}

}  // namespace

hipError_t launch_attention_stream(const PagedAttention& p, const AttentionPlan& plan, hipStream_t stream) {
  const size_t lds = plan.split ? sizeof(Line) : 0;
#define KAIO_STREAM(BF, DIM)                                                                                  \
  hipLaunchKernelGGL((attention_stream_kernel<BF, DIM>), dim3(plan.workgroups), dim3(256), lds, stream, p,    \
                     plan.split, plan.tiles)
  if (p.kv.head_dim == 128) {
    if (p.bf16) KAIO_STREAM(true, 128);
    else KAIO_STREAM(false, 128);
  } else {
    if (p.bf16) KAIO_STREAM(true, 64);
    else KAIO_STREAM(false, 64);
  }
#undef KAIO_STREAM
  return hipGetLastError();
}

}  // namespace kaio
