// Joins the pieces of attention tiles whose keys were split over workgroups.
//
// Workgroup w of the split form left a note if it began a tile that others go
// on with (attention_schedule.hpp): its own piece is in slot 2w + 1, theirs in
// slots 2 (w + 1), 2 (w + 2), ...  Each row's result is
//
//   o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i,  m = max m_i.
//
// Four columns per thread.  Tile form: a workgroup per note, 32 rows and 32
// columns, threads in the order of the pieces' layout (fragment_of).  Stream
// form: a workgroup per note, RPB rows at a time; few rows (decode: the pieces
// are many, the rows few) leave threads over: they take the pieces in turns, and
// the partial sums meet in LDS, in a fixed order.

#include "attention_common.hpp"

namespace kaio {
namespace {

template <int D, uint32_t R, uint32_t THREADS>
constexpr uint32_t groups_of() {   // workgroups per note
  if (R == kTileRows) return R / 32 * (D / 32);
  constexpr uint32_t rpb = THREADS / (D / 4);
  return R > rpb ? R / rpb : 1;
}

template <bool kBf16, int D, uint32_t R, uint32_t THREADS>
__global__ void __launch_bounds__(THREADS) attention_join_kernel(PagedAttention p, uint32_t workers) {
  constexpr bool kFragments = R == kTileRows;
  static_assert(!kFragments || THREADS == 256, "32 rows of 8 x 4 columns");
  constexpr uint32_t TPR = kFragments ? 8 : D / 4;          // threads per row
  constexpr uint32_t RPB = THREADS / TPR;                   // rows per workgroup
  constexpr uint32_t GROUPS = groups_of<D, R, THREADS>();
  __shared__ floatx4 part_o[THREADS];
  __shared__ float part_m[RPB], part_l[RPB];
  const uint32_t tid = threadIdx.x, w = blockIdx.x / GROUPS, part_id = blockIdx.x % GROUPS;
  const uint32_t row0 = (kFragments ? part_id / (D / 32) : part_id) * RPB;
  const JoinNote note = static_cast<const JoinNote*>(p.workspace)[w];
  if (note.more == 0 || row0 >= note.rows) return;
  const uint32_t rows = note.rows - row0 < RPB ? note.rows - row0 : RPB;
  const uint32_t turns = kFragments ? 1 : RPB / rows;       // threads' turns at the pieces
  const uint32_t rg = kFragments ? tid % 32 : tid / TPR;
  const uint32_t col = kFragments ? part_id % (D / 32) * 32 + tid / 32 * 4 : tid % TPR * 4;
  if (kFragments && rg >= rows) return;
  const uint32_t row = row0 + rg % rows, turn = rg / rows;
  float m = -INFINITY, l = 0.f;
  floatx4 acc = {0.f, 0.f, 0.f, 0.f};
  if (turn < turns) {
#pragma unroll 4
    for (uint32_t i = turn; i <= note.more; i += turns) {
      const float* const part = partial_of<R, D>(p, workers, i == 0 ? 2 * w + 1 : 2 * (w + i));
      const floatx4 v = *reinterpret_cast<const floatx4*>(part + (kFragments ? fragment_of<D>(row, col) : row * D + col));
      const float mi = part[R * D + row], li = part[R * D + R + row];
      const float m1 = fmaxf(m, mi), base = m1 == -INFINITY ? 0.f : m1;
      const float fo = exp2_fast(m - base), fi = exp2_fast(mi - base);
      l = l * fo + li * fi;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = acc[e] * fo + v[e] * fi;
      m = m1;
    }
  }
  if (turns > 1) {
    part_o[tid] = acc;
    if (col == 0) {
      part_m[rg] = m;
      part_l[rg] = l;
    }
    __syncthreads();
  }
  if (turn != 0) return;
  if (turns > 1) {
    for (uint32_t k = 1; k < turns; ++k) {
      const uint32_t o = rg + k * rows;
      const floatx4 v = part_o[o * TPR + tid % TPR];
      const float m1 = fmaxf(m, part_m[o]), base = m1 == -INFINITY ? 0.f : m1;
      const float fo = exp2_fast(m - base), fi = exp2_fast(part_m[o] - base);
      l = l * fo + part_l[o] * fi;
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[e] = acc[e] * fo + v[e] * fi;
      m = m1;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const uint32_t pr = note.row0 + row, tok = p.group.div(pr), g = p.group.d;
  uint16_t* const dst = p.out + ((size_t)(note.q0 + (int32_t)tok) * p.q_heads + note.head * g + (pr - tok * g)) * D + col;
  *reinterpret_cast<u32x2*>(dst) = u32x2{pack2<kBf16>(acc[0] * inv, acc[1] * inv), pack2<kBf16>(acc[2] * inv, acc[3] * inv)};
}

// The stream form's few rows get 1024 threads: 131000 keys, one row of 4
// heads, 64 pieces each: 27 us with a thread to every four columns of a row
// alone, 15 with two turns, 7 with eight.
template <bool kBf16, int D, uint32_t R>
void launch(const PagedAttention& p, uint32_t workers, hipStream_t stream) {
  constexpr uint32_t threads = R == kStreamRows ? 1024 : 256;
  constexpr uint32_t groups = groups_of<D, R, threads>();
  hipLaunchKernelGGL((attention_join_kernel<kBf16, D, R, threads>), dim3(workers * groups), dim3(threads), 0, stream, p,
                     workers);
}
template <bool kBf16, int D>
void launch_rows(const PagedAttention& p, const AttentionPlan& plan, hipStream_t stream) {
  if (plan.stream) launch<kBf16, D, kStreamRows>(p, plan.workgroups, stream);
  else launch<kBf16, D, kTileRows>(p, plan.workgroups, stream);
}

}  // namespace

hipError_t launch_attention_join(const PagedAttention& p, const AttentionPlan& plan, hipStream_t stream) {
  if (p.kv.head_dim == 128) {
    if (p.bf16) launch_rows<true, 128>(p, plan, stream);
    else launch_rows<false, 128>(p, plan, stream);
  } else {
    if (p.bf16) launch_rows<true, 64>(p, plan, stream);
    else launch_rows<false, 64>(p, plan, stream);
  }
  return hipGetLastError();
}

}  // namespace kaio
