// A mixture-of-experts feed-forward on packed W4A16 weights, for a few tokens:
//
//   z[t, e] = sum_h x[t, h] R[e, h];  the top_k experts of a token by z (ties: lowest index) have the shares
//   p[t, e] = exp(z[t, e]) / sum exp(z[t, .]), the sum over all experts or (normalized) over the chosen ones
//   y[t] = sum_e p[t, e] ( act(x[t] . G_e) * (x[t] . U_e) ) . D_e + r[t]
//
// Four launches: scores, routes, up, down, in blocks of 64 tokens.  With few
// tokens the chosen experts' weights are the work, each read once per block:
// 0.516 bytes a weight, against 2 operations for each of an expert's rows, 1 to
// 16 of them, so that the bound is memory throughout.
//
// * scores: f64 sums of exact products, so that the order of experts is the
//   formula's wherever f64 tells them apart; a workgroup takes one expert and
//   up to four tokens.
// * routes: a block per workgroup (a wave for a token alone).  16 lanes find a token's top_k by top_k
//   maxima over keys in their registers; every expert's tokens are a mask of 64
//   bits, and the experts with any, in order, are the active ones.  An active
//   expert's rows are consecutive, so that h holds no empty ones.
// * up: one workgroup per active expert and 32 inner columns; its waves share
//   out the groups along the hidden axis, 16 of the expert's tokens at a time.
//   One workgroup is launched for every expert that could be active (the host
//   does not know how many are), the rest return.
// * down: one workgroup per 32 hidden columns and a part of the (active expert,
//   group) units, each of its waves a run of consecutive ones, so that an
//   expert's result stays in registers until the next expert.  The waves' sums
//   are in LDS, the parts' in the workspace, in f32, and the last workgroup to
//   arrive adds them in order: no sum depends on who came first.
//
// Measured, in us, scores + routes + up + down; E experts of I inner and H hidden
// columns, the active ones' weights over the last two: 1 token, E 64, top 8, I
// 1024, H 2048: 3 + 3 + 8 + 8 (latency: one wait for memory each).  8 tokens, E 8,
// top 2, I 8192, H 4096: 5 + 5 + 49 + 36 (374 MB, 4.4 TB/s).  33 tokens, E 128, top
// 8, I 768, H 2048: 6 + 8 + 41 + 30 (274 MB, 3.9 TB/s).  64 tokens, E 60, top 4, I
// 1408, H 2048: 6 + 6 + 40 + 30 (262 MB, 3.7 TB/s).  A copy reaches 5.2 TB/s.

#include "attention_common.hpp"
#include "common.hpp"
#include "epilogue.hpp"
#include "launch.hpp"

namespace kaio {
namespace {

constexpr uint32_t kBlock = kMoeBlock;   // tokens of a block (bits of a mask)
constexpr int kDownWaves = 8;

typedef unsigned long long u64;

// ---- scores -----------------------------------------------------------------
// One expert and kTokens tokens per workgroup.
template <int kTokens>
__global__ void __launch_bounds__(256) moe_scores_kernel(Moe p) {
  __shared__ double part[4][kTokens];
  const uint32_t tid = threadIdx.x, e = blockIdx.x, t0 = blockIdx.y * kTokens;
  const half8_t* const r = reinterpret_cast<const half8_t*>(p.router + (size_t)e * p.hidden);
  double sum[kTokens] = {};
  for (uint32_t c = tid; c < p.hidden / 8; c += 256) {
    const half8_t rv = r[c];
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      const uint32_t t = t0 + i < p.tokens ? t0 + i : p.tokens - 1;
      const half8_t xv = reinterpret_cast<const half8_t*>(p.x + (size_t)t * p.hidden)[c];
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[i] += (double)((float)rv[j] * (float)xv[j]);   // the product is exact in f32
    }
  }
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
#pragma unroll
    for (int s = 32; s; s >>= 1) sum[i] += __shfl_xor(sum[i], s);
    if (tid % 64 == 0) part[tid / 64][i] = sum[i];
  }
  __syncthreads();
  if (tid < kTokens && t0 + tid < p.tokens)
    p.scores[(size_t)(t0 + tid) * p.experts + e] = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
}

// ---- routes -----------------------------------------------------------------
// f64 numbers as integers of the same order; NaN below -infinity; 0: none
__device__ __forceinline__ u64 key_of(double z) {
  const u64 b = __builtin_bit_cast(u64, z);
  if ((b & 0x7FFFFFFFFFFFFFFFull) > 0x7FF0000000000000ull) return 1;
  if (b == 0x8000000000000000ull) return 0x8000000000000000ull;   // -0 is 0
  return b >> 63 ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ double score_of(u64 k) {
  return k == 1 ? (double)NAN : __builtin_bit_cast(double, k >> 63 ? k & 0x7FFFFFFFFFFFFFFFull : ~k);
}
// The largest and the smallest of the 16 values of a row of lanes, in each of them (rotations within the row).
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
  auto with = [&](int o) { x = x > (uint32_t)o ? x : (uint32_t)o; };
  with(__builtin_amdgcn_update_dpp(0, (int)x, 0x121, 0xF, 0xF, false));
  with(__builtin_amdgcn_update_dpp(0, (int)x, 0x122, 0xF, 0xF, false));
  with(__builtin_amdgcn_update_dpp(0, (int)x, 0x124, 0xF, 0xF, false));
  with(__builtin_amdgcn_update_dpp(0, (int)x, 0x128, 0xF, 0xF, false));
  return x;
}
__device__ __forceinline__ uint32_t row_min(uint32_t x) { return ~row_max(~x); }

struct RouteShared {
  u64 mask[kMoeMaxExperts];         // tokens of each expert
  uint32_t first[kMoeMaxExperts];   // its first row of h
  uint32_t choice[kBlock][kMoeMaxTop];
  float share[kBlock][kMoeMaxTop];
  uint32_t waves[2][16];
};

// The top_k of a token by 16 lanes, by top_k maxima; V keys per lane, those of experts lane * V + v.  Lane j < top_k gets the j-th
// best and its share.  (A wave for each token, its maxima by way of scalar registers, took 0.2 us for each: 9.7 us in all for
// 33 tokens and top_k 8.)
struct Choice {
  uint32_t expert;
  float share;
};
template <int V>
__device__ __forceinline__ Choice choose(const Moe& p, uint32_t token) {
  const uint32_t lane = threadIdx.x % 16;
  const double* const scores = p.scores + (size_t)token * p.experts;
  u64 key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const uint32_t e = lane * V + v;
    key[v] = e < p.experts ? key_of(scores[e]) : 0;
  }
  u64 mine = 0, first = 0;   // lane j: the key of the j-th best; and the first's
  uint32_t chosen = 0;       // and its expert
  for (uint32_t j = 0; j < p.top_k; ++j) {
    u64 best = key[0];
    uint32_t at = 0;
#pragma unroll
    for (int v = 1; v < V; ++v)
      if (key[v] > best) {
        best = key[v];
        at = v;
      }
    const uint32_t hi = row_max((uint32_t)(best >> 32));
    const uint32_t lo = row_max((uint32_t)(best >> 32) == hi ? (uint32_t)best : 0u);
    const u64 top = (u64)hi << 32 | lo;
    const uint32_t e = row_min(best == top ? lane * V + at : ~0u);   // ties: the lowest expert
    if (j == 0) first = top;
    mine = lane == j ? top : mine;
    chosen = lane == j ? e : chosen;
#pragma unroll
    for (int v = 0; v < V; ++v) key[v] = e == lane * V + v ? 0 : key[v];
  }
  const double top = score_of(first);
  auto part = [&](u64 k) { return __expf((float)(score_of(k) - top)); };
  const float own = lane < p.top_k ? part(mine) : 0.f;
  float sum = own;
  if (!p.normalize) {   // those that were not chosen
#pragma unroll
    for (int v = 0; v < V; ++v) sum += key[v] ? part(key[v]) : 0.f;
  }
#pragma unroll
  for (int x = 8; x; x >>= 1) sum += __shfl_xor(sum, x);
  return Choice{chosen, own / sum};
}

// One token: its choices are the active experts, in order of score.  (By the workgroup below: 4.9 us, here 3.2.)
template <int V>
__global__ void __launch_bounds__(64) moe_route_kernel(Moe p) {
  const uint32_t lane = threadIdx.x;
  for (uint32_t i = lane; i < p.hidden / kMoeStrip; i += 64) p.arrived[i] = 0;
  if (lane == 0) p.active[0] = p.top_k;
  const Choice c = choose<V>(p, 0);
  if (lane < p.top_k) {
    p.route[lane] = MoeRoute{c.expert, lane, 1};
    p.pair[lane] = MoePair{0, c.share};
  }
}

// Routes of one block by a workgroup of 1024 threads.
template <int V>
__global__ void __launch_bounds__(1024) moe_routes_kernel(Moe p) {
  __shared__ RouteShared s;
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, b = blockIdx.x, t0 = b * kBlock;
  const uint32_t tokens = p.tokens - t0 < kBlock ? p.tokens - t0 : kBlock;
  if (tid < kMoeMaxExperts) s.mask[tid] = 0;
  for (uint32_t i = tid; i < p.hidden / kMoeStrip; i += 1024) p.arrived[(size_t)b * (p.hidden / kMoeStrip) + i] = 0;
  __syncthreads();
  if (wave * 4 < tokens) {
    const uint32_t t = tid / 16, j = tid % 16;
    const Choice c = choose<V>(p, t0 + (t < tokens ? t : 0));
    if (t < tokens && j < p.top_k) {
      s.choice[t][j] = c.expert;
      s.share[t][j] = c.share;
      atomicOr(&s.mask[c.expert], 1ull << t);
    }
  }
  __syncthreads();
  // places of the active experts and of their tokens
  const u64 mask = tid < kMoeMaxExperts ? s.mask[tid] : 0;
  const uint32_t any = mask != 0, count = __popcll(mask);
  uint32_t place = any, rows = count;
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) {
    const uint32_t a = __shfl_up(place, x), c = __shfl_up(rows, x);
    if (lane >= (uint32_t)x) {
      place += a;
      rows += c;
    }
  }
  if (lane == 63) {
    s.waves[0][wave] = place;
    s.waves[1][wave] = rows;
  }
  __syncthreads();
  uint32_t active = 0;
  for (uint32_t w = 0; w < 16; ++w) {
    const uint32_t a = s.waves[0][w], c = s.waves[1][w];
    if (w < wave) {
      place += a;
      rows += c;
    }
    active += a;
  }
  if (tid == 0) p.active[b] = active;
  if (any) {
    p.route[(size_t)b * p.slots + place - 1] = MoeRoute{tid, rows - count, count};
    s.first[tid] = rows - count;
  }
  __syncthreads();
  MoePair* const pairs = p.pair + (size_t)b * kBlock * p.top_k;
  for (uint32_t o = tid; o < tokens * p.top_k; o += 1024) {
    const uint32_t t = o / p.top_k, j = o % p.top_k, e = s.choice[t][j];
    pairs[s.first[e] + __popcll(s.mask[e] & ((1ull << t) - 1))] = MoePair{t, s.share[t][j]};
  }
}

// ---- products ---------------------------------------------------------------
// Workgroups take strips of kMoeStrip columns (64 to a strip: 50 instead of 43 us for the up product of 33 tokens and 128
// experts, with half as many waves resident).  A lane holds two words of each of a group's four 32-k steps: row (lane / 16)
// of the step's four, columns 2 (lane % 16) and the next; word i is then the B operand of the MFMA whose column c stands for
// column 2 c + i.  Rows are 16 at a time (32: 6 to 10% less where every expert has more than 16, 20% more elsewhere).
constexpr int C = 2;
constexpr uint32_t N = 16 * C;
static_assert(N == kMoeStrip, "columns of a strip");
typedef float Columns __attribute__((ext_vector_type(C)));
struct Words {
  typedef uint32_t Row __attribute__((ext_vector_type(C)));
  typedef _Float16 Scales __attribute__((ext_vector_type(C)));
  Row w[4];
  Scales s;
  // Of group g (wave-uniform as the bases); there: whether there is one.  Loads are issued all the same, of an empty buffer:
  // under a branch, the compiler's waits for older loads would have to wait for these too.
  __device__ __forceinline__ void load(const uint32_t* w_, const uint16_t* s_, uint32_t n, uint32_t g, uint32_t kq, uint32_t col,
                                       bool there) {
    const __amdgpu_buffer_rsrc_t rw = __builtin_amdgcn_make_buffer_rsrc((void*)(w_ + (size_t)g * 16 * n), 0, there ? 64 * n : 0, 0x00020000);
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc((void*)(s_ + (size_t)g * n), 0, there ? 2 * n : 0, 0x00020000);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = __builtin_bit_cast(Row, __builtin_amdgcn_raw_buffer_load_b64(rw, (kq * n + col) * 4, i * 16 * n, 0));
    s = __builtin_bit_cast(Scales, __builtin_amdgcn_raw_buffer_load_b32(rs, col * 2, 0, 0));
  }
  __device__ __forceinline__ half8_t operand(int step, int i) const { return unpack_int4x8_scaled(w[step][i]); }
  __device__ __forceinline__ float scale(int i) const { return (float)s[i] * kUnpackScaledInv; }
};

// a lane's 16-k pieces of one row in a group's four steps
struct Rows {
  half8_t v[4];
};

// Adds the product of 16 rows with a group's words to acc.
__device__ __forceinline__ void multiply(floatx4 (&acc)[C], const Words& v, const Rows& rows) {
#pragma unroll
  for (int i = 0; i < C; ++i) {
    // one column set's operands at a time: unpacked ahead they take more registers than there are
    __builtin_amdgcn_sched_barrier(0);
    floatx4 c = {};
    half8_t w[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) w[s] = v.operand(s, i);
#pragma unroll
    for (int s = 0; s < 4; ++s) c = mfma16x16x32(rows.v[s], w[s], c);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[i][e] = __builtin_fmaf(c[e], v.scale(i), acc[i][e]);
  }
  __builtin_amdgcn_sched_barrier(0);
}

// N columns of act(x G) * (x U) for the tokens of one active expert, 16 of them at a time
template <int WAVES>
__global__ void __launch_bounds__(WAVES * 64, 4) moe_up_kernel(Moe p) {
  __shared__ float part[WAVES][2][16][N];
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, kq = lane >> 4;
  const uint32_t b = blockIdx.y, strips = p.inner / N, a = blockIdx.x / strips, n0 = blockIdx.x % strips * N;
  const MoeRoute route = p.route[(size_t)b * p.slots + a];   // whatever it is past the active ones
  const uint32_t active = p.active[b];
  asm volatile("" ::"s"(active), "s"(route.expert), "s"(route.first), "s"(route.count));   // both loads on the way at once
  if (a >= active) return;
  const uint32_t col = n0 + C * l16, H = p.hidden, I = p.inner, groups = H / kGroup;
  const size_t wat = (size_t)route.expert * (H / 8) * I, sat = (size_t)route.expert * groups * I;
  const uint32_t *wg = p.w_gate + wat, *wu = p.w_up + wat;
  const uint16_t *sg = p.s_gate + sat, *su = p.s_up + sat;
  const MoePair* const pairs = p.pair + (size_t)b * kBlock * p.top_k + route.first;
  struct Group {
    Words gate, up;
  };
  auto load = [&](Group& v, uint32_t g) {
    v.gate.load(wg, sg, I, g, kq, col, g < groups);
    v.up.load(wu, su, I, g, kq, col, g < groups);
  };
  for (uint32_t r0 = 0; r0 < route.count; r0 += 16) {
    Group ahead;
    load(ahead, wave);   // (the first ones before their rows are known)
    const uint32_t row = r0 + l16 < route.count ? r0 + l16 : route.count - 1;   // past the last that one
    const uint16_t* const x = p.x + ((size_t)b * kBlock + pairs[row].token) * H + 8 * kq;
    floatx4 gate[C] = {}, up[C] = {};
    auto read = [&](Rows& v, uint32_t g) {   // past the last group that one
#pragma unroll
      for (int s = 0; s < 4; ++s) v.v[s] = *reinterpret_cast<const half8_t*>(x + (g < groups ? g : groups - 1) * kGroup + 32 * s);
    };
    // Loads come back in order: the next group's rows and then its weights are on the way while one is multiplied.
    Rows rows;
    read(rows, wave);
#pragma unroll 1
    for (uint32_t g = wave; g < groups; g += WAVES) {
      const Group now = ahead;
      const Rows with = rows;
      read(rows, g + WAVES);
      load(ahead, g + WAVES);
      multiply(gate, now.gate, with);
      multiply(up, now.up, with);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      Columns vg, vu;
#pragma unroll
      for (int i = 0; i < C; ++i) vg[i] = gate[i][e], vu[i] = up[i][e];
      *reinterpret_cast<Columns*>(&part[wave][0][4 * kq + e][C * l16]) = vg;
      *reinterpret_cast<Columns*>(&part[wave][1][4 * kq + e][C * l16]) = vu;
    }
    __syncthreads();
    for (uint32_t o = tid; o < 16 * N; o += WAVES * 64) {
      const uint32_t at = r0 + o / N, c = o % N;
      if (at >= route.count) break;
      float y[1] = {0.f}, z = 0.f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        y[0] += part[w][0][o / N][c];
        z += part[w][1][o / N][c];
      }
      activations<1>(y, p.act);
      // rounded to f16, as the next product's other operand
      p.h[((size_t)b * kBlock * p.top_k + route.first + at) * I + n0 + c] = __builtin_bit_cast(uint16_t, (_Float16)(y[0] * z));
    }
    __syncthreads();
  }
}

// Units (a group's weights and rows) on the way to a wave of the down product, one after the other into the same registers:
// copied from register to register, a unit is waited for as soon as it is asked for (31.3 us instead of 30.0 for 33 tokens of
// 128 experts).  In the up product, with two matrices' weights for each of x's rows, the copies cost less than the loads gain by
// being sent before the product instead of after it (41 us, 49 in turns).
constexpr int kAhead = 3;

// N hidden columns of one part of the (active expert, group) units.  A wave takes consecutive ones and adds an expert's
// result, times the shares, to sums of its own in LDS, [token][column]; the waves' sums are added at the end.
__global__ void __launch_bounds__(kDownWaves * 64, 4) moe_down_kernel(Moe p) {
  extern __shared__ __attribute__((aligned(16))) float sums[];   // [wave][tokens of the block][N]
  __shared__ MoeRoute routes[kMoeMaxExperts];            // of the block's active experts
  __shared__ MoePair pairs[kBlock * kMoeMaxTop];         // and their rows
  __shared__ uint32_t last;
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, kq = lane >> 4;
  const uint32_t H = p.hidden, I = p.inner, groups = I / kGroup, strips = H / N;
  const uint32_t b = blockIdx.y, strip = blockIdx.x % strips, split = blockIdx.x / strips, n0 = strip * N, col = n0 + C * l16;
  const uint32_t tokens = p.tokens - b * kBlock < kBlock ? p.tokens - b * kBlock : kBlock;
  // All of them at once, whichever this part needs, and before the number of active ones is known (past it the workspace holds
  // anything): one wait for memory instead of three.
  const uint32_t active = p.active[b];   // (first: after stores the compiler would load it by vectors)
  for (uint32_t i = tid; i < p.slots; i += kDownWaves * 64) routes[i] = p.route[(size_t)b * p.slots + i];
  for (uint32_t i = tid; i < tokens * p.top_k; i += kDownWaves * 64) pairs[i] = p.pair[(size_t)b * kBlock * p.top_k + i];
  const u64 units = (u64)active * groups;
  const uint32_t u0 = (uint32_t)(units * split / p.splits), u1 = (uint32_t)(units * (split + 1) / p.splits), n = u1 - u0;
  const uint32_t wu0 = u0 + n * wave / kDownWaves, wu1 = u0 + n * (wave + 1) / kDownWaves;
  float* const mine = sums + wave * tokens * N;
  for (uint32_t i = lane; i < tokens * N / 4; i += 64) reinterpret_cast<floatx4*>(mine)[i] = floatx4{0.f, 0.f, 0.f, 0.f};
  __syncthreads();
  const uint16_t* const h0 = p.h + (size_t)b * kBlock * p.top_k * I + 8 * kq;
  // rows r0 .. of every expert (a second pass only where an expert has more than 16 tokens of the block)
  for (uint32_t r0 = 0; r0 < tokens; r0 += 16) {
    // the wave's units whose expert has such rows, one after the other; past the last that one, and not there
    struct Unit {
      uint32_t u, a, g;   // the unit, its expert's place in routes, its group
      bool there;
    };
    auto settle = [&](Unit t) {
      while (t.there && r0 >= routes[t.a].count) {   // on to the next expert
        t.u += groups - t.g;
        ++t.a;
        t.g = 0;
        t.there = t.u < wu1;
      }
      return t;
    };
    auto after = [&](const Unit& t) {
      if (t.u + 1 >= wu1) return Unit{t.u, t.a, t.g, false};
      const bool same = t.g + 1 < groups;
      const Unit n = settle(Unit{t.u + 1, same ? t.a : t.a + 1, same ? t.g + 1 : 0, true});
      return n.there ? n : Unit{t.u, t.a, t.g, false};
    };
    auto load = [&](Words& v, const Unit& t) {
      const size_t e = __builtin_amdgcn_readfirstlane(routes[t.a].expert);
      v.load(p.w_down + e * (I / 8) * H, p.s_down + e * groups * H, H, t.g, kq, col, t.there);
    };
    auto read = [&](Rows& v, const Unit& t) {   // past the last row that one, whose results go nowhere
      const uint32_t first = routes[t.a].first, count = routes[t.a].count, row = r0 + l16;
      const uint16_t* const h = h0 + (size_t)(first + (row < count ? row : count - 1)) * I + t.g * kGroup;
#pragma unroll
      for (int s = 0; s < 4; ++s) v.v[s] = *reinterpret_cast<const half8_t*>(h + 32 * s);
    };
    floatx4 acc[C] = {};
    uint32_t expert = ~0u;   // whose rows acc holds
    auto flush = [&] {
      if (expert == ~0u) return;
      const MoeRoute route = routes[expert];
      const uint32_t row = r0 + 4 * kq;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (row + e < route.count) {
          const MoePair pair = pairs[route.first + row + e];
          Columns* const to = reinterpret_cast<Columns*>(mine + pair.token * N + C * l16);
          Columns y = *to;
#pragma unroll
          for (int i = 0; i < C; ++i) y[i] = __builtin_fmaf(acc[i][e], pair.share, y[i]);
          *to = y;
        }
#pragma unroll
        for (int i = 0; i < C; ++i) acc[i][e] = 0.f;
      }
    };
    if (wu0 >= wu1) break;
    Unit t = settle(Unit{wu0, wu0 / groups, wu0 % groups, true});
    if (!t.there) continue;
    Words words[kAhead];
    Rows rows[kAhead];
    Unit next = after(t), second = after(next);
    read(rows[0], t);
    load(words[0], t);
    read(rows[1], next);
    load(words[1], next);
    read(rows[2], second);
    load(words[2], second);
    auto step = [&](int j) {
      if (t.a != expert) {
        flush();
        expert = t.a;
      }
      multiply(acc, words[j], rows[j]);
      const Unit third = after(second);
      read(rows[j], third);
      load(words[j], third);
      const bool more = next.there;
      t = next;
      next = second;
      second = third;
      return more;
    };
    while (step(0) && step(1) && step(2)) {
    }
    flush();
  }
  __syncthreads();
  // four columns of a token at a time
  const size_t first = (size_t)b * kBlock * H + n0;   // the block's first token
  auto finish = [&](uint32_t off, floatx4 y) {
    const size_t at = first + off;
    half4_t out;
    half4_t r = {};
    if (p.residual) r = *reinterpret_cast<const half4_t*>(p.residual + at);
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = (_Float16)(y[e] + (float)r[e]);
    *reinterpret_cast<half4_t*>(p.y + at) = out;
  };
  // Parts are written and read past the L2 of one XCD (scope bits of the device, 17) and are there once the stores are done: a
  // fence instead would have every workgroup write back all that its L2 holds (5 times the time of this kernel).
  constexpr int kDevice = 17;
  auto part = [&](uint32_t s) {
    return __builtin_amdgcn_make_buffer_rsrc(p.partial + (size_t)s * p.tokens * H + first, 0, 0xFFFFFFFFu, 0x00020000);
  };
  for (uint32_t o = tid; o < tokens * (N / 4); o += kDownWaves * 64) {
    floatx4 y = reinterpret_cast<const floatx4*>(sums)[o];
#pragma unroll
    for (int w = 1; w < kDownWaves; ++w) y += reinterpret_cast<const floatx4*>(sums + w * tokens * N)[o];
    const uint32_t off = o / (N / 4) * H + o % (N / 4) * 4;
    if (p.splits == 1) finish(off, y);
    else __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y), part(split), off * 4, 0, kDevice);
  }
  if (p.splits == 1) return;
  // the last of the strip's workgroups adds the parts, in order
  wait_vm<0>();
  __syncthreads();
  if (tid == 0) last = __hip_atomic_fetch_add(&p.arrived[(size_t)b * strips + strip], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == p.splits - 1;
  __syncthreads();
  if (!last) return;
  for (uint32_t o = tid; o < tokens * (N / 4); o += kDownWaves * 64) {
    const uint32_t off = o / (N / 4) * H + o % (N / 4) * 4;
    floatx4 y = {};
    for (uint32_t s0 = 0; s0 < p.splits; s0 += 8) {   // eight loads at a time
      u32x4 v[8];
#pragma unroll
      for (uint32_t i = 0; i < 8; ++i) v[i] = __builtin_amdgcn_raw_buffer_load_b128(part(s0 + i < p.splits ? s0 + i : s0), off * 4, 0, kDevice);
#pragma unroll
      for (uint32_t i = 0; i < 8; ++i)
        if (s0 + i < p.splits) y += __builtin_bit_cast(floatx4, v[i]);
    }
    finish(off, y);
  }
}

}  // namespace

hipError_t launch_moe_w4a16(const Moe& p, hipStream_t stream) {
  const uint32_t blocks = (p.tokens + kBlock - 1) / kBlock;
  if (p.tokens == 1) hipLaunchKernelGGL(moe_scores_kernel<1>, dim3(p.experts), dim3(256), 0, stream, p);
  else hipLaunchKernelGGL(moe_scores_kernel<4>, dim3(p.experts, (p.tokens + 3) / 4), dim3(256), 0, stream, p);
  if (hipError_t e = hipGetLastError()) return e;
  auto routes = [&](auto* one, auto* kern) {
    if (p.tokens == 1) hipLaunchKernelGGL(one, dim3(1), dim3(64), 0, stream, p);
    else hipLaunchKernelGGL(kern, dim3(blocks), dim3(1024), 0, stream, p);
  };
  if (p.experts <= 64) routes(&moe_route_kernel<4>, &moe_routes_kernel<4>);
  else if (p.experts <= 128) routes(&moe_route_kernel<8>, &moe_routes_kernel<8>);
  else if (p.experts <= 256) routes(&moe_route_kernel<16>, &moe_routes_kernel<16>);
  else routes(&moe_route_kernel<32>, &moe_routes_kernel<32>);
  if (hipError_t e = hipGetLastError()) return e;
  // Waves of the up product: four have twice as many groups each to load ahead (46 -> 43 us of 2700 workgroups), eight are
  // done sooner where there are not enough workgroups for the compute units.
  const uint32_t wgs = p.inner / N * p.slots;
  if ((uint64_t)wgs * blocks <= 4 * kComputeUnits) hipLaunchKernelGGL(moe_up_kernel<8>, dim3(wgs, blocks), dim3(8 * 64), 0, stream, p);
  else hipLaunchKernelGGL(moe_up_kernel<4>, dim3(wgs, blocks), dim3(4 * 64), 0, stream, p);
  if (hipError_t e = hipGetLastError()) return e;
  const uint32_t tokens = p.tokens < kBlock ? p.tokens : kBlock;
  static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(&moe_down_kernel),
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, kDownWaves * kBlock * N * 4);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL(moe_down_kernel, dim3(p.hidden / N * p.splits, blocks), dim3(kDownWaves * 64), kDownWaves * tokens * N * 4, stream, p);
  return hipGetLastError();
}

}  // namespace kaio
