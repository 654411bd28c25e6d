// A mixture-of-experts feed-forward on packed W4A16 weights, for a few tokens:
//
//   z[t, e] = sum_h x[t, h] R[e, h];  the top_k experts of a token by z (ties: lowest index) have the shares
//   p[t, e] = exp(z[t, e]) / sum exp(z[t, .]), the sum over all experts or (normalized) over the chosen ones
//   y[t] = sum_e p[t, e] ( act(x[t] . G_e) * (x[t] . U_e) ) . D_e + r[t]
//
// Four launches: scores, routes, up, down, in blocks of 64 tokens.  With few
// tokens the chosen experts' weights are the work, 0.516 bytes each against 2
// operations for each of an expert's rows.  A block's tokens that chose an expert
// are taken 16 at a time, and its weights are read again for each 16 (the down
// product: 8 and 16), from the caches where they fit: mostly once with many
// experts; 64 tokens evenly over 8 experts, top 2, 1.4 times on average, over 4,
// top 4, four times.  One token is bound by latency, more by memory and the
// unpacking of the weights.
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
// * h between them: two f16 numbers each and an exponent per 32 columns (below).
// * down: one workgroup per 32 hidden columns and a part of the (active expert,
//   group) units, each of its waves a run of consecutive ones, so that an
//   expert's result stays in registers until the next expert.  Eight rows of h
//   at a time, sixteen of experts that have more than eight.  The waves' sums
//   are in LDS, the parts' in the workspace, in f32, and the last workgroup to
//   arrive adds them in order: no sum depends on who came first.
//
// Measured, in us, scores + routes + up + down; E experts of I inner and H hidden
// columns, the active ones' weights over the last two, from HBM but for the first:
// 1 token, E 64, top 8, I 1024, H 2048: 3 + 3 + 8 + 9 (latency: one wait for memory
// each).  8 tokens, E 8, top 2, I 8192, H 4096: 5 + 5 + 53 + 40 (374 MB, 4.0 TB/s).
// 33 tokens, E 128, top 8, I 768, H 2048: 6 + 9 + 42 + 31 (274 MB, 3.8 TB/s).  64
// tokens, E 60, top 4, I 1408, H 2048: 6 + 7 + 42 + 34 to 38 (262 MB, 3.3 to 3.5 TB/s).
// 64 tokens of I 4096, H 2048: E 8, top 2 70 in all, E 4, top 4 91; I 2048, E 16, top 8
// 112.  512 tokens of E 16, top 2, I 1024, H 1024: 76.  A copy reaches 5.2 TB/s.

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
  // to about a step of f32: what rounding the argument took comes back as a factor (the hardware's exponential of it alone is
  // off by up to 2^-18, an argument's absolute error being its result's relative one)
  auto part = [&](u64 k) {
    const double d = score_of(k) - top;
    const float f = (float)d, e = expf(f), rest = f > -110.f ? (float)(d - (double)f) : 0.f;   // (not of infinities: e is 0)
    return __builtin_fmaf(e, rest, e);
  };
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
  if (lane == 0) {
    p.active[0] = p.top_k;
    p.odd[0] = 0;
  }
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
  if (tid == 0) {
    p.active[b] = active;
    p.odd[b] = 0;
  }
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
// Workgroups take strips of kMoeStrip columns (64 to a strip: 50 instead of 43 us for an earlier up product of 33 tokens and
// 128 experts, now 42, with half as many waves resident).  A lane holds two words of each of a group's four 32-k steps: row (lane / 16)
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

// Adds the products of TILES times 16 rows with a group's words to acc.
template <int TILES>
__device__ __forceinline__ void multiply(floatx4 (&acc)[TILES][C], const Words& v, const Rows (&rows)[TILES]) {
#pragma unroll
  for (int i = 0; i < C; ++i) {
    // one column set's operands at a time: unpacked ahead they take more registers than there are
    __builtin_amdgcn_sched_barrier(0);
    half8_t w[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) w[s] = v.operand(s, i);
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      floatx4 c = {};
#pragma unroll
      for (int s = 0; s < 4; ++s) c = mfma16x16x32(rows[t].v[s], w[s], c);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[t][i][e] = __builtin_fmaf(c[e], v.scale(i), acc[t][i][e]);
    }
  }
  __builtin_amdgcn_sched_barrier(0);
}

// ---- h between the products ---------------------------------------------------
// f16 alone would cost h 13 of its 24 bits, and all of it past 65504 or far below 2^-14.  It is two f16 numbers instead: with
// t = h / 2^e, high = f16(t) and low = f16((t - high) 2^11), together within 2^-22 of h and 2^-36 of 2^e.  e is that of a
// strip's N columns of a row, from the largest finite magnitude in them: where that is in [2^(28 b - 156), 2^(28 b - 128)), b the
// strip's bin, 1 to 10, e is 28 b - 143, which brings it to [2^-13, 2^15).  The usual bin, 5, is 2^-16 to 2^12.  Bin 0: no finite
// one but zeros (of any e).  Infinities and NaN are high themselves.
//
// The high and the low numbers are rows of their own to the matrix instruction, one after the other, so that eight rows of h
// fill the 16 that it takes; the low row's sums count 2^-11.  Strips that add up must be of one e: where a block has any of an
// odd bin (neither 0 nor the usual one) the down product takes the units once for each bin, without the strips of others
// (33 tokens of 128 experts: 143 us in all instead of 86).
constexpr uint32_t kUsualBin = 5;
constexpr float kLow = 0x1p-11f;
__device__ __forceinline__ int exponent_of(uint32_t bin) { return 28 * (int)(bin ? bin : kUsualBin) - 143; }
__device__ __forceinline__ uint32_t bin_of(uint32_t most) { return most ? ((most >> 23) + 29) / 28 : 0; }   // f32's bits
static_assert(29 / 28 == 1 && (254 + 29) / 28 == 10 && (127 - 16 + 29) / 28 == kUsualBin && (127 + 11 + 29) / 28 == kUsualBin, "bins");
struct Pieces {
  uint16_t high, low;
  uint32_t bin;
};
// of one number of a strip per lane, 32 lanes to a strip
__device__ __forceinline__ Pieces pieces(float h) {
  const uint32_t bits = __builtin_bit_cast(uint32_t, h) & 0x7FFFFFFFu;
  const bool finite = bits < 0x7F800000u;
  uint32_t most = finite ? bits : 0;
#pragma unroll
  for (int x = 16; x; x >>= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)most, x);
    most = most > o ? most : o;
  }
  const uint32_t bin = bin_of(most);
  const float t = __builtin_ldexpf(h, -exponent_of(bin));
  const _Float16 high = (_Float16)t;
  const _Float16 low = finite ? (_Float16)((t - (float)high) * (1 / kLow)) : (_Float16)0.f;
  return Pieces{__builtin_bit_cast(uint16_t, high), __builtin_bit_cast(uint16_t, low), bin};
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
    floatx4 gate[1][C] = {}, up[1][C] = {};
    auto read = [&](Rows& v, uint32_t g) {   // past the last group that one
#pragma unroll
      for (int s = 0; s < 4; ++s) v.v[s] = *reinterpret_cast<const half8_t*>(x + (g < groups ? g : groups - 1) * kGroup + 32 * s);
    };
    // Loads come back in order: the next group's rows and then its weights are on the way while one is multiplied.
    Rows rows[1];
    read(rows[0], wave);
#pragma unroll 1
    for (uint32_t g = wave; g < groups; g += WAVES) {
      const Group now = ahead;
      const Rows with[1] = {rows[0]};
      read(rows[0], g + WAVES);
      load(ahead, g + WAVES);
      multiply(gate, now.gate, with);
      multiply(up, now.up, with);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      Columns vg, vu;
#pragma unroll
      for (int i = 0; i < C; ++i) vg[i] = gate[0][i][e], vu[i] = up[0][i][e];
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
      const Pieces h = pieces(y[0] * z);
      const size_t row = (size_t)b * kBlock * p.top_k + route.first + at;
      p.h[2 * row * I + n0 + c] = h.high;
      p.h[(2 * row + 1) * I + n0 + c] = h.low;
      if (c == 0) {
        p.bin[(row * I + n0) / N] = (uint8_t)h.bin;
        if (h.bin && h.bin != kUsualBin) __hip_atomic_store(&p.odd[b], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    }
    __syncthreads();
  }
}

// Units (a group's weights and rows) on the way to a wave of the down product, one after the other into the same registers:
// copied from register to register, a unit is waited for as soon as it is asked for (33 tokens of 128 experts with h in f16:
// 31.3 us instead of 30.0).  In the up product, with two matrices' weights for each of x's rows, the copies cost less than the
// loads gain by being sent before the product instead of after it (41 us, 49 in turns).  With sixteen rows at a time one unit
// is on the way: for two there are not the registers (64 tokens of 60 experts: 48 us instead of 34).
constexpr int kAhead = 3;

struct DownShared {
  MoeRoute routes[kMoeMaxExperts];      // of the block's active experts
  MoePair pairs[kBlock * kMoeMaxTop];   // and their rows
  uint32_t bins;                        // that the block has, as bits
  uint32_t last;
};

// A wave's units [first, last), TILES times 8 rows from r0 on, of those experts of the block that have LEAST to MOST rows from
// there on.  Adds an expert's result, times the shares, to mine ([token][column]).  PICK: takes only the strips of `bin`.
template <int TILES, int AHEAD, uint32_t LEAST, uint32_t MOST, bool PICK>
__device__ __forceinline__ void down_rows(const Moe& p, const DownShared& shared, float* mine, uint32_t r0, uint32_t first,
                                          uint32_t last, uint32_t b, uint32_t n0, uint32_t bin) {
  const uint32_t lane = threadIdx.x & 63, l16 = lane & 15, kq = lane >> 4, col = n0 + C * l16;
  const uint32_t H = p.hidden, I = p.inner, groups = I / kGroup;
  const MoeRoute* const routes = shared.routes;
  const size_t row0 = (size_t)b * kBlock * p.top_k;
  const uint16_t* const h0 = p.h + 2 * row0 * I + (size_t)(l16 & 1) * I + 8 * kq;
  // past the last unit that one, and not there
  struct Unit {
    uint32_t u, a, g;   // the unit, its expert's place in routes, its group
    bool there;
  };
  auto settle = [&](Unit t) {
    auto takes = [&](uint32_t count) { return count >= r0 + LEAST && count <= r0 + MOST; };
    while (t.there && !takes(routes[t.a].count)) {   // on to the next expert
      t.u += groups - t.g;
      ++t.a;
      t.g = 0;
      t.there = t.u < last;
    }
    return t;
  };
  auto after = [&](const Unit& t) {
    if (t.u + 1 >= last) return Unit{t.u, t.a, t.g, false};
    const bool same = t.g + 1 < groups;
    const Unit n = settle(Unit{t.u + 1, same ? t.a : t.a + 1, same ? t.g + 1 : 0, true});
    return n.there ? n : Unit{t.u, t.a, t.g, false};
  };
  auto load = [&](Words& v, const Unit& t) {
    const size_t e = __builtin_amdgcn_readfirstlane(routes[t.a].expert);
    v.load(p.w_down + e * (I / 8) * H, p.s_down + e * groups * H, H, t.g, kq, col, t.there);
  };
  // a lane's row of tile i, of the block's; past the last row that one, whose results go nowhere
  auto row_of = [&](const Unit& t, int i) {
    const uint32_t row = r0 + 8 * i + l16 / 2, count = routes[t.a].count;
    return routes[t.a].first + (row < count ? row : count - 1);
  };
  auto read = [&](Rows (&v)[TILES], const Unit& t) {
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
      const uint16_t* const h = h0 + (size_t)row_of(t, i) * 2 * I + t.g * kGroup;
#pragma unroll
      for (int s = 0; s < 4; ++s) v[i].v[s] = *reinterpret_cast<const half8_t*>(h + 32 * s);
    }
  };
  auto pick = [&](Rows (&v)[TILES], const Unit& t) {
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
      const uint32_t bins = *reinterpret_cast<const uint32_t*>(p.bin + (row0 + row_of(t, i)) * (I / N) + t.g * (kGroup / N));
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if ((bins >> 8 * s & 0xFF) != bin) v[i].v[s] = half8_t{};
      }
    }
  };
  static_assert(kGroup / N == 4, "the strips of a group are the steps of its product, and their bins a word");
  floatx4 acc[TILES][C] = {};
  uint32_t expert = ~0u;   // whose rows acc holds
  auto flush = [&] {
    if (expert == ~0u) return;
    const MoeRoute route = routes[expert];
#pragma unroll
    for (int i = 0; i < TILES; ++i)
#pragma unroll
      for (int e = 0; e < 4; e += 2) {   // of a lane's four sums two rows', high and low
        const uint32_t row = r0 + 8 * i + 2 * kq + e / 2;
        if (row < route.count) {
          const MoePair pair = shared.pairs[route.first + row];
          Columns* const to = reinterpret_cast<Columns*>(mine + pair.token * N + C * l16);
          Columns y = *to;
#pragma unroll
          for (int c = 0; c < C; ++c)
            y[c] = __builtin_fmaf(__builtin_ldexpf(__builtin_fmaf(acc[i][c][e + 1], kLow, acc[i][c][e]), exponent_of(bin)), pair.share, y[c]);
          *to = y;
        }
#pragma unroll
        for (int c = 0; c < C; ++c) acc[i][c][e] = acc[i][c][e + 1] = 0.f;
      }
  };
  Unit next[AHEAD];   // the unit to multiply and those on the way
  next[0] = settle(Unit{first, first / groups, first % groups, true});
  if (!next[0].there) return;
  Words words[AHEAD];
  Rows rows[AHEAD][TILES];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) {
    if (i) next[i] = after(next[i - 1]);
    read(rows[i], next[i]);
    load(words[i], next[i]);
  }
  auto step = [&](int j) {
    if (next[0].a != expert) {
      flush();
      expert = next[0].a;
    }
    if (PICK) pick(rows[j], next[0]);
    multiply(acc, words[j], rows[j]);
    const Unit n = after(next[AHEAD - 1]);
    read(rows[j], n);
    load(words[j], n);
#pragma unroll
    for (int i = 0; i + 1 < AHEAD; ++i) next[i] = next[i + 1];
    next[AHEAD - 1] = n;
    return next[0].there;
  };
  if constexpr (AHEAD == 3) {
    while (step(0) && step(1) && step(2)) {
    }
  } else {
    static_assert(AHEAD == 1);
    while (step(0)) {
    }
  }
  flush();
}

// N hidden columns of one part of the (active expert, group) units.  A wave takes consecutive ones and adds an expert's
// result, times the shares, to sums of its own in LDS, [token][column]; the waves' sums are added at the end.
__global__ void __launch_bounds__(kDownWaves * 64, 4) moe_down_kernel(Moe p) {
  extern __shared__ __attribute__((aligned(16))) float sums[];   // [wave][tokens of the block][N]
  __shared__ DownShared shared;
  constexpr uint32_t kThreads = kDownWaves * 64;
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t H = p.hidden, groups = p.inner / kGroup, strips = H / N;
  const uint32_t b = blockIdx.y, strip = blockIdx.x % strips, split = blockIdx.x / strips, n0 = strip * N;
  const uint32_t tokens = p.tokens - b * kBlock < kBlock ? p.tokens - b * kBlock : kBlock;
  // All of them at once, whichever this part needs, and before the number of active ones is known (past it the workspace holds
  // anything): one wait for memory instead of three.
  const uint32_t active = p.active[b], odd = p.odd[b];   // (first: after stores the compiler would load them by vectors)
  for (uint32_t i = tid; i < p.slots; i += kThreads) shared.routes[i] = p.route[(size_t)b * p.slots + i];
  const size_t row0 = (size_t)b * kBlock * p.top_k;
  for (uint32_t i = tid; i < tokens * p.top_k; i += kThreads) shared.pairs[i] = p.pair[row0 + i];
  if (tid == 0) shared.bins = 0;
  const u64 units = (u64)active * groups;
  const uint32_t u0 = (uint32_t)(units * split / p.splits), u1 = (uint32_t)(units * (split + 1) / p.splits), n = u1 - u0;
  const uint32_t wu0 = u0 + n * wave / kDownWaves, wu1 = u0 + n * (wave + 1) / kDownWaves;
  float* const mine = sums + wave * tokens * N;
  for (uint32_t i = lane; i < tokens * N / 4; i += 64) reinterpret_cast<floatx4*>(mine)[i] = floatx4{0.f, 0.f, 0.f, 0.f};
  __syncthreads();
  if (odd) {
    // the bins of a group's strips are a word
    const uint32_t* const bins = reinterpret_cast<const uint32_t*>(p.bin) + row0 * groups;
    uint32_t seen = 0;
    for (uint32_t i = tid; i < tokens * p.top_k * groups; i += kThreads) {
      const uint32_t word = bins[i];
      seen |= 1u << (word & 0xFF) | 1u << (word >> 8 & 0xFF) | 1u << (word >> 16 & 0xFF) | 1u << (word >> 24);
    }
    if (seen) atomicOr(&shared.bins, seen);
    __syncthreads();
  }
  // of the wave's experts the one with the most rows (of those that a lane looks at)
  uint32_t most = 0;
  if (wu0 < wu1)
    for (uint32_t a = wu0 / groups + lane; a <= (wu1 - 1) / groups; a += 64) most = shared.routes[a].count > most ? shared.routes[a].count : most;
  // (a second pass only where an expert has more than 16 tokens of the block)
  for (uint32_t r0 = 0; __any(most > r0); r0 += 16) {
    if (odd) {
      for (uint32_t bins = shared.bins; bins; bins &= bins - 1)
        down_rows<2, 1, 1, kBlock, true>(p, shared, mine, r0, wu0, wu1, b, n0, __builtin_ctz(bins));
    } else {
      down_rows<1, kAhead, 1, 8, false>(p, shared, mine, r0, wu0, wu1, b, n0, kUsualBin);
      if (__any(most > r0 + 8)) down_rows<2, 1, 9, kBlock, false>(p, shared, mine, r0, wu0, wu1, b, n0, kUsualBin);
    }
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
  if (tid == 0) shared.last = __hip_atomic_fetch_add(&p.arrived[(size_t)b * strips + strip], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == p.splits - 1;
  __syncthreads();
  if (!shared.last) return;
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
  static LdsOf of;
  if (hipError_t e = of.allow(reinterpret_cast<const void*>(&moe_down_kernel), kDownWaves * kBlock * N * 4)) return e;
  hipLaunchKernelGGL(moe_down_kernel, dim3(p.hidden / N * p.splits, blocks), dim3(kDownWaves * 64), kDownWaves * tokens * N * 4, stream, p);
  return hipGetLastError();
}

}  // namespace kaio
