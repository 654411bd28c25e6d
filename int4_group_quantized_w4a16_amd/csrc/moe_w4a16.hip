// A mixture-of-experts feed-forward on packed W4A16 weights, for a few tokens:
//
//   z[t, e] = sum_h x[t, h] R[e, h];  the top_k experts of a token by z (ties: lowest index) have the shares
//   p[t, e] = exp(z[t, e]) / sum exp(z[t, .]), the sum over all experts or (normalized) over the chosen ones
//   y[t] = sum_e p[t, e] ( act(x[t] . G_e) * (x[t] . U_e) ) . D_e + r[t]
//
// Four launches: scores, routes, up, down.  With few tokens the chosen experts'
// weights are the work, each read once:
//
// * scores: f64 sums of exact products, so that the order of experts is the
//   formula's wherever f64 tells them apart; a workgroup takes one expert and
//   up to four tokens.
// * routes: 64 tokens (a block) per workgroup.  A wave finds a token's top_k by
//   top_k maxima over keys in its registers; every expert's tokens are a mask
//   of 64 bits, and the experts with any, in order, are the active ones.
// * up: one workgroup per active expert and 64 inner columns; its waves share
//   out the groups along the hidden axis, 16 of the expert's tokens at a time.
// * down: one workgroup per 64 hidden columns and a part of the (active expert,
//   group) units, its waves taking every eighth.  All of the block's tokens are
//   rows of the product (zeros where the expert was not chosen), so that every
//   expert's result is added in the same registers.  The parts' sums go to the
//   workspace in f32, and the last workgroup to arrive adds them in order.

#include "attention_common.hpp"
#include "common.hpp"
#include "epilogue.hpp"
#include "launch.hpp"

namespace kaio {
namespace {

constexpr uint32_t kBlock = kMoeBlock;   // tokens of a block (bits of a mask)
constexpr int kUpWaves = 8, kDownWaves = 8;

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
// The largest of the wave's values (row shifts, then the rows' last lanes to the next; lane 63 ends with it).
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  auto with = [&](uint32_t o) { x = x > o ? x : o; };
  with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xF, 0xF, false));
  with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xF, 0xF, false));
  with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xF, 0xF, false));
  with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xF, 0xF, false));
  with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xA, 0xF, false));
  with((uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xC, 0xF, false));
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

struct RouteShared {
  u64 mask[kMoeMaxExperts];
  MoeRoute route[kMoeMaxExperts];   // of the active experts
  uint32_t choice[kBlock][kMoeMaxTop];
  float share[kBlock][kMoeMaxTop];
  uint32_t waves[2][16];
};

// the top_k of token t (of the block): V keys per lane, expert lane * V + v
template <int V>
__device__ __forceinline__ void choose(const Moe& p, RouteShared& s, uint32_t t, size_t token, uint32_t lane) {
  u64 key[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const uint32_t e = lane * V + v;
    key[v] = e < p.experts ? key_of(p.scores[token * p.experts + e]) : 0;
  }
  double top = 0;
  float sum = 0.f, mine = 0.f;
  uint32_t chosen = 0;
  for (uint32_t j = 0; j < p.top_k; ++j) {
    u64 best = key[0];
    uint32_t at = 0;
#pragma unroll
    for (int v = 1; v < V; ++v)
      if (key[v] > best) {
        best = key[v];
        at = v;
      }
    const uint32_t hi = wave_max((uint32_t)(best >> 32));
    const bool first = (uint32_t)(best >> 32) == hi;
    const uint32_t lo = wave_max(first ? (uint32_t)best : 0u);
    const int l = __builtin_ctzll(__ballot(first && (uint32_t)best == lo));   // ties: the lowest lane, the lowest expert
    const uint32_t v0 = __builtin_amdgcn_readlane(at, l);
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (lane == (uint32_t)l && v0 == (uint32_t)v) key[v] = 0;
    const double z = score_of((u64)hi << 32 | lo);
    if (j == 0) {
      top = z;
      if (!p.normalize) {   // all of them; the best's own is added with the chosen below
#pragma unroll
        for (int v = 0; v < V; ++v)
          if (key[v]) sum += __expf((float)(score_of(key[v]) - top));
#pragma unroll
        for (int x = 32; x; x >>= 1) sum += __shfl_xor(sum, x);
      }
    }
    const float part = __expf((float)(z - top));
    if (p.normalize || j == 0) sum += part;
    if (lane == j) {
      mine = part;
      chosen = l * V + v0;
    }
  }
  if (lane < p.top_k) {
    s.choice[t][lane] = chosen;
    s.share[t][lane] = mine / sum;
    atomicOr(&s.mask[chosen], 1ull << t);
  }
}

// Routes of one block by a workgroup of 1024 threads.
template <int V>
__global__ void __launch_bounds__(1024) moe_routes_kernel(Moe p) {
  __shared__ RouteShared s;
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, b = blockIdx.x, t0 = b * kBlock;
  const uint32_t tokens = p.tokens - t0 < kBlock ? p.tokens - t0 : kBlock;
  if (tid < kMoeMaxExperts) s.mask[tid] = 0;
  for (uint32_t i = tid; i < p.hidden / 64; i += 1024) p.arrived[(size_t)b * (p.hidden / 64) + i] = 0;
  __syncthreads();
  for (uint32_t t = wave; t < tokens; t += 16) choose<V>(p, s, t, t0 + t, lane);
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
  const size_t slot0 = (size_t)b * p.slots;
  if (any) s.route[place - 1] = p.route[slot0 + place - 1] = MoeRoute{mask, tid, rows - count};
  __syncthreads();
  for (uint32_t o = tid; o < active * kBlock; o += 1024) {
    const uint32_t t = o % kBlock;
    const MoeRoute r = s.route[o / kBlock];
    float share = 0.f;
    if (r.mask >> t & 1)   // (a token chooses an expert once)
      for (uint32_t j = 0; j < p.top_k; ++j) share = s.choice[t][j] == r.expert ? s.share[t][j] : share;
    p.share[slot0 * kBlock + o] = share;
  }
}

// ---- products ---------------------------------------------------------------
// A lane's four words of a 32-k step: row (lane / 16) of the step's four, columns 4 (lane % 16) .. + 3 of the strip;
// word i is then the B operand of the MFMA whose column c stands for column 4c + i.
struct Words {
  uint4 w[4];
  half4_t s;
  __device__ __forceinline__ void load(const uint32_t* w_, const uint16_t* s_, uint32_t n, uint32_t g, uint32_t kq, uint32_t col) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint4*>(w_ + (size_t)(g * 16 + i * 4 + kq) * n + col);
    s = *reinterpret_cast<const half4_t*>(s_ + (size_t)g * n + col);
  }
  __device__ __forceinline__ half8_t operand(int step, int i) const {
    const uint4& v = w[step];
    return unpack_int4x8_scaled(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
  }
};

// 64 columns of act(x G) * (x U) for the tokens of one active expert
__global__ void __launch_bounds__(kUpWaves * 64) moe_up_kernel(Moe p) {
  __shared__ float part[kUpWaves][2][16][64];
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l16 = lane & 15, kq = lane >> 4;
  const uint32_t b = blockIdx.y, strips = p.inner / 64, a = blockIdx.x / strips, n0 = blockIdx.x % strips * 64;
  if (a >= p.active[b]) return;
  const MoeRoute route = p.route[(size_t)b * p.slots + a];
  const uint32_t rows = __popcll(route.mask), col = n0 + 4 * l16;
  const uint32_t H = p.hidden, I = p.inner;
  const size_t wat = (size_t)route.expert * (H / 8) * I, sat = (size_t)route.expert * (H / kGroup) * I;
  const uint32_t *wg = p.w_gate + wat, *wu = p.w_up + wat;
  const uint16_t *sg = p.s_gate + sat, *su = p.s_up + sat;
  for (uint32_t r0 = 0; r0 < rows; r0 += 16) {
    // the token of this lane's row: the (r0 + l16)-th bit of the mask
    u64 left = route.mask;
    const uint32_t skip = r0 + l16 < rows ? r0 + l16 : rows - 1;
    for (uint32_t i = 0; i < skip; ++i) left &= left - 1;
    const uint16_t* const x = p.x + ((size_t)b * kBlock + __builtin_ctzll(left)) * H + 8 * kq;
    floatx4 gate[4] = {}, up[4] = {};
    for (uint32_t g = wave; g < H / kGroup; g += kUpWaves) {
      Words vg, vu;
      half8_t xv[4];
      vg.load(wg, sg, I, g, kq, col);
      vu.load(wu, su, I, g, kq, col);
#pragma unroll
      for (int s = 0; s < 4; ++s) xv[s] = *reinterpret_cast<const half8_t*>(x + g * kGroup + 32 * s);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        floatx4 cg = {}, cu = {};
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          cg = mfma16x16x32(xv[s], vg.operand(s, i), cg);
          cu = mfma16x16x32(xv[s], vu.operand(s, i), cu);
        }
        const float fg = (float)vg.s[i] * kUnpackScaledInv, fu = (float)vu.s[i] * kUnpackScaledInv;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          gate[i][e] = __builtin_fmaf(cg[e], fg, gate[i][e]);
          up[i][e] = __builtin_fmaf(cu[e], fu, up[i][e]);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      *reinterpret_cast<floatx4*>(&part[wave][0][4 * kq + e][4 * l16]) = floatx4{gate[0][e], gate[1][e], gate[2][e], gate[3][e]};
      *reinterpret_cast<floatx4*>(&part[wave][1][4 * kq + e][4 * l16]) = floatx4{up[0][e], up[1][e], up[2][e], up[3][e]};
    }
    __syncthreads();
    for (uint32_t o = tid; o < 16 * 64; o += kUpWaves * 64) {
      const uint32_t r = o / 64, c = o % 64;
      if (r0 + r >= rows) break;
      float y[1] = {0.f}, z = 0.f;
#pragma unroll
      for (int w = 0; w < kUpWaves; ++w) {
        y[0] += part[w][0][r][c];
        z += part[w][1][r][c];
      }
      activations<1>(y, p.act);
      // rounded to f16, as the next product's other operand
      p.h[((size_t)b * kBlock * p.top_k + route.first + r0 + r) * I + n0 + c] = __builtin_bit_cast(uint16_t, (_Float16)(y[0] * z));
    }
    __syncthreads();
  }
}

// 64 hidden columns of one part of the (active expert, group) units, for RT tiles of 16 tokens
template <int RT>
__global__ void __launch_bounds__(kDownWaves * 64) moe_down_kernel(Moe p) {
  __shared__ float part[kDownWaves][16][64];
  __shared__ uint32_t last;
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l16 = lane & 15, kq = lane >> 4;
  const uint32_t H = p.hidden, I = p.inner, groups = I / kGroup, strips = H / 64;
  const uint32_t b = blockIdx.y, strip = blockIdx.x % strips, split = blockIdx.x / strips, n0 = strip * 64, col = n0 + 4 * l16;
  const uint32_t tokens = p.tokens - b * kBlock < kBlock ? p.tokens - b * kBlock : kBlock;
  const u64 units = (u64)p.active[b] * groups;
  const uint32_t u0 = (uint32_t)(units * split / p.splits), u1 = (uint32_t)(units * (split + 1) / p.splits);
  struct Unit {
    Words v;
    MoeRoute route;
    uint32_t a, g;
    __device__ __forceinline__ void load(const Moe& p, uint32_t u, uint32_t b, uint32_t groups, uint32_t kq, uint32_t col) {
      a = u / groups;
      g = u - a * groups;
      route = p.route[(size_t)b * p.slots + a];
      v.load(p.w_down + (size_t)route.expert * (p.inner / 8) * p.hidden, p.s_down + (size_t)route.expert * groups * p.hidden,
             p.hidden, g, kq, col);
    }
  };
  floatx4 acc[RT][4] = {};
  auto multiply = [&](const Unit& u) {
    const uint16_t* const h = p.h + ((size_t)b * kBlock * p.top_k + u.route.first) * I + u.g * kGroup + 8 * kq;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const uint32_t here = (uint32_t)(u.route.mask >> (16 * r)) & 0xFFFFu;
      if (here == 0) continue;
      const uint32_t t = 16 * r + l16;
      half8_t hv[4];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        hv[s] = half8_t{};
        if (here >> l16 & 1)
          hv[s] = *reinterpret_cast<const half8_t*>(h + (size_t)__popcll(u.route.mask & ((1ull << t) - 1)) * I + 32 * s);
      }
      const floatx4 share = *reinterpret_cast<const floatx4*>(p.share + ((size_t)b * p.slots + u.a) * kBlock + 16 * r + 4 * kq);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        floatx4 c = {};
#pragma unroll
        for (int s = 0; s < 4; ++s) c = mfma16x16x32(hv[s], u.v.operand(s, i), c);
        const float f = (float)u.v.s[i] * kUnpackScaledInv;
        // nothing of an expert that a token did not choose, whatever its scales hold
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[r][i][e] = here >> (4 * kq + e) & 1 ? __builtin_fmaf(c[e] * f, share[e], acc[r][i][e]) : acc[r][i][e];
      }
    }
  };
  // the next unit's weights are on the way while one is multiplied
  Unit even, odd;
  uint32_t u = u0 + wave;
  if (u < u1) even.load(p, u, b, groups, kq, col);
  for (; u < u1; u += 2 * kDownWaves) {
    if (u + kDownWaves < u1) odd.load(p, u + kDownWaves, b, groups, kq, col);
    multiply(even);
    if (u + kDownWaves >= u1) break;
    if (u + 2 * kDownWaves < u1) even.load(p, u + 2 * kDownWaves, b, groups, kq, col);
    multiply(odd);
  }
  auto finish = [&](size_t t, uint32_t c, float y) {
    if (p.residual) y += h2f(p.residual[t * H + c]);
    p.y[t * H + c] = __builtin_bit_cast(uint16_t, (_Float16)y);
  };
#pragma unroll
  for (int r = 0; r < RT; ++r) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<floatx4*>(&part[wave][4 * kq + e][4 * l16]) = floatx4{acc[r][0][e], acc[r][1][e], acc[r][2][e], acc[r][3][e]};
    __syncthreads();
    for (uint32_t o = tid; o < 16 * 64; o += kDownWaves * 64) {
      const uint32_t t = 16 * r + o / 64, c = o % 64;
      if (t >= tokens) break;
      float y = 0.f;
#pragma unroll
      for (int w = 0; w < kDownWaves; ++w) y += part[w][o / 64][c];
      const size_t token = (size_t)b * kBlock + t;
      if (p.splits == 1) finish(token, n0 + c, y);
      else __hip_atomic_store(&p.partial[((size_t)split * p.tokens + token) * H + n0 + c], y, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
  }
  if (p.splits == 1) return;
  // The last of the strip's workgroups adds the parts, in order.  Parts are written and read past the L2 of one XCD (relaxed
  // atomics of the device's scope) and are there once the stores are done: a fence instead would have every workgroup
  // write back all that its L2 holds (5 times the time of this kernel).
  wait_vm<0>();
  __syncthreads();
  if (tid == 0) last = __hip_atomic_fetch_add(&p.arrived[(size_t)b * strips + strip], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == p.splits - 1;
  __syncthreads();
  if (!last) return;
  for (uint32_t o = tid; o < tokens * 64; o += kDownWaves * 64) {
    const size_t token = (size_t)b * kBlock + o / 64;
    float y = 0.f;
    for (uint32_t s = 0; s < p.splits; ++s)
      y += __hip_atomic_load(&p.partial[(s * (size_t)p.tokens + token) * H + n0 + o % 64], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    finish(token, n0 + o % 64, y);
  }
}

}  // namespace

hipError_t launch_moe_w4a16(const Moe& p, hipStream_t stream) {
  const uint32_t blocks = (p.tokens + kBlock - 1) / kBlock;
  if (p.tokens == 1) hipLaunchKernelGGL(moe_scores_kernel<1>, dim3(p.experts), dim3(256), 0, stream, p);
  else hipLaunchKernelGGL(moe_scores_kernel<4>, dim3(p.experts, (p.tokens + 3) / 4), dim3(256), 0, stream, p);
  if (hipError_t e = hipGetLastError()) return e;
  if (p.experts <= 64) hipLaunchKernelGGL(moe_routes_kernel<1>, dim3(blocks), dim3(1024), 0, stream, p);
  else if (p.experts <= 128) hipLaunchKernelGGL(moe_routes_kernel<2>, dim3(blocks), dim3(1024), 0, stream, p);
  else if (p.experts <= 256) hipLaunchKernelGGL(moe_routes_kernel<4>, dim3(blocks), dim3(1024), 0, stream, p);
  else hipLaunchKernelGGL(moe_routes_kernel<8>, dim3(blocks), dim3(1024), 0, stream, p);
  if (hipError_t e = hipGetLastError()) return e;
  hipLaunchKernelGGL(moe_up_kernel, dim3(p.inner / 64 * p.slots, blocks), dim3(kUpWaves * 64), 0, stream, p);
  if (hipError_t e = hipGetLastError()) return e;
  const dim3 grid(p.hidden / 64 * p.splits, blocks);
  const uint32_t tiles = p.tokens >= kBlock ? 4 : (p.tokens + 15) / 16;
  if (tiles == 1) hipLaunchKernelGGL(moe_down_kernel<1>, grid, dim3(kDownWaves * 64), 0, stream, p);
  else if (tiles == 2) hipLaunchKernelGGL(moe_down_kernel<2>, grid, dim3(kDownWaves * 64), 0, stream, p);
  else if (tiles == 3) hipLaunchKernelGGL(moe_down_kernel<3>, grid, dim3(kDownWaves * 64), 0, stream, p);
  else hipLaunchKernelGGL(moe_down_kernel<4>, grid, dim3(kDownWaves * 64), 0, stream, p);
  return hipGetLastError();
}

}  // namespace kaio
