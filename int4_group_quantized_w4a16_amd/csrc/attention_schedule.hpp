// Work of one paged-attention call: tiles of packed rows, blocks of keys, and
// which workgroup takes which.
//
// Packed rows.  The g = q_heads / kv_heads query heads that share a K/V head
// read the same keys, so the rows of a (sequence, K/V head) are numbered
// token * g + head and cut into tiles of R rows: one pass over the keys serves
// every head of the group.
//
// Blocks.  A tile sees the keys of `count` blocks of B: all from 0 up to its
// last row's position, or with a window the ns blocks that hold the sinks and
// those from the first row's window on; blocks between them are never touched.
// A tile that sees nothing still counts as one unit, in which its zeros are
// written.
//
// Split form.  The units of all tiles, K/V head by K/V head, form one line
// that is cut into equal parts, one per workgroup, wherever the cuts fall:
// lengths may differ as they like.  A tile inside one part is finished there;
// a part's first piece (of a tile begun earlier) and its last (of a tile that
// goes on) are partial results -- running maximum, sum and unnormalized
// output in f32 -- in the workspace, slots 2w and 2w + 1 of workgroup w.  The
// workgroup that begins a tile it does not finish notes the tile and how many
// workgroups go on with it, and a second kernel joins the pieces in order.
// The lengths are only known on the device, so every workgroup derives the
// line from them by itself (2 us; it needs one load of each array).
//
// Direct form, one workgroup per tile and K/V head, nothing to join: for calls
// with so few blocks that splitting does not pay (attention_direct in
// launch.hpp), and for those with four tiles for every resident workgroup or
// more than kSchedTiles of them.  The latter balance by themselves where the
// lengths are alike (256 decodes of 500 keys, 8 K/V heads of 128 columns: 98
// us, 5.4 TB/s); one of 100000 keys among them takes its own time, 1632 us.
#pragma once

#include "common.hpp"
#include "launch.hpp"
#include "paged.hpp"

namespace kaio {

struct Tile {
  uint32_t row0, rows;      // packed rows of the sequence
  int32_t q0;               // row of q of the sequence's first new token
  int32_t p0, p1;           // positions of the tile's first and last row
  int32_t hi;               // keys from here on are not visible to any row
  int32_t shift;            // position of row t of q = t + shift
  uint32_t ns, wb0, count;  // blocks: ns from 0, then from wb0
};

// A sequence's rows of q, [a, a + n) (inside q whatever q_start holds), and shift.
struct Seq {
  int32_t a, n, shift;
};
__device__ __forceinline__ int32_t clamp_row(int32_t x, uint32_t tokens) {
  return x < 0 ? 0 : x > (int32_t)tokens ? (int32_t)tokens : x;
}
__device__ __forceinline__ Seq seq_of(const PagedKV& kv, uint32_t s) {
  const int32_t lo = kv.q_start[s], hi = kv.q_start[s + 1], len = kv.lens[s];
  const int32_t a = clamp_row(lo, kv.tokens), b = clamp_row(hi, kv.tokens);
  return Seq{a, b > a ? b - a : 0, (len > 0 ? len : 0) - hi};
}
template <uint32_t R>
__device__ __forceinline__ uint32_t seq_tiles(const PagedAttention& p, const Seq& q) {
  return ((uint32_t)q.n * p.group.d + R - 1) / R;
}

template <uint32_t R, uint32_t B>
__device__ __forceinline__ Tile tile_info(const PagedAttention& p, const Seq& q, uint32_t i) {
  Tile t;
  const uint32_t rows = (uint32_t)q.n * p.group.d;
  t.q0 = q.a;
  t.row0 = i * R;
  t.rows = rows - t.row0 < R ? rows - t.row0 : R;
  t.shift = q.shift;
  t.p0 = q.a + (int32_t)p.group.div(t.row0) + t.shift;
  t.p1 = q.a + (int32_t)p.group.div(t.row0 + t.rows - 1) + t.shift;
  t.hi = t.p1 < (int32_t)p.kv.cap ? t.p1 + 1 : (int32_t)p.kv.cap;
  t.ns = t.wb0 = t.count = 0;
  if (t.hi <= 0 || p.kv.pages == 0) {
    t.hi = 0;
    return t;
  }
  const uint32_t nb = ((uint32_t)t.hi + B - 1) / B;
  if (p.window == 0) {
    t.count = nb;
    return t;
  }
  const int64_t lo = (int64_t)t.p0 - p.window + 1;
  const uint32_t sinks = p.sinks < (uint32_t)t.hi ? p.sinks : (uint32_t)t.hi;
  t.ns = (sinks + B - 1) / B;
  const uint32_t w = lo > 0 ? (uint32_t)lo / B : 0;
  t.wb0 = w > t.ns ? w : t.ns;
  t.count = t.ns + (nb > t.wb0 ? nb - t.wb0 : 0);
  return t;
}
__device__ __forceinline__ uint32_t units_of(const Tile& t) { return t.count ? t.count : 1; }

// Positions a row does not see below: a row at pos sees c > this or c < sinks.
__device__ __forceinline__ int32_t window_floor(const PagedAttention& p, int32_t pos) {
  if (p.window == 0) return -1;
  const int64_t f = (int64_t)pos - p.window;
  return f < -1 ? -1 : (int32_t)f;
}

// ---- the direct form: tile `index` of one K/V head; false past the last ----
template <uint32_t R>
__device__ __forceinline__ bool direct_tile(const PagedAttention& p, uint32_t index, uint32_t lane, uint32_t& seq,
                                            uint32_t& i) {
  uint32_t base = 0;
  for (uint32_t s0 = 0; s0 < p.kv.seqs; s0 += 64) {
    const uint32_t s = s0 + lane;
    uint32_t n = s < p.kv.seqs ? seq_tiles<R>(p, seq_of(p.kv, s)) : 0, end = n;
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) {
      const uint32_t o = __shfl_up(end, x);
      end += lane >= (uint32_t)x ? o : 0;
    }
    const uint64_t past = __ballot(base + end > index);
    if (past) {
      const int l = __builtin_ctzll(past);
      seq = s0 + l;
      i = index - (base + __builtin_amdgcn_readlane(end, l) - __builtin_amdgcn_readlane(n, l));
      return true;
    }
    base += __builtin_amdgcn_readlane(end, 63);
  }
  return false;
}

// ---- the split form ---------------------------------------------------------
constexpr uint32_t kSchedThreads = 256;
constexpr uint32_t kSchedPer = kSchedTiles / kSchedThreads;

struct Line {
  uint32_t first[kSchedTiles + 1];   // first tile of each sequence
  uint32_t start[kSchedTiles + 1];   // first unit of each tile
  Seq seq[kSchedTiles];
  uint32_t wave_sum[kSchedThreads / 64];
};

// exclusive prefix sums of v[kSchedPer] per thread (thread order), written to dst[0 .. n], the total in dst[n]
__device__ __forceinline__ void block_scan(const uint32_t (&v)[kSchedPer], uint32_t n, uint32_t* dst, uint32_t* wave_sum) {
  const uint32_t tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  uint32_t sum = 0;
#pragma unroll
  for (uint32_t k = 0; k < kSchedPer; ++k) sum += v[k];
  uint32_t end = sum;
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) {
    const uint32_t o = __shfl_up(end, x);
    end += lane >= (uint32_t)x ? o : 0;
  }
  if (lane == 63) wave_sum[wave] = end;
  __syncthreads();
  uint32_t at = end - sum;
#pragma unroll
  for (uint32_t w = 0; w < kSchedThreads / 64; ++w) at += w < wave ? wave_sum[w] : 0;
#pragma unroll
  for (uint32_t k = 0; k < kSchedPer; ++k) {
    if (tid * kSchedPer + k <= n) dst[tid * kSchedPer + k] = at;
    at += v[k];
  }
  if (tid == kSchedThreads - 1 && n == kSchedTiles) dst[n] = at;
  __syncthreads();
}

// index of the part of [0, n) that holds x: the last i with start[i] <= x (start[0] = 0, start[n] > x)
__device__ __forceinline__ uint32_t part_of(const uint32_t* start, uint32_t n, uint32_t x) {
  uint32_t lo = 0, hi = n;
  while (hi - lo > 1) {
    const uint32_t mid = (lo + hi) / 2;
    if (start[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Builds the line (every thread of a kSchedThreads workgroup); returns the tile count.
// seqs <= kSchedTiles and the host's bound on the tiles <= kSchedTiles hold in the split form.
template <uint32_t R, uint32_t B>
__device__ __forceinline__ uint32_t build_line(const PagedAttention& p, Line& line) {
  const uint32_t tid = threadIdx.x, n = p.kv.seqs;
  uint32_t v[kSchedPer];
#pragma unroll
  for (uint32_t k = 0; k < kSchedPer; ++k) {
    const uint32_t s = tid * kSchedPer + k;
    v[k] = 0;
    if (s < n) {
      line.seq[s] = seq_of(p.kv, s);
      v[k] = seq_tiles<R>(p, line.seq[s]);
    }
  }
  block_scan(v, n, line.first, line.wave_sum);
  // overlapping sequences (q_start not ascending) could have more tiles than rows: those past the bound are dropped
  const uint32_t tiles = line.first[n] < kSchedTiles ? line.first[n] : kSchedTiles;
#pragma unroll
  for (uint32_t k = 0; k < kSchedPer; ++k) {
    const uint32_t i = tid * kSchedPer + k;
    v[k] = 0;
    if (i < tiles) {
      const uint32_t s = part_of(line.first, n, i);
      v[k] = units_of(tile_info<R, B>(p, line.seq[s], i - line.first[s]));
    }
  }
  block_scan(v, tiles, line.start, line.wave_sum);
  return tiles;
}

// Inclusive prefix sum over the wave, on the vector unit alone (row shifts, then the rows' last lanes to the next).
__device__ __forceinline__ uint32_t wave_scan(uint32_t x) {
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xF, 0xF, false);   // row_shr:1
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xF, 0xF, false);
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xF, 0xF, false);
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xF, 0xF, false);
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xA, 0xF, false);   // row_bcast:15 to rows 1 and 3
  x += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xC, 0xF, false);   // row_bcast:31 to rows 2 and 3
  return x;
}

// The cut of `total` units over `parts` workgroups.
struct Cut {
  uint32_t per, rem;
  __device__ __forceinline__ uint32_t start(uint32_t w) const { return w * per + (w < rem ? w : rem); }
  __device__ __forceinline__ uint32_t owner(uint32_t u) const {
    const uint32_t big = rem * (per + 1);
    return u < big ? u / (per + 1) : rem + (u - big) / per;
  }
};
// no part shorter than kMinUnits where there are fewer units than that for everyone
template <uint32_t kMinUnits>
__device__ __forceinline__ Cut cut_of(uint32_t total, uint32_t workers) {
  uint32_t parts = (total + kMinUnits - 1) / kMinUnits;
  parts = parts < workers ? parts : workers;
  parts = parts ? parts : 1;
  const uint32_t per = total / parts;
  return Cut{per, total - per * parts};
}

// What a workgroup notes of a tile that it begins and others go on with.
struct JoinNote {
  uint32_t more;     // workgroups after it with a piece of the tile (0: no such tile)
  uint32_t head;
  int32_t q0;
  uint32_t row0, rows, pad[3];
};

// The pieces of one workgroup, in order.
template <uint32_t R, uint32_t B, uint32_t kMinUnits>
struct Walk {
  const PagedAttention& p;
  Line& line;             // split form only
  const bool split;
  uint32_t wg, unit = 0, end = 0, total = 0, tiles = 0, tile = 0;
  uint32_t head = 0;
  Cut cut{0, 0};
  // Up to 64 sequences of at most one tile each (decode): the line in registers, lane s sequence s, in every wave --
  // no LDS, no barrier (a call with one key per row: 8.2 us with the line in LDS, 6.3 so).
  bool small = false;
  uint32_t lane_start = 0, lane_units = 0;
  Seq lane_seq{};
  uint32_t seq_index = 0; // the piece's sequence
  Seq seq{};              // direct form: the same,
  uint32_t direct = 0;    // and the tile within it
  JoinNote note{};

  // the current piece: blocks b0 .. b1-1 of tile t; complete: all of it
  Tile t;
  uint32_t b0 = 0, b1 = 0;
  bool complete = true;

  // split form: every thread of the workgroup (barriers inside)
  __device__ __forceinline__ Walk(const PagedAttention& p_, Line& line_, bool split_, uint32_t tiles_bound, uint32_t lane)
      : p(p_), line(line_), split(split_), wg(xcd_remap(blockIdx.x, gridDim.x)) {
    if (split) {
      if (p.kv.seqs <= 64) {
        if (lane < p.kv.seqs) lane_seq = seq_of(p.kv, lane);
        const uint32_t n = seq_tiles<R>(p, lane_seq);
        if (!__any(n > 1)) {
          small = true;
          if (n) lane_units = units_of(tile_info<R, B>(p, lane_seq, 0));
          const uint32_t end_unit = wave_scan(lane_units);
          lane_start = end_unit - lane_units;
          total = __builtin_amdgcn_readlane(end_unit, 63);
          tiles = total ? 1 : 0;
        }
      }
      if (!small) {
        tiles = build_line<R, B>(p, line);
        total = line.start[tiles];
      }
      if (tiles == 0) return;
      const uint32_t all = total * p.kv.kv_heads;
      cut = cut_of<kMinUnits>(all, gridDim.x);
      unit = cut.start(wg);
      end = cut.start(wg + 1);
      if (end > all) end = all;
      if (unit >= end) return;
      head = unit / total;
      if (!small) tile = part_of(line.start, tiles, unit - head * total);
    } else {
      uint32_t s;
      head = wg / tiles_bound;
      // later tiles see more keys: they start first
      if (direct_tile<R>(p, tiles_bound - 1 - wg % tiles_bound, lane, s, direct)) {
        seq = seq_of(p.kv, s);
        seq_index = s;
        end = 1;
      }
    }
  }

  __device__ __forceinline__ bool next() {
    if (unit >= end) return false;
    if (split) {
      uint32_t tile_start;
      if (small) {
        if (unit - head * total == total) ++head;
        const uint32_t v = unit - head * total;
        const int l = __builtin_ctzll(__ballot(lane_start + lane_units > v));
        const Seq q{__builtin_amdgcn_readlane(lane_seq.a, l), __builtin_amdgcn_readlane(lane_seq.n, l),
                    __builtin_amdgcn_readlane(lane_seq.shift, l)};
        seq_index = l;
        tile_start = __builtin_amdgcn_readlane(lane_start, l);
        t = tile_info<R, B>(p, q, 0);
      } else {
        if (tile == tiles) {
          tile = 0;
          ++head;
        }
        seq_index = part_of(line.first, p.kv.seqs, tile);
        tile_start = line.start[tile];
        t = tile_info<R, B>(p, line.seq[seq_index], tile - line.first[seq_index]);
      }
      b0 = unit - head * total - tile_start;
      const uint32_t whole = units_of(t);
      b1 = whole - b0 < end - unit ? whole : b0 + (end - unit);
      complete = b0 == 0 && b1 == whole;
      if (b0 == 0 && !complete) {
        const uint32_t last = head * total + tile_start + whole - 1;
        note = JoinNote{cut.owner(last) - wg, head, t.q0, t.row0, t.rows, {}};
      }
      unit += b1 - b0;
      ++tile;
    } else {
      t = tile_info<R, B>(p, seq, direct);
      b1 = units_of(t);
      unit = end;
    }
    return true;
  }
  // rows of q that some sequence may have: [a, b)
  __device__ __forceinline__ void owned(uint32_t& a, uint32_t& b) const {
    const uint32_t T = p.kv.tokens, n = p.kv.seqs;
    if (n == 0) {
      a = b = T;
    } else if (small) {
      a = __builtin_amdgcn_readlane(lane_seq.a, 0);
      b = (uint32_t)__builtin_amdgcn_readlane(lane_seq.a + lane_seq.n, (int)n - 1);
    } else {
      a = (uint32_t)clamp_row(p.kv.q_start[0], T);
      b = (uint32_t)clamp_row(p.kv.q_start[n], T);
    }
  }
  __device__ __forceinline__ void leave_note() const {
    if (split && threadIdx.x == 0) static_cast<JoinNote*>(p.workspace)[wg] = note;
  }
};

}  // namespace kaio
