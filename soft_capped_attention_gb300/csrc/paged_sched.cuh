// How attention of many new tokens is split over a persistent grid.
//
// A query tile is `tokens` consecutive new tokens of one sequence with the query heads
// of one KV head (or a part of them); its keys are cut into steps of TK slots, from the
// first that its oldest window reaches to its last token's own slot.  A unit of work is
// one step; a tile counts kTileCost units more (its first ones) for its start and end.
// Units are numbered by sequence, KV head (part), tile, step, and each CTA takes an equal
// run of them, so that causal tiles of unequal length, long caches with few new tokens
// and batches of unequal sequences all end together.  A tile that several CTAs share
// leaves partial results, which a second kernel adds up in the order of their CTAs
// (paged_finish.cu).
//
// Where no tile has more than kWholeSteps steps, units are whole tiles: joining costs more.
// (With 10 in its place a tree of 24 tokens on 1021 keys took 19.2 us, split 14.9.  A CTA takes
// two units at least, for the same reason.  Tiles that count one, two, three units more: nine
// unequal prompts 278, 257, 261 us.)
//
// The steps of a sequence's tiles are sums of floor((a t + b) / TK) over tiles t, which
// Euclid's recursion gives in a few divisions (floor_sum), so every CTA finds its range
// from lens and cu_new by itself; nothing is planned ahead and lengths stay on the device.
#pragma once

#include <limits.h>

#include "cache_math.cuh"
#include "paged_internal.h"
#include "tc_common.cuh"

namespace capattn {

constexpr int kTileCost = 2;
constexpr int kWholeSteps = 2;

struct SeqShape {
  int32_t row0, n, len, base;  // first row, new tokens, slots, slots before the new tokens
};

// A sequence's rows and slots, checked: one that is out of range has no new tokens.
__device__ __forceinline__ SeqShape seq_shape(const PagedParams& p, int b) {
  SeqShape s;
  s.row0 = p.cu_new[b];
  const int end = p.cu_new[b + 1];
  s.len = p.c.lens[b];
  uint32_t bad = 0;
  if (s.len < 0 || s.len > p.c.max_len) bad |= kStatusBadLensBit;
  if (s.row0 < 0 || end < s.row0 || end > p.n_rows) bad |= kStatusBadNewRowsBit;
  s.n = bad ? 0 : end - s.row0;
  if (!bad && s.n > s.len) bad |= kStatusBadNewRowsBit;
  if (p.parents && s.n > CAPATTN_PAGED_MAX_TREE) bad |= kStatusBadParentBit;
  if (bad) {
    atomicOr(p.c.status, bad);
    s.n = 0;
    s.len = 0;
  }
  s.base = s.len - s.n;
  return s;
}

// sum of floor((a i + b) / M) over 0 <= i < n; a <= M, M a power of two.  32 bits hold all
// but the sum: a n and b are at most a sequence's slots (2^30) and a little more.
template <int M>
__device__ __forceinline__ uint64_t floor_sum(uint32_t n, uint32_t a, uint32_t b) {
  uint64_t sum = (uint64_t)n * (b / M);
  b %= M;
  if (a == M) return n ? sum + (uint64_t)n * (n - 1) / 2 : 0;  // (b < M)
  uint32_t m = M;
  for (;;) {
    const uint32_t y = a * n + b;
    if (y < m) return sum;
    n = y / m;
    b = y % m;
    const uint32_t t = m;
    m = a;
    a = t;
    sum += (uint64_t)n * (n - 1) / 2 * (a / m) + (uint64_t)n * (b / m);
    a %= m;
    b %= m;
  }
}

// x / y where x rarely needs more than 32 bits (a division of 64 is some 100 instructions).
__device__ __forceinline__ uint64_t quotient(uint64_t x, uint32_t y) {
  return (x >> 32) == 0 ? (uint64_t)((uint32_t)x / y) : x / y;
}

template <int TK>
struct Tiles {
  // First slot (not below 0) that a tile's window reaches, and its steps.
  static __device__ __forceinline__ int first_slot(const PagedParams& p, const SeqShape& s, int t) {
    if (p.c.window_len <= 0 || p.c.pos) return 0;
    return max(0, s.base + (p.parents ? 0 : t * p.tokens) - p.c.window_len + 1);
  }
  static __device__ __forceinline__ int steps(const PagedParams& p, const SeqShape& s, int t) {
    const int last = s.base + min(s.n, (t + 1) * p.tokens);
    return (last + TK - 1) / TK - first_slot(p, s, t) / TK;
  }
  static __device__ __forceinline__ int count(const PagedParams& p, const SeqShape& s) {
    return (s.n + p.tokens - 1) / p.tokens;
  }
  // Units of the tiles before tile t < count (every one of them has all its tokens).
  static __device__ __forceinline__ int64_t before(const PagedParams& p, const SeqShape& s, int t, bool whole) {
    if (whole || t == 0) return t;
    int64_t sum = (int64_t)floor_sum<TK>(t, p.tokens, s.base + p.tokens + TK - 1) + (int64_t)t * kTileCost;
    if (p.c.window_len > 0 && !p.c.pos) {
      const int x0 = s.base - p.c.window_len + 1;
      if (p.parents) {
        sum -= (int64_t)t * (max(0, x0) / TK);
      } else {
        const int skip = x0 < 0 ? (-x0 + p.tokens - 1) / p.tokens : 0;
        if (t > skip) sum -= (int64_t)floor_sum<TK>(t - skip, p.tokens, x0 + skip * p.tokens);
      }
    }
    return sum;
  }
  static __device__ __forceinline__ int64_t units(const PagedParams& p, const SeqShape& s, bool whole) {
    const int c = count(p, s);
    if (c == 0 || whole) return c;
    return before(p, s, c - 1, false) + steps(p, s, c - 1) + kTileCost;
  }
};

// The units of all sequences, shared out.
struct Shares {
  uint64_t units, q;   // all; those of a CTA
  uint32_t more, ctas; // CTAs that take one more
  bool whole;
  __device__ __forceinline__ uint64_t begin_of(uint32_t c) const {
    return c >= ctas ? units : q * c + (c < more ? c : more);
  }
  __device__ __forceinline__ int cta_of(uint64_t x) const {
    const uint64_t cut = (q + 1) * more;
    if ((units >> 32) == 0) {
      const uint32_t y = (uint32_t)x, z = (uint32_t)cut;
      return (int)(y < z ? y / ((uint32_t)q + 1u) : more + (y - z) / (uint32_t)q);
    }
    return (int)(x < cut ? x / (q + 1) : more + (x - cut) / q);
  }
};

__device__ __forceinline__ int piece_slot(const Piece& x, int c) { return 2 * c + (c == x.c0 ? x.late : 0); }

__device__ __forceinline__ uint64_t lane_scan64(uint64_t x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint64_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// The shares, and where this CTA's range begins.
struct Schedule {
  Shares sh;
  int32_t b;        // its first sequence
  uint64_t in;      // units of that sequence before it
};
struct ScheduleMem {
  Schedule out;
  int32_t longest[32];
  uint64_t sums[32], tiles[32];
};

__device__ __forceinline__ Shares shares_of(const PagedParams& p, uint64_t sum, uint64_t tiles, int longest) {
  Shares sh;
  sh.whole = longest <= kWholeSteps;
  sh.units = (uint64_t)(p.c.Hkv * p.parts) * (sh.whole ? tiles : sum);
  const uint64_t want = quotient(sh.units, sh.whole ? 1 : p.min_units);
  sh.ctas = (uint32_t)(want < 1 ? 1 : want < (uint64_t)gridDim.x ? want : gridDim.x);
  sh.q = quotient(sh.units, sh.ctas);
  sh.more = (uint32_t)(sh.units - sh.q * sh.ctas);
  return sh;
}

// What sequences [b0, b1) have: units, tiles, the most steps of a tile.
template <int TK>
__device__ __forceinline__ void sum_sequences(const PagedParams& p, int b0, int b1, uint64_t* sum, uint64_t* tiles,
                                              int* longest) {
  *sum = *tiles = 0;
  *longest = 0;
  for (int b = b0; b < b1; ++b) {
    const SeqShape s = seq_shape(p, b);
    const int c = Tiles<TK>::count(p, s);
    if (c == 0) continue;
    *sum += Tiles<TK>::units(p, s, false);
    *tiles += c;
    // (a windowed tile never has more steps than its window and its tokens span)
    *longest = max(*longest, Tiles<TK>::steps(p, s, c - 1));
    if (c > 1) *longest = max(*longest, Tiles<TK>::steps(p, s, c - 2));
  }
}

// The start of range u0, if it lies in sequences [b0, b1), which `at` units come before.
template <int TK>
__device__ __forceinline__ bool find_start(const PagedParams& p, const Shares& sh, uint64_t u0, int b0, int b1,
                                           uint64_t at, uint64_t mine, int* b_out, uint64_t* in_out) {
  const uint64_t heads = (uint64_t)(p.c.Hkv * p.parts);
  if (mine == 0 || u0 < heads * at || u0 >= heads * (at + mine)) return false;
  int b = b0;
  for (; b + 1 < b1; ++b) {
    const uint64_t n = Tiles<TK>::units(p, seq_shape(p, b), sh.whole);
    if (u0 < heads * (at + n)) break;
    at += n;
  }
  *b_out = b;
  *in_out = u0 - heads * at;
  return true;
}

// Batches of at most kWarpSeqs sequences: by one warp alone, which nobody waits for.
constexpr int kWarpSeqs = 128;
template <int TK>
__device__ __forceinline__ Schedule schedule_by_warp(const PagedParams& p, int lane) {
  const int per = (p.c.B + 31) / 32, b0 = min(p.c.B, lane * per), b1 = min(p.c.B, b0 + per);
  uint64_t sum, tiles;
  int longest;
  sum_sequences<TK>(p, b0, b1, &sum, &tiles, &longest);
  const uint64_t up_sum = lane_scan64(sum, lane), up_tiles = lane_scan64(tiles, lane);
  Schedule s;
  s.sh = shares_of(p, __shfl_sync(0xFFFFFFFFu, up_sum, 31), __shfl_sync(0xFFFFFFFFu, up_tiles, 31),
                   __reduce_max_sync(0xFFFFFFFFu, longest));
  int b = 0;
  uint64_t in = 0;
  const bool here = find_start<TK>(p, s.sh, s.sh.begin_of(blockIdx.x), b0, b1, s.sh.whole ? up_tiles - tiles : up_sum - sum,
                                   s.sh.whole ? tiles : sum, &b, &in);
  const uint32_t mask = __ballot_sync(0xFFFFFFFFu, here);
  const int from = mask ? __ffs(mask) - 1 : 0;
  s.b = __shfl_sync(0xFFFFFFFFu, b, from);
  s.in = __shfl_sync(0xFFFFFFFFu, in, from);
  return s;
}

// Larger ones: by all threads of the CTA, into m.out.
template <int TK>
__device__ __noinline__ void schedule_by_cta(const PagedParams& p, int threads, ScheduleMem& m) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = threads / 32;
  const int per = (p.c.B + threads - 1) / threads;
  const int b0 = min(p.c.B, (int)threadIdx.x * per), b1 = min(p.c.B, b0 + per);
  uint64_t sum, tiles;
  int longest;
  sum_sequences<TK>(p, b0, b1, &sum, &tiles, &longest);
  const uint64_t up_sum = lane_scan64(sum, lane), up_tiles = lane_scan64(tiles, lane);
  longest = __reduce_max_sync(0xFFFFFFFFu, longest);
  if (lane == 31) {
    m.sums[warp] = up_sum;
    m.tiles[warp] = up_tiles;
    m.longest[warp] = longest;
  }
  __syncthreads();
  const uint64_t ws = lane < warps ? m.sums[lane] : 0, wt = lane < warps ? m.tiles[lane] : 0;
  const uint64_t as = lane_scan64(ws, lane), at = lane_scan64(wt, lane);
  const int top = __reduce_max_sync(0xFFFFFFFFu, lane < warps ? m.longest[lane] : 0);
  const Shares sh = shares_of(p, __shfl_sync(0xFFFFFFFFu, as, 31), __shfl_sync(0xFFFFFFFFu, at, 31), top);
  if (threadIdx.x == 0) m.out.sh = sh;
  const uint64_t before = __shfl_sync(0xFFFFFFFFu, (sh.whole ? at : as) - (sh.whole ? wt : ws), warp) +
                          (sh.whole ? up_tiles - tiles : up_sum - sum);
  int b;
  uint64_t in;
  if (find_start<TK>(p, sh, sh.begin_of(blockIdx.x), b0, b1, before, sh.whole ? tiles : sum, &b, &in)) {
    m.out.b = b;
    m.out.in = in;
  }
  __syncthreads();
}

// Walks a CTA's pieces; every lane of one warp alike.
template <int TK>
struct PieceWalk {
  Shares sh;
  uint64_t u, end, begin;
  SeqShape s;
  int b, part, t, tiles, lane;
  int at;  // units of the tile before u

  __device__ PieceWalk(const PagedParams& p, const Schedule& m, int lane_in) {
    lane = lane_in;
    sh = m.sh;
    begin = u = sh.begin_of(blockIdx.x);
    end = sh.begin_of(blockIdx.x + 1);
    b = part = t = tiles = at = 0;
    if (u >= end) return;
    b = m.b;
    s = seq_shape(p, b);
    tiles = Tiles<TK>::count(p, s);
    const uint64_t per = (uint64_t)Tiles<TK>::units(p, s, sh.whole);
    part = (per >> 32) == 0 ? (int)quotient(m.in, (uint32_t)per) : (int)(m.in / per);
    const int64_t rest = (int64_t)(m.in - per * part);
    int lo = 0, hi = tiles;  // before(lo) <= rest < before(hi)
    while (hi - lo > 1) {
      const int w = (hi - lo + 31) / 32, x = lo + (lane + 1) * w;
      const bool in = x < hi && Tiles<TK>::before(p, s, x, sh.whole) <= rest;
      const int k = __popc(__ballot_sync(0xFFFFFFFFu, in));
      lo += k * w;
      hi = min(hi, lo + w);
    }
    t = lo;
    at = (int)(rest - Tiles<TK>::before(p, s, t, sh.whole));
  }

  // The next piece, or steps = -1.
  __device__ Piece next(const PagedParams& p) {
    Piece x;
    x.steps = -1;
    while (u < end) {
      const int steps = Tiles<TK>::steps(p, s, t), cost = sh.whole ? 0 : kTileCost;
      const int all = sh.whole ? 1 : steps + cost;
      const uint64_t left = end - u;
      const int take = left < (uint64_t)(all - at) ? (int)left : all - at;
      const int from = sh.whole ? 0 : max(0, at - cost), to = sh.whole ? steps : max(0, at + take - cost);
      if (to > from) {
        const uint64_t s0 = u - at + cost;  // the tile's first step
        x.b = b;
        x.part = part;
        x.row0 = s.row0;
        x.n = s.n;
        x.base = s.base;
        x.len = s.len;
        x.i0 = t * p.tokens;
        x.count = min(p.tokens, s.n - x.i0);
        x.first = Tiles<TK>::first_slot(p, s, t);
        x.tile0 = x.first / TK + from;
        x.steps = to - from;
        x.whole = from == 0 && to == steps;
        x.slot = x.c0 = x.c1 = x.late = 0;
        if (!x.whole) {
          x.c0 = sh.cta_of(s0);
          x.c1 = sh.cta_of(s0 + steps - 1);
          x.late = s0 > sh.begin_of(x.c0) ? 1 : 0;
          x.slot = piece_slot(x, blockIdx.x);
        }
      }
      u += take;
      at = 0;
      if (u < end && ++t == tiles) {
        t = 0;
        if (++part == p.c.Hkv * p.parts) {
          part = 0;
          next_sequence(p);
        }
      }
      if (x.steps > 0) break;
    }
    return x;
  }

  // The next sequence that has new tokens (there is one: the range goes on).
  __device__ __forceinline__ void next_sequence(const PagedParams& p) {
    for (int b0 = b + 1; b0 < p.c.B; b0 += 32) {
      SeqShape x{};
      if (b0 + lane < p.c.B) x = seq_shape(p, b0 + lane);
      const uint32_t some = __ballot_sync(0xFFFFFFFFu, x.n > 0);
      if (some == 0u) continue;
      const int l = __ffs(some) - 1;
      b = b0 + l;
      s.row0 = __shfl_sync(0xFFFFFFFFu, x.row0, l);
      s.n = __shfl_sync(0xFFFFFFFFu, x.n, l);
      s.len = __shfl_sync(0xFFFFFFFFu, x.len, l);
      s.base = __shfl_sync(0xFFFFFFFFu, x.base, l);
      tiles = Tiles<TK>::count(p, s);
      return;
    }
    u = end;  // (never reached)
  }
};

// Row of the cache that holds a slot of sequence b (a bad page is flagged and read as page 0).
__device__ __forceinline__ size_t cache_row(const CacheParams& c, int b, int g, int slot) {
  int page = c.table[(size_t)b * c.max_pages + (slot >> c.page_shift)];
  if (page < 0 || page >= c.num_pages) {
    atomicOr(c.status, kStatusBadPageBit);
    page = 0;
  }
  return (((size_t)page * c.Hkv + g) << c.page_shift) + (slot & (c.page_size - 1));
}

// ---------------------------------------------------------------- live slots of a row
struct RowMask {
  int32_t lo, hi;    // live slots [lo, hi), before the test of pos
  int32_t node;      // with parents: the row's index among the new tokens, else -1
  int32_t row0, base;
  int32_t reach;     // with parents: ancestors (and itself) that the window reaches
  int32_t oldest;    // by pos: positions above this one
  const int32_t* pos;  // of the KV head, or null
};

// Row r0 + i's parent, checked (a bad one is flagged and taken for -1).
__device__ __forceinline__ int parent_of(const PagedParams& p, int row0, int i) {
  const int up = __ldg(p.parents + row0 + i);
  if (up < -1 || up >= i) {
    atomicOr(p.c.status, kStatusBadParentBit);
    return -1;
  }
  return up;
}

__device__ __forceinline__ RowMask row_mask(const PagedParams& p, int b, int g, const SeqShape& s, int i) {
  RowMask r;
  const int W = p.c.window_len;
  r.row0 = s.row0;
  r.base = s.base;
  r.node = -1;
  r.reach = INT_MAX;
  r.pos = nullptr;
  r.oldest = 0;
  int depth = i;
  r.hi = s.base + i + 1;
  if (p.parents) {
    r.node = i;
    r.hi = s.base;
    depth = 0;
    const int up = parent_of(p, s.row0, i);
    if (W > 0) {
      r.reach = W;
      for (int x = up; x >= 0; x = parent_of(p, s.row0, x)) ++depth;
    }
    if (up < 0) r.reach = 1;
  }
  r.lo = 0;
  if (W > 0) {
    if (p.c.pos) {
      r.pos = p.c.pos + ((size_t)b * p.c.Hkv + g) * p.c.max_len;
      r.oldest = p.c.qpos[b] - s.n + 1 + depth - W;
    } else {
      r.lo = max(0, s.base + depth + 1 - W);
    }
  }
  return r;
}
__device__ __forceinline__ RowMask dead_row() {
  RowMask r;
  r.lo = r.hi = 0;
  r.node = -1;
  r.row0 = r.base = r.oldest = 0;
  r.reach = INT_MAX;
  r.pos = nullptr;
  return r;
}

// Whether the row's slots c0 .. c0 + n - 1 are all live without a look at pos or parents.
__device__ __forceinline__ bool all_live(const RowMask& r, int c0, int n) {
  return r.lo <= c0 && c0 + n <= r.hi && !r.pos;
}

// Whether the row has one live slot (by pos: not whether it has no more than one).
__device__ __forceinline__ bool only_one(const RowMask& r) {
  return r.node < 0 ? r.hi - r.lo == 1 : r.hi <= r.lo && r.reach == 1;
}

// Bit e: slot c0 + e is live, 32 of them.
__device__ __forceinline__ uint32_t live_slots(const PagedParams& p, const RowMask& r, int c0) {
  const int lo = min(max(r.lo - c0, 0), 32), hi = min(max(r.hi - c0, 0), 32);
  uint32_t bits = 0u;
  if (hi > lo) bits = (hi >= 32 ? 0xFFFFFFFFu : (1u << hi) - 1u) & ~((1u << lo) - 1u);  // lo < 32
  if (r.pos)
    for (uint32_t left = bits; left; left &= left - 1u) {
      const int e = __ffs(left) - 1;
      if (__ldg(r.pos + c0 + e) <= r.oldest) bits &= ~(1u << e);
    }
  if (r.node >= 0 && c0 + 32 > r.base) {
    // up the tree, as far as these slots (a parent comes before its children)
    int left = r.reach;
    for (int x = r.node; x >= 0 && r.base + x >= c0 && left > 0; x = parent_of(p, r.row0, x), --left)
      if (r.base + x < c0 + 32) bits |= 1u << (r.base + x - c0);
  }
  return bits;
}

}  // namespace capattn
