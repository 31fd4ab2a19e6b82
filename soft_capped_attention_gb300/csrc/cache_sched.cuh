// How a decode's work is split over a persistent grid.
//
// The live slots of sequence b are cut into tiles of TK keys; a unit of work is
// one tile of one (sequence, group of query heads).  Units are numbered
// sequence by sequence, group by group, tile by tile, and each CTA takes an equal
// run of them, to one unit, whatever the lengths.  A (sequence, group) counts
// kGroupCost units more than it has tiles (its first ones) for what its end costs,
// so that a CTA with many short sequences does not finish last.
//
// Where no sequence has more than kWholeTiles tiles (twice as many when there are
// groups enough for half of the CTAs), the units are whole (sequence, group)s instead:
// joining the parts of so short a one takes longer than reading it (100 keys of 8
// heads: 5.4 us against 8.9; 32 sequences of 50 to 300 keys, 8 heads: 8.3 against
// 11.1; one of 500 keys, 8 heads, is faster split: 9.5 against 10.1).
//
// A CTA's part of one (sequence, group) is a piece; a piece that is not the whole
// leaves (m, l, O) in the CTA's slot 2c (the piece at the start of its range) or
// 2c + 1 (the one at its end; pieces between the two are whole).  The CTA that
// leaves the last piece of a (sequence, group) joins them, in an order that their CTAs'
// numbers alone decide (join_pieces); it is found by a counter that belongs to the CTA where
// the group starts (at most one split group starts in a CTA) and returns to zero.
// Every warp computes the split from lens by itself, so the lengths stay on the
// device.
#pragma once

#include "cache_internal.h"
#include "tc_common.cuh"

namespace capattn {

constexpr int kGroupCost = 1;
constexpr int kWholeTiles = 4;
static_assert(kGroupCost >= 1, "an empty sequence has to belong to a CTA too");

struct SeqSpan {
  int32_t first, len;    // live slots [first, len) (before the test of pos)
  int32_t tile0, tiles;  // tiles that hold them
  int32_t units;         // tiles + kGroupCost
};

// The span of a sequence of length len as read.
template <int TK>
__device__ __forceinline__ SeqSpan span_of(const CacheParams& p, int len) {
  SeqSpan s;
  s.len = len;
  if (s.len < 0 || s.len > p.max_len) {
    atomicOr(p.status, kStatusBadLensBit);
    s.len = s.len < 0 ? 0 : p.max_len;
  }
  s.first = p.window_len > 0 && !p.pos ? max(0, s.len - p.window_len) : 0;
  s.tile0 = s.first / TK;
  s.tiles = (s.len + TK - 1) / TK - s.tile0;
  s.units = s.tiles + kGroupCost;
  return s;
}
template <int TK>
__device__ __forceinline__ SeqSpan seq_span(const CacheParams& p, int b) { return span_of<TK>(p, p.lens[b]); }

// Inclusive sum over the lanes.
__device__ __forceinline__ int lane_scan(int x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

constexpr int kSchedSums = 256;

// Batches of more than 64: sums over runs of whole groups of 32 sequences, at most
// kSchedSums of them, in shared memory (built by all threads of the CTA); returns
// the units of all sequences.
__device__ __forceinline__ int run_groups(const CacheParams& p) {
  return ((p.B + 31) / 32 + kSchedSums - 1) / kSchedSums;
}
// (and the longest sequence's, in s_sums[kSchedSums .. kSchedSums + warps)).
template <int TK>
__device__ __noinline__ int sum_large(const CacheParams& p, int warp, int lane, int warps, int* s_sums, int* longest) {
  const int run = run_groups(p) * 32, runs = (p.B + run - 1) / run;
  int top = 0;
#pragma unroll 4
  for (int r = warp; r < runs; r += warps) {
    int sum = 0;
    for (int x = r * run + lane; x < min(p.B, (r + 1) * run); x += 32) {
      const int n = seq_span<TK>(p, x).units;
      sum += n;
      top = max(top, n);
    }
    sum = __reduce_add_sync(0xFFFFFFFFu, sum);
    if (lane == 0) s_sums[r] = sum;
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if (lane == 0) s_sums[kSchedSums + warp] = top;
  __syncthreads();
  int all = 0;
  for (int r = lane; r < runs; r += 32) all += s_sums[r];
  *longest = __reduce_max_sync(0xFFFFFFFFu, lane < warps ? s_sums[kSchedSums + lane] : 0);
  return __reduce_add_sync(0xFFFFFFFFu, all);
}
// The sequence that holds unit `want`, its length as read and the units before it.
template <int TK>
__device__ __noinline__ int3 find_large(const CacheParams& p, int lane, const int* s_sums, int want) {
  const int run = run_groups(p) * 32, runs = (p.B + run - 1) / run;
  int before = 0, from = 0;
  for (int r0 = 0; r0 < runs; r0 += 32) {
    const int x = r0 + lane < runs ? s_sums[r0 + lane] : 0, up = lane_scan(x, lane);
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, want < before + up);
    if (mask) {
      from = (r0 + __ffs(mask) - 1) * run;
      before += __shfl_sync(0xFFFFFFFFu, up - x, __ffs(mask) - 1);
      break;
    }
    before += __shfl_sync(0xFFFFFFFFu, up, 31);
  }
  for (int b0 = from; b0 < p.B; b0 += 32) {
    const int r = b0 + lane < p.B ? p.lens[b0 + lane] : 0;
    const int x = b0 + lane < p.B ? span_of<TK>(p, r).units : 0, up = lane_scan(x, lane);
    const uint32_t mask = __ballot_sync(0xFFFFFFFFu, want < before + up);
    if (mask) {
      const int l = __ffs(mask) - 1;
      return make_int3(b0 + l, __shfl_sync(0xFFFFFFFFu, r, l), before + __shfl_sync(0xFFFFFFFFu, up - x, l));
    }
    before += __shfl_sync(0xFFFFFFFFu, up, 31);
  }
  return make_int3(p.B - 1, 0, before);
}

// Walks a CTA's pieces (every lane of a warp alike).
template <int TK>
struct PieceIter {
  uint32_t units, ctas;           // all units, the CTAs that share them
  uint32_t q, more;               // units / ctas, units % ctas
  uint32_t u, end, begin;         // next unit, this CTA's range
  int b, vh, t0;                  // the next piece: sequence, group, first unit of the group
  int len;                        // lens[b], read ahead of its use
  // of the piece that next() gave
  int n;                   // tiles (maybe none)
  bool whole;
  int slot;                // its partial slot, when not whole
  uint32_t s0, s1;         // units [s0, s1) of its (sequence, group)

  bool groups;             // the units are whole (sequence, group)s: none is split

  // All threads of the CTA (whole warps) build it together; s_sums: kSchedSums + 32
  // ints of shared memory, written by this alone.
  __device__ PieceIter(const CacheParams& p, int warp, int lane, int warps, int* s_sums) {
    b = vh = t0 = len = 0;
    // A batch of 64 stays in registers: one read of lens decides it, in little code
    // (which every launch fetches anew: unrolled over more sequences, or with the
    // large batch's path inline, this cost a launch 1 to 3 us).
    int raw0 = 0, raw1 = 0, n0 = 0, n1 = 0, sum0 = 0, all, longest;
    const bool small = p.B <= 64;
    if (small) {
      if (lane < p.B) raw0 = p.lens[lane];
      if (lane + 32 < p.B) raw1 = p.lens[lane + 32];
      if (lane < p.B) n0 = span_of<TK>(p, raw0).units;
      if (lane + 32 < p.B) n1 = span_of<TK>(p, raw1).units;
      sum0 = __reduce_add_sync(0xFFFFFFFFu, n0);
      all = sum0 + __reduce_add_sync(0xFFFFFFFFu, n1);
      longest = __reduce_max_sync(0xFFFFFFFFu, max(n0, n1));
    } else {
      all = sum_large<TK>(p, warp, lane, warps, s_sums, &longest);
    }
    groups = longest <= (2 * p.B * p.VH >= p.ctas ? 2 : 1) * kWholeTiles + kGroupCost;
    units = (uint32_t)(groups ? p.B : all) * (uint32_t)p.VH;
    ctas = min((uint32_t)p.ctas, max(1u, units / (uint32_t)(groups ? 1 : p.min_tiles)));
    q = units / ctas;
    more = units - q * ctas;
    begin = u = begin_of(blockIdx.x);
    end = begin_of(blockIdx.x + 1);
    if (u >= end) return;
    const int want = (int)(u / (uint32_t)p.VH);  // counted over the sequences
    int before;
    if (groups) {
      b = want;
      vh = (int)(u - (uint32_t)want * (uint32_t)p.VH);
      len = p.lens[b];
      if (!small) __syncthreads();
      return;
    }
    if (small) {
      const bool low = want < sum0;
      const int x = low ? n0 : n1;
      before = low ? 0 : sum0;
      const int up = lane_scan(x, lane);
      const int hit = __ffs(__ballot_sync(0xFFFFFFFFu, want < before + up)) - 1;
      before += __shfl_sync(0xFFFFFFFFu, up - x, hit);
      len = __shfl_sync(0xFFFFFFFFu, low ? raw0 : raw1, hit);
      b = low ? hit : hit + 32;
    } else {
      const int3 f = find_large<TK>(p, lane, s_sums, want);
      b = f.x;
      len = f.y;
      before = f.z;
      __syncthreads();  // every warp has read s_sums (all of them get here: the range is the CTA's)
    }
    const SeqSpan sp = span_of<TK>(p, len);
    const uint32_t in = u - (uint32_t)before * (uint32_t)p.VH;
    vh = (int)(in / (uint32_t)sp.units);
    t0 = (int)(in % (uint32_t)sp.units);
  }
  // First unit of CTA c's range, and the CTA that holds a unit: the first `more` of
  // them take q + 1 units, the others q.
  __device__ __forceinline__ uint32_t begin_of(uint32_t c) const { return c >= ctas ? units : q * c + min(c, more); }
  __device__ __forceinline__ int cta_of(uint32_t x) const {
    const uint32_t cut = (q + 1) * more;
    return (int)(x < cut ? x / (q + 1) : more + (x - cut) / q);
  }
  // Gives the piece (b, vh, tiles [tile, tile + n) of the sequence's span).
  __device__ bool next(const CacheParams& p, int* b_out, int* vh_out, int* tile_out, SeqSpan* sp_out) {
    if (u >= end) return false;
    const SeqSpan sp = span_of<TK>(p, len);
    const int take = groups ? 1 : (int)min((uint32_t)(sp.units - t0), end - u);
    const int first = max(0, t0 - kGroupCost);
    n = groups ? sp.tiles : max(0, t0 + take - kGroupCost) - first;
    whole = groups || (t0 == 0 && take == sp.units);
    slot = 2 * (int)blockIdx.x + (u == begin ? 0 : 1);
    s0 = u - (uint32_t)t0;
    s1 = s0 + (uint32_t)sp.units;
    *b_out = b;
    *vh_out = vh;
    *tile_out = sp.tile0 + first;
    *sp_out = sp;
    u += (uint32_t)take;
    if (u < end) {
      t0 = 0;
      if (++vh == p.VH) {
        vh = 0;
        ++b;
        len = p.lens[b];  // not looked at before the next call
      }
    }
    return true;
  }
};

// The pieces of one split (sequence, group): CTAs c0 .. c1, and their slots.
struct Pieces {
  int c0, c1, late;  // late: the first one starts inside c0's range
  __device__ Pieces(int first, int last, int starts_late) : c0(first), c1(last), late(starts_late) {}
  template <int TK>
  __device__ explicit Pieces(const PieceIter<TK>& it) {
    c0 = it.cta_of(it.s0);
    c1 = it.cta_of(it.s1 - 1);
    late = it.s0 != it.begin_of(c0) ? 1 : 0;
  }
  __device__ __forceinline__ int slot_of(int c) const { return 2 * c + (c == c0 ? late : 0); }
};

// First of the query heads of group vh, its count, and the KV head.
struct HeadGroup {
  int h0, count, g;
};
__device__ __forceinline__ HeadGroup head_group(const CacheParams& p, int vh) {
  HeadGroup x;
  x.g = vh / p.HG;
  const int part = vh - x.g * p.HG;
  x.h0 = x.g * p.G + part * kDecodeHeads;
  x.count = min(kDecodeHeads, p.G - part * kDecodeHeads);
  return x;
}

// Page of a slot, checked (a bad page is flagged and read as page 0).
__device__ __forceinline__ int page_of(const CacheParams& p, int b, int slot) {
  const int page = p.table[(size_t)b * p.max_pages + (slot >> p.page_shift)];
  if (page < 0 || page >= p.num_pages) {
    atomicOr(p.status, kStatusBadPageBit);
    return 0;
  }
  return page;
}

// Adds up four parts of a head: maxima m (-inf: no live keys), sums l and this lane's
// columns of O.
template <int V>
__device__ __forceinline__ void merge_parts(const float (&m)[4], const float (&l)[4], const float (&o)[4][V],
                                            float (&y)[V], float* sum_out, float* top_out) {
  float top = -INFINITY, sum = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) top = fmaxf(top, m[w]);
#pragma unroll
  for (int x = 0; x < V; ++x) y[x] = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    // a part without live keys adds nothing; one with nothing but NaN scores (no
    // maximum, but a sum) comes through
    const float f = m[w] != -INFINITY ? __expf(m[w] - top) : l[w] != 0.f ? 1.f : 0.f;
    sum = fmaf(l[w], f, sum);
#pragma unroll
    for (int x = 0; x < V; ++x) y[x] = fmaf(o[w][x], f, y[x]);
  }
  *sum_out = sum;
  *top_out = top;
}

// The same for what four warps left of head e of four: results buf [4][4][D], maxima sm
// and sums sl [4][4], all shared; a lane takes D / 32 columns.
template <int D>
__device__ __forceinline__ void merge_warps(const float* buf, const float* sm, const float* sl, int e, int lane,
                                            float (&y)[D / 32], float* sum_out, float* top_out) {
  constexpr int V = D / 32;
  float m[4], l[4], o[4][V];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    m[w] = sm[4 * w + e];
    l[w] = sl[4 * w + e];
#pragma unroll
    for (int x = 0; x < V; ++x) o[w][x] = buf[(w * 4 + e) * D + lane * V + x];
  }
  merge_parts<V>(m, l, o, y, sum_out, top_out);
}

// Counts a piece in (one thread, after everything of the piece's partial results
// has been written by threads that it has met at a barrier): whether it is the
// last one of its (sequence, group).
__device__ __forceinline__ bool count_piece(const CacheParams& p, const Pieces& pc) {
  // release: with the barrier before it, it covers what the others wrote; acquire:
  // for those that read the other pieces after the next barrier
  uint32_t before;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(p.counters + pc.c0) : "memory");
  const bool last = before == (uint32_t)(pc.c1 - pc.c0);
  if (last) p.counters[pc.c0] = 0u;
  return last;
}
// The same for a piece that one whole warp has left (every lane gets the answer): the
// lanes meet before lane 0 counts, and after it, since a shuffle alone orders no memory
// and the last piece's lanes go on to read what other CTAs wrote.
__device__ __forceinline__ bool count_piece_warp(const CacheParams& p, const Pieces& pc, int lane) {
  int last = 0;
  __syncwarp();
  if (lane == 0) last = count_piece(p, pc);
  __syncwarp();
  return __shfl_sync(0xFFFFFFFFu, last, 0) != 0;
}

// A running sum over some of a head's pieces: maximum m (0 until there is one), sum and
// this lane's V columns of O.
template <int V>
struct Chain {
  float m, l, o[V];
  bool any;
  __device__ __forceinline__ Chain() : m(0.f), l(0.f), any(false) {
#pragma unroll
    for (int x = 0; x < V; ++x) o[x] = 0.f;
  }
  // N pieces in order (one that is not there: maximum -inf, zeros).  Fewer than four give
  // what four would whose last ones are not there, but for the sign of a zero.
  template <int N>
  __device__ __forceinline__ void add(const float2 (&ml)[N], const float (&v)[N][V]) {
    float top = ml[0].x;
#pragma unroll
    for (int y = 1; y < N; ++y) top = fmaxf(top, ml[y].x);
    if (top != -INFINITY) {
      top = any ? fmaxf(top, m) : top;
      const float scale = any ? __expf(m - top) : 1.f;  // without a maximum l and o are 0 or NaN
      l *= scale;
#pragma unroll
      for (int x = 0; x < V; ++x) o[x] *= scale;
      m = top;
      any = true;
    }
#pragma unroll
    for (int y = 0; y < N; ++y) {
      const float w = __expf(ml[y].x - m);
      l = fmaf(ml[y].y, w, l);
#pragma unroll
      for (int x = 0; x < V; ++x) o[x] = fmaf(v[y][x], w, o[x]);
    }
  }
};

// Piece c of a head: its (m, l) and this lane's columns; not there when !in.
template <int D>
__device__ __forceinline__ void load_piece(const CacheParams& p, const Pieces& pc, int c, int head, int lane, bool in,
                                           float2& ml, float (&v)[D / 32]) {
  constexpr int V = D / 32;
  ml = make_float2(-INFINITY, 0.f);
#pragma unroll
  for (int x = 0; x < V; ++x) v[x] = 0.f;
  if (!in) return;
  const size_t at = (size_t)pc.slot_of(c) * kDecodeHeads + head;
  ml = __ldcg(&p.part_ml[at]);
  const float* po = p.part_o + at * D + lane * V;
  if constexpr (V == 4) {
    const float4 f = __ldcg(reinterpret_cast<const float4*>(po));
    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
  } else {
    const float2 f = __ldcg(reinterpret_cast<const float2*>(po));
    v[0] = f.x; v[1] = f.y;
  }
}

// Writes row `row` of o and lse from the sum of its pieces.
template <typename T, int V>
__device__ __forceinline__ void write_row(const CacheParams& p, size_t row, int lane, const float (&y)[V], float sum,
                                          float top) {
#pragma unroll
  for (int x = 0; x < V; ++x) static_cast<T*>(p.o)[row * (32 * V) + lane * V + x] = (T)(sum == 0.f ? 0.f : y[x] / sum);
  if (lane == 0) p.lse[row] = sum == 0.f ? -INFINITY : top + logf(sum);
}

// The join by one warp: four chains of HEADS heads at a time, 4 / HEADS pieces of each in
// flight (with more than one head: all that there are).
template <typename T, int D, int HEADS>
__device__ __forceinline__ void join_by_warp(const CacheParams& p, const Pieces& pc, int b, const HeadGroup& hg, int lane) {
  constexpr int V = D / 32, N = 4 / HEADS;
  for (int h0 = 0; h0 < hg.count; h0 += HEADS) {
    Chain<V> chains[HEADS][4];
    for (int c = pc.c0; c <= pc.c1; c += 4 * N) {
      float2 ml[HEADS][4][N];
      float v[HEADS][4][N][V];
#pragma unroll
      for (int e = 0; e < HEADS; ++e)
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
          for (int y = 0; y < N; ++y)
            load_piece<D>(p, pc, c + w + 4 * y, h0 + e, lane, c + w + 4 * y <= pc.c1 && h0 + e < hg.count, ml[e][w][y],
                          v[e][w][y]);
#pragma unroll
      for (int e = 0; e < HEADS; ++e)
#pragma unroll
        for (int w = 0; w < 4; ++w)
          if (c + w <= pc.c1) chains[e][w].template add<N>(ml[e][w], v[e][w]);
      if (HEADS > 1) break;
    }
#pragma unroll
    for (int e = 0; e < HEADS; ++e) {
      if (h0 + e >= hg.count) break;
      float m[4], l[4], o[4][V], y[V], sum, top;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        m[w] = chains[e][w].any ? chains[e][w].m : -INFINITY;
        l[w] = chains[e][w].l;
#pragma unroll
        for (int x = 0; x < V; ++x) o[w][x] = chains[e][w].o[x];
      }
      merge_parts<V>(m, l, o, y, &sum, &top);
      write_row<T, V>(p, (size_t)b * p.Hq + hg.h0 + h0 + e, lane, y, sum, top);
    }
  }
}

// Adds the pieces of (b, group) up and writes o and lse, by WARPS warps (4 that meet
// at named barrier `bar`, with buf 4 x 4 x D floats and sbuf 32, both shared; or 1).
// Either way four chains take every fourth piece each, four pieces at a time with a
// running maximum, so that nothing is read twice or waits for a first pass, and are then
// added in order: the result does not depend on which CTA came last.  Four warps take a
// chain each, of four heads at a time; one warp all four, of as many heads at a time as
// its registers hold (a head at a time whatever the pieces: 32 users of 1024 to 3968
// keys a pass of 25 us against 23).
template <typename T, int D, int WARPS>
__device__ __forceinline__ void join_pieces(const CacheParams& p, const Pieces& pc, int b, const HeadGroup& hg, int warp,
                                            int lane, int bar, float* buf, float* sbuf) {
  static_assert(WARPS == 1 || WARPS == 4, "four chains, by one warp or four");
  constexpr int V = D / 32;
  if constexpr (WARPS == 1) {
    const int n = pc.c1 - pc.c0 + 1;
    if (n <= 4) join_by_warp<T, D, 4>(p, pc, b, hg, lane);
    else if (n <= 8) join_by_warp<T, D, 2>(p, pc, b, hg, lane);
    else join_by_warp<T, D, 1>(p, pc, b, hg, lane);
  } else {
    for (int g0 = 0; g0 < hg.count; g0 += 4) {
      const int heads = min(4, hg.count - g0);
      Chain<V> chains[4];  // of the four heads
      for (int c = pc.c0 + warp; c <= pc.c1; c += 16) {
        float2 ml[4][4];
        float v[4][4][V];
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            load_piece<D>(p, pc, c + 4 * y, g0 + e, lane, c + 4 * y <= pc.c1 && e < heads, ml[e][y], v[e][y]);
#pragma unroll
        for (int e = 0; e < 4; ++e) chains[e].template add<4>(ml[e], v[e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int x = 0; x < V; ++x) buf[(warp * 4 + e) * D + lane * V + x] = chains[e].o[x];
        if (lane == 0) {
          sbuf[warp * 4 + e] = chains[e].any ? chains[e].m : -INFINITY;
          sbuf[16 + warp * 4 + e] = chains[e].l;
        }
      }
      named_bar_sync(bar, 128);
      if (warp < heads) {  // a head a warp
        float y[V], sum, top;
        merge_warps<D>(buf, sbuf, sbuf + 16, warp, lane, y, &sum, &top);
        write_row<T, V>(p, (size_t)b * p.Hq + hg.h0 + g0 + warp, lane, y, sum, top);
      }
      named_bar_sync(bar, 128);
    }
  }
}

}  // namespace capattn
