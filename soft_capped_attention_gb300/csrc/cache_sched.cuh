// How a decode's work is split over a persistent grid.
//
// The live slots of sequence b are cut into tiles of TK keys; a unit of work is
// one tile of one (sequence, group of query heads).  Units are numbered
// sequence by sequence, group by group, tile by tile, and CTA c takes units
// [c q, (c + 1) q): equal shares whatever the lengths.  A CTA's part of one
// (sequence, group) is a piece; a piece that is not the whole leaves (m, l, O) in
// the CTA's slot 2c (the piece at the start of its range) or 2c + 1 (the one at
// its end; pieces between the two are whole), and the join adds the pieces up in
// order: the CTA that leaves the last piece of a (sequence, group) does it, found
// by a counter per split group, which belongs to the CTA where the group starts
// (at most one split group starts in a CTA) and returns to zero.  Pieces are
// added in the order of their CTAs, whichever comes last.  Every role computes the split from lens by itself, so the lengths stay
// on the device.
#pragma once

#include "cache_internal.h"
#include "tc_common.cuh"

namespace capattn {

struct SeqSpan {
  int32_t first, len;    // live slots [first, len) (before the test of pos)
  int32_t tile0, tiles;  // tiles that hold them (one dead tile when there are none)
};

template <int TK>
__device__ __forceinline__ SeqSpan seq_span(const CacheParams& p, int b) {
  SeqSpan s;
  s.len = p.lens[b];
  if (s.len < 0 || s.len > p.max_len) {
    atomicOr(p.status, kStatusBadLensBit);
    s.len = s.len < 0 ? 0 : p.max_len;
  }
  s.first = p.window_len > 0 && !p.pos ? max(0, s.len - p.window_len) : 0;
  s.tile0 = s.first / TK;
  s.tiles = max(1, (s.len + TK - 1) / TK - s.tile0);
  return s;
}

// A CTA's share in units.
__device__ __forceinline__ uint32_t share_of(const CacheParams& p, uint32_t units) {
  return max((uint32_t)p.min_tiles, (units + p.ctas - 1) / (uint32_t)p.ctas);
}

// Inclusive sum over the lanes.
__device__ __forceinline__ int lane_scan(int x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// Walks a CTA's pieces (every lane of a warp alike).
template <int TK>
struct PieceIter {
  uint32_t u, end, begin, share;  // next unit, the CTA's range, its size
  int b, vh, t0;                  // the next piece: sequence, group, first tile of the group
  SeqSpan sp;
  // of the piece that next() gave
  int n;                   // tiles
  bool whole;
  int slot;                // its partial slot, when not whole
  int c0, c1;              // the CTAs that share its (sequence, group)
  bool first_at_begin;     // whether that starts at the begin of c0's range

  __device__ PieceIter(const CacheParams& p, int lane) {
    // the first 32 sequences' tiles stay in a register: one read of lens decides
    // a small batch
    const int n0 = lane < p.B ? seq_span<TK>(p, lane).tiles : 0;
    int all = n0;
    for (int x = lane + 32; x < p.B; x += 32) all += seq_span<TK>(p, x).tiles;
    const uint32_t units = (uint32_t)__reduce_add_sync(0xFFFFFFFFu, all) * (uint32_t)p.VH;
    share = share_of(p, units);
    begin = u = min(units, share * blockIdx.x);
    end = min(units, u + share);
    b = vh = t0 = 0;
    if (u >= end) return;
    const int want = (int)(u / (uint32_t)p.VH);  // the tile, counted over the sequences
    int before = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int x = b0 == 0 ? n0 : b0 + lane < p.B ? seq_span<TK>(p, b0 + lane).tiles : 0;
      const int up = lane_scan(x, lane);
      const uint32_t hit = __ballot_sync(0xFFFFFFFFu, want < before + up);
      if (hit) {
        const int l = __ffs(hit) - 1;
        b = b0 + l;
        before += __shfl_sync(0xFFFFFFFFu, up - x, l);
        break;
      }
      before += __shfl_sync(0xFFFFFFFFu, up, 31);
    }
    sp = seq_span<TK>(p, b);
    const uint32_t in = u - (uint32_t)before * (uint32_t)p.VH;
    vh = (int)(in / (uint32_t)sp.tiles);
    t0 = (int)(in % (uint32_t)sp.tiles);
  }
  // Gives the piece (b, vh, tiles [tile, tile + n) of the sequence's span).
  __device__ bool next(const CacheParams& p, int* b_out, int* vh_out, int* tile_out, SeqSpan* sp_out) {
    if (u >= end) return false;
    n = (int)min((uint32_t)(sp.tiles - t0), end - u);
    whole = t0 == 0 && n == sp.tiles;
    slot = 2 * (int)blockIdx.x + (u == begin ? 0 : 1);
    const uint32_t s0 = u - (uint32_t)t0;
    c0 = (int)(s0 / share);
    c1 = (int)((s0 + (uint32_t)sp.tiles - 1) / share);
    first_at_begin = s0 == share * (uint32_t)c0;
    *b_out = b;
    *vh_out = vh;
    *tile_out = sp.tile0 + t0;
    *sp_out = sp;
    u += (uint32_t)n;
    if (u < end) {
      t0 = 0;
      if (++vh == p.VH) {
        vh = 0;
        ++b;
        sp = seq_span<TK>(p, b);
      }
    }
    return true;
  }
  // Partial slot of the piece that CTA c (c0 .. c1) has of it.
  __device__ __forceinline__ int slot_of(int c) const { return 2 * c + (c == c0 && !first_at_begin ? 1 : 0); }
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

// Leaves a piece's last word and, in the CTA that comes last, joins the pieces of
// (b, group): called by 128 threads after they wrote their part of the partial
// results; `bar` is a named barrier of those threads, buf 4 x 4 x D floats,
// flag one int, both shared.  Warp w adds every fourth piece, four heads at a time.
template <typename T, int D, int TK>
__device__ __forceinline__ void join_pieces(const CacheParams& p, const PieceIter<TK>& it, int b, const HeadGroup& hg,
                                            int tid, int bar, float* buf, float* lbuf, int* flag) {
  __threadfence();
  named_bar_sync(bar, 128);
  if (tid == 0) {
    const uint32_t left = atomicAdd(&p.counters[it.c0], 1u);
    const bool last = left == (uint32_t)(it.c1 - it.c0);
    if (last) p.counters[it.c0] = 0u;
    __threadfence();
    *flag = last;
  }
  named_bar_sync(bar, 128);
  const bool last = *flag != 0;
  named_bar_sync(bar, 128);
  if (!last) return;
  constexpr int V = D / 32;
  const int warp = tid >> 5, lane = tid & 31;
  for (int g0 = 0; g0 < hg.count; g0 += 4) {
    const int heads = min(4, hg.count - g0);
    float mx[4], l[4], o[4][V];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      mx[e] = -INFINITY;
      l[e] = 0.f;
#pragma unroll
      for (int x = 0; x < V; ++x) o[e][x] = 0.f;
    }
    for (int c = it.c0 + lane; c <= it.c1; c += 32)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < heads) mx[e] = fmaxf(mx[e], __ldcg(&p.part_ml[(size_t)it.slot_of(c) * kDecodeHeads + g0 + e]).x);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xFFFFFFFFu, mx[e], x));
      if (mx[e] == -INFINITY) mx[e] = 0.f;
    }
#pragma unroll 2
    for (int c = it.c0 + warp; c <= it.c1; c += 4) {
      const size_t at = (size_t)it.slot_of(c) * kDecodeHeads + g0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (e >= heads) continue;
        const float2 ml = __ldcg(&p.part_ml[at + e]);
        const float* po = p.part_o + (at + e) * D + lane * V;
        float v[V];
        if constexpr (V == 4) {
          const float4 f = __ldcg(reinterpret_cast<const float4*>(po));
          v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
        } else {
          const float2 f = __ldcg(reinterpret_cast<const float2*>(po));
          v[0] = f.x; v[1] = f.y;
        }
        const float w = __expf(ml.x - mx[e]);
        l[e] = fmaf(ml.y, w, l[e]);
#pragma unroll
        for (int x = 0; x < V; ++x) o[e][x] = fmaf(v[x], w, o[e][x]);
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int x = 0; x < V; ++x) buf[(warp * 4 + e) * D + lane * V + x] = o[e][x];
      if (lane == 0) lbuf[warp * 4 + e] = l[e];
    }
    named_bar_sync(bar, 128);
    for (int i = tid; i < heads * D; i += 128) {
      const int e = i / D, d = i % D;
      const float sum = (lbuf[e] + lbuf[4 + e]) + (lbuf[8 + e] + lbuf[12 + e]);
      const float x = (buf[e * D + d] + buf[(4 + e) * D + d]) + (buf[(8 + e) * D + d] + buf[(12 + e) * D + d]);
      const size_t row = (size_t)b * p.Hq + hg.h0 + g0 + e;
      static_cast<T*>(p.o)[row * D + d] = (T)(sum == 0.f ? 0.f : x / sum);
      if (d == 0) p.lse[row] = sum == 0.f ? -INFINITY : (e == 0 ? mx[0] : e == 1 ? mx[1] : e == 2 ? mx[2] : mx[3]) + logf(sum);
    }
    named_bar_sync(bar, 128);
  }
}

}  // namespace capattn
