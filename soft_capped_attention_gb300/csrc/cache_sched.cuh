// How a decode's work is split over a persistent grid.
//
// The live slots of sequence b are cut into tiles of TK keys; a unit of work is
// one tile of one (sequence, group of query heads).  Units are numbered
// sequence by sequence, group by group, tile by tile, and CTA c takes units
// [c q, (c + 1) q): equal shares whatever the lengths.  A CTA's part of one
// (sequence, group) is a piece; a piece that is not the whole leaves (m, l, O) in
// the CTA's slot 2c (the piece at the start of its range) or 2c + 1 (the one at
// its end; pieces between the two are whole), and the join adds the pieces up in
// order.  Every role computes the split from lens by itself, so the lengths stay
// on the device.
#pragma once

#include "cache_internal.h"

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

// Tiles of all sequences (warp-collective).
template <int TK>
__device__ __forceinline__ int total_tiles(const CacheParams& p, int lane) {
  int n = 0;
  for (int b = lane; b < p.B; b += 32) n += seq_span<TK>(p, b).tiles;
  return __reduce_add_sync(0xFFFFFFFFu, n);
}

// A CTA's share in units.
__device__ __forceinline__ uint32_t share_of(const CacheParams& p, uint32_t units) {
  return max((uint32_t)p.min_tiles, (units + p.ctas - 1) / (uint32_t)p.ctas);
}

// The sequence that holds tile number `want` of all, and the tiles before it
// (warp-collective; want below the total).
template <int TK>
__device__ __forceinline__ void find_tile(const CacheParams& p, int lane, int want, int* b_out, int* before_out) {
  int before = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int b = b0 + lane;
    int n = b < p.B ? seq_span<TK>(p, b).tiles : 0;
    int up = n;  // inclusive sum over the lanes
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int x = __shfl_up_sync(0xFFFFFFFFu, up, d);
      if (lane >= d) up += x;
    }
    const uint32_t hit = __ballot_sync(0xFFFFFFFFu, want < before + up);
    if (hit) {
      const int l = __ffs(hit) - 1;
      *b_out = b0 + l;
      *before_out = before + __shfl_sync(0xFFFFFFFFu, up - n, l);
      return;
    }
    before += __shfl_sync(0xFFFFFFFFu, up, 31);
  }
  *b_out = p.B - 1;
  *before_out = before;
}

// Walks a CTA's pieces.
template <int TK>
struct PieceIter {
  uint32_t u, end, begin;  // next unit, the range
  int b, vh, t0;           // the next piece: sequence, group, first tile of the group
  SeqSpan sp;
  // of the piece that next() gave
  int n;                   // tiles
  bool whole;
  int slot;                // partial slot when not whole

  __device__ PieceIter(const CacheParams& p, int lane) {
    const int tiles = total_tiles<TK>(p, lane);
    const uint32_t units = (uint32_t)tiles * (uint32_t)p.VH;
    const uint32_t share = share_of(p, units);
    begin = u = min(units, share * blockIdx.x);
    end = min(units, u + share);
    b = vh = t0 = 0;
    if (u < end) {
      int before;
      find_tile<TK>(p, lane, (int)(u / (uint32_t)p.VH), &b, &before);
      // units of sequence b start at before * VH
      sp = seq_span<TK>(p, b);
      const uint32_t in = u - (uint32_t)before * (uint32_t)p.VH;
      vh = (int)(in / (uint32_t)sp.tiles);
      t0 = (int)(in % (uint32_t)sp.tiles);
    }
  }
  // Gives the piece (b, vh, tiles [tile, tile + n) of the sequence's span).
  __device__ bool next(const CacheParams& p, int* b_out, int* vh_out, int* tile_out, SeqSpan* sp_out) {
    if (u >= end) return false;
    const int left = sp.tiles - t0;
    n = (int)min((uint32_t)left, end - u);
    whole = t0 == 0 && n == sp.tiles;
    slot = 2 * (int)blockIdx.x + (u == begin ? 0 : 1);
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

}  // namespace capattn
