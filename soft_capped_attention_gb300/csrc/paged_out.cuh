// Results of a query tile's rows: whole ones, partial ones and their join.
//
// m is the reference of a row's exponentials in log2 units, l the sum of 2^(x - m), O the
// unnormalised output.  A row whose result cannot be trusted (see row_bad) gets NaN for
// its lse and raises the redo flag: paged_redo_kernel then forms it once more.
#pragma once

#include "cap_math.cuh"
#include "paged_sched.cuh"

namespace capattn {

constexpr float kNaN32 = __builtin_nanf("");

__device__ __forceinline__ void ask_redo(const PagedParams& p) {
  *reinterpret_cast<volatile uint32_t*>(p.redo) = 1u;  // (every writer writes the same)
}

// N consecutive values of a row of o.
template <typename T, int N>
__device__ __forceinline__ void store_values(T* dst, const float (&y)[N]) {
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int e = 0; e < N; e += 8)
      *reinterpret_cast<uint4*>(dst + e) = make_uint4(pack_bf16x2(y[e], y[e + 1]), pack_bf16x2(y[e + 2], y[e + 3]),
                                                      pack_bf16x2(y[e + 4], y[e + 5]), pack_bf16x2(y[e + 6], y[e + 7]));
  } else {
#pragma unroll
    for (int e = 0; e < N; e += 4) *reinterpret_cast<float4*>(dst + e) = make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]);
  }
}

// Counts a piece in (one thread, after every thread that wrote partial results has met it):
// whether it is the last one of its tile.
__device__ __forceinline__ bool count_tile_piece(const PagedParams& p, const Piece& x) {
  uint32_t before;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(p.c.counters + x.c0) : "memory");
  const bool last = before == (uint32_t)(x.c1 - x.c0);
  if (last) p.c.counters[x.c0] = 0u;
  return last;
}

// Adds the pieces of row r of a tile up, D / 4 columns from cq D / 4 on, in the order of
// their CTAs, and writes them (and, cq == 0, the row's lse).
template <typename T, int D, int ROWS>
__device__ __forceinline__ void join_row(const PagedParams& p, const Piece& x, int r, int cq, size_t out_row) {
  constexpr int N = D / 4;
  float m = -INFINITY, l = 0.f, o[N];
  bool bad = false;
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] = 0.f;
#pragma unroll 1
  for (int c = x.c0; c <= x.c1; ++c) {
    const size_t at = (size_t)piece_slot(x, c) * ROWS + r;
    const float2 ml = __ldcg(p.part_ml + at);
    const float4* src = reinterpret_cast<const float4*>(p.part_o + at * D + cq * N);
    float4 v[N / 4];
#pragma unroll
    for (int e = 0; e < N / 4; ++e) v[e] = __ldcg(src + e);
    if (ml.y == 0.f) continue;  // no live slot there
    bad = bad || __ldcg(reinterpret_cast<const uint32_t*>(p.part_bad) + at) != 0u;
    const float top = fmaxf(m, ml.x);
    const float a = ex2_approx(m - top), f = ex2_approx(ml.x - top);  // (m = -inf: a = 0)
    m = top;
    l = fmaf(ml.y, f, l * a);
#pragma unroll
    for (int e = 0; e < N / 4; ++e) {
      o[4 * e] = fmaf(v[e].x, f, o[4 * e] * a);
      o[4 * e + 1] = fmaf(v[e].y, f, o[4 * e + 1] * a);
      o[4 * e + 2] = fmaf(v[e].z, f, o[4 * e + 2] * a);
      o[4 * e + 3] = fmaf(v[e].w, f, o[4 * e + 3] * a);
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int e = 0; e < N; ++e) o[e] *= inv;
  store_values(static_cast<T*>(p.c.o) + out_row * D + cq * N, o);
  if (cq == 0) {
    bad = bad || !(l < INFINITY);
    if (bad) ask_redo(p);
    p.c.lse[out_row] = bad ? kNaN32 : l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
  }
}

}  // namespace capattn
