// Results of a query tile's rows: whole ones and partial ones.
//
// m is the reference of a row's exponentials in log2 units, l the sum of 2^(x - m), O the
// unnormalised output.  A tile that several CTAs share leaves (m, l, O) of each piece in the
// workspace, and its first CTA a record of it; paged_finish_kernel adds them up.  A row whose
// result cannot be trusted gets NaN for its lse and raises the redo flag: that kernel then
// forms it once more.
//
// O of a piece lies in blocks of 32 rows x D / 4 columns, four columns of the 32 rows after
// the other four, so that a warp whose lanes are rows writes and reads whole lines (row by
// row each of its instructions met 32 lines: a tile of 128 rows shared by 19 CTAs took
// 110 us to join).
#pragma once

#include "cap_math.cuh"
#include "paged_sched.cuh"

namespace capattn {

constexpr float kNaN32 = __builtin_nanf("");

// Place (in float4) of columns [4 e, 4 e + 4) of quarter cq of row r of a slot.
template <int D, int ROWS>
__device__ __forceinline__ size_t part_at(int slot, int r, int cq, int e) {
  return ((((size_t)slot * (ROWS / 32) + (r >> 5)) * 4 + cq) * (D / 16) + e) * 32 + (r & 31);
}

__device__ __forceinline__ void ask_redo(const PagedParams& p) {
  *reinterpret_cast<volatile uint32_t*>(p.redo) = 1u;  // (every writer writes the same)
}

// Which shared tile begins in this CTA, if any (x) or none.
__device__ __forceinline__ void leave_record(const PagedParams& p, const Piece& x) { p.records[blockIdx.x] = x; }
__device__ __forceinline__ void leave_no_record(const PagedParams& p) { p.records[blockIdx.x].steps = -1; }

}  // namespace capattn
