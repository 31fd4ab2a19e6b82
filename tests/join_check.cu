// Runs the joins of a split decode (csrc/cache_sched.cuh) on given partial results:
// group g has `pieces` pieces in the slots of CTAs g * pieces .. (g + 1) * pieces - 1,
// every second group starting inside its first CTA's range.
#include "../soft_capped_attention_gb300/csrc/cache_sched.cuh"

#include <string.h>

namespace capattn {
namespace {

__device__ __forceinline__ Pieces pieces_of(int g, int pieces) {
  return Pieces(g * pieces, (g + 1) * pieces - 1, g & 1);
}

// One warp a piece: leaves it, counts it in, and joins the group when it is the last.
template <int D>
__global__ void __launch_bounds__(32) leave_kernel(CacheParams p, const float2* ml, const float* o, int pieces) {
  const int g = blockIdx.x / pieces, lane = threadIdx.x;
  const Pieces pc = pieces_of(g, pieces);
  const int slot = pc.slot_of(blockIdx.x);
  for (int h = 0; h < p.Hq; ++h) {
    const size_t at = (size_t)slot * kDecodeHeads + h;
    for (int x = 0; x < D / 32; ++x) p.part_o[at * D + lane * (D / 32) + x] = o[at * D + lane * (D / 32) + x];
    if (lane == 0) p.part_ml[at] = ml[at];
  }
  const HeadGroup hg = {0, p.Hq, 0};
  if (count_piece_warp(p, pc, lane)) join_pieces<float, D, 1>(p, pc, g, hg, 0, lane, 0, nullptr, nullptr);
}

// One CTA a group, over partial results that are there.
template <int D, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) join_kernel(CacheParams p, int pieces) {
  __shared__ __align__(16) float buf[16 * D];
  __shared__ float sbuf[32];
  const int g = blockIdx.x;
  const HeadGroup hg = {0, p.Hq, 0};
  join_pieces<float, D, WARPS>(p, pieces_of(g, pieces), g, hg, threadIdx.x >> 5, threadIdx.x & 31, 1, buf, sbuf);
}

template <int D>
cudaError_t run(const CacheParams& p, const float2* ml, const float* o, int groups, int pieces, int form, cudaStream_t s) {
  if (form == 0) leave_kernel<D><<<groups * pieces, 32, 0, s>>>(p, ml, o, pieces);
  else if (form == 1) join_kernel<D, 1><<<groups, 32, 0, s>>>(p, pieces);
  else join_kernel<D, 4><<<groups, 128, 0, s>>>(p, pieces);
  return cudaGetLastError();
}

}  // namespace
}  // namespace capattn

// ml [2 * 608][16] float2, o_parts [2 * 608][16][D]: the partial results by slot; part_ml
// and part_o as large, counters [608] zero.  form 0: they are left by a warp a piece and
// joined by the last; 1 and 4: part_ml and part_o joined by one warp, by four.
extern "C" int join_check(int D, int groups, int pieces, int heads, const void* ml, const float* o_parts, void* part_ml,
                          float* part_o, unsigned* counters, float* o, float* lse, int form, void* stream) {
  using namespace capattn;
  if ((D != 64 && D != 128) || groups < 1 || pieces < 1 || groups * pieces > kDecodeMaxCtas || heads < 1 ||
      heads > kDecodeHeads)
    return -1;
  CacheParams p;
  memset(&p, 0, sizeof(p));
  p.Hq = heads;
  p.part_ml = static_cast<float2*>(part_ml);
  p.part_o = part_o;
  p.counters = counters;
  p.o = o;
  p.lse = lse;
  const float2* m = static_cast<const float2*>(ml);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return (int)(D == 64 ? run<64>(p, m, o_parts, groups, pieces, form, s) : run<128>(p, m, o_parts, groups, pieces, form, s));
}
