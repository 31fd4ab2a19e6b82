// The tables and slot maps of a step from request lengths, in one launch.
//
// Every CTA of one cluster (or a single CTA, for small steps) goes over all sequences and
// sums up what they add, give back and need: new tokens, pages, pages.  The cluster meets;
// if everything fits, pages that come back go on the stack, it meets again (a page may
// come back and go out in the same step), and missing pages and the new rows' slots are
// shared out over all threads by binary search in the sums.  Every place is a function of
// the sums alone, so the result does not depend on scheduling.  Bound by latency: the sums
// and the two meetings.
#include <cooperative_groups.h>

#include "paged_internal.h"
#include "tc_common.cuh"

namespace capattn {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kCluster = 8;
constexpr int kSmemSeqs = 4096;  // sequences whose sums fit shared memory

// Sums before a sequence and what it has: x rows, y pages back, z pages out; w pages held.
// After all sequences one more entry holds the totals.
struct Totals {
  int64_t rows, back, out;
};

__device__ __forceinline__ int64_t scan64(int64_t x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

struct Seq {
  int32_t add, len, held, need;
  bool bad;
};
__device__ __forceinline__ Seq read_seq(const PlanParams& p, int b) {
  Seq s;
  const int n = p.n_new[b], len = p.lens[b];
  s.held = p.held[b];
  s.add = max(n, 0);
  const int64_t after = n < 0 ? 0 : (int64_t)len + n;
  s.bad = s.held < 0 || s.held > p.max_pages || after > p.max_len || len < 0 || len > p.max_len;
  s.len = s.bad ? 0 : (int)after;
  s.need = (s.len + p.page_size - 1) >> p.page_shift;
  return s;
}

// The last b of B with sums[b].<part> <= x (the entry that holds item x).
template <int PART>
__device__ __forceinline__ int find(const int4* sums, int B, int x) {
  int lo = 0, hi = B;  // sum(lo) <= x < sum(hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    const int v = PART == 0 ? sums[mid].x : PART == 1 ? sums[mid].y : sums[mid].z;
    if (v <= x) lo = mid; else hi = mid;
  }
  return lo;
}

template <bool CLUSTER>
__global__ void __launch_bounds__(kThreads)
plan_kernel(PlanParams p) {
  extern __shared__ int4 smem_sums[];
  __shared__ int64_t s_sum[3][32];
  __shared__ int s_bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = CLUSTER ? (int)blockIdx.x : 0, ctas = CLUSTER ? kCluster : 1;
  int4* sums = p.B <= kSmemSeqs ? smem_sums : p.seqs + (size_t)rank * p.B;
  auto meet = [&]() {
    if constexpr (CLUSTER) cg::this_cluster().sync(); else __syncthreads();
  };
  if (tid == 0) s_bad = 0;
  pdl_trigger();
  pdl_wait();
  __syncthreads();
  const int per = (p.B + kThreads - 1) / kThreads, b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  int64_t add = 0, back = 0, out = 0;
  for (int b = b0; b < b1; ++b) {
    const Seq s = read_seq(p, b);
    if (s.bad) s_bad = 1;
    add += s.add;
    back += max(0, s.held - s.need);
    out += max(0, s.need - s.held);
  }
  const int64_t ia = scan64(add, lane), ib = scan64(back, lane), io = scan64(out, lane);
  if (lane == 31) {
    s_sum[0][warp] = ia;
    s_sum[1][warp] = ib;
    s_sum[2][warp] = io;
  }
  const int64_t n_free = p.n_free[0];
  __syncthreads();
  Totals before{ia - add, ib - back, io - out}, all{0, 0, 0};
  {
    const int64_t a = scan64(s_sum[0][lane], lane), b = scan64(s_sum[1][lane], lane), o = scan64(s_sum[2][lane], lane);
    all.rows = __shfl_sync(0xFFFFFFFFu, a, 31);
    all.back = __shfl_sync(0xFFFFFFFFu, b, 31);
    all.out = __shfl_sync(0xFFFFFFFFu, o, 31);
    const int up = max(0, warp - 1);
    const int64_t wa = __shfl_sync(0xFFFFFFFFu, a, up), wb = __shfl_sync(0xFFFFFFFFu, b, up), wo = __shfl_sync(0xFFFFFFFFu, o, up);
    if (warp > 0) {
      before.rows += wa;
      before.back += wb;
      before.out += wo;
    }
  }
  const bool ok = !s_bad && all.rows <= p.n_rows && n_free >= 0 && n_free + all.back <= p.num_pages &&
                  all.out <= n_free + all.back;
  if (!ok && rank == 0 && tid == 0) atomicOr(p.status, kStatusBadPlanBit);
  // the sums, and what belongs to the sequences (rank 0's threads keep it over the meeting:
  // the outputs may be the inputs)
  for (int b = b0; b < b1; ++b) {
    const Seq s = read_seq(p, b);
    if (ok) sums[b] = make_int4((int)before.rows, (int)before.back, (int)before.out, s.held);
    before.rows += s.add;
    before.back += max(0, s.held - s.need);
    before.out += max(0, s.need - s.held);
  }
  __syncthreads();
  const int threads = ctas * kThreads, me = rank * kThreads + tid;
  if (!ok) {
    // nothing changes; other CTAs may still read what the outputs overwrite with itself
    for (int b = me; b < p.B; b += threads) {
      if (p.lens_out != p.lens) p.lens_out[b] = p.lens[b];
      if (p.held_out != p.held) p.held_out[b] = p.held[b];
      if (p.qpos && p.qpos_out != p.qpos) p.qpos_out[b] = p.qpos[b];
    }
    for (int b = me; b <= p.B; b += threads) p.cu_new[b] = 0;
    if (me == 0 && p.n_free_out != p.n_free) p.n_free_out[0] = (int)n_free;
    for (int r = me; r < p.n_rows; r += threads) {
      if (p.slots) p.slots[r] = -1;
      if (p.positions) p.positions[r] = -1;
    }
    return;
  }
  // pages that come back
  const int rows = (int)all.rows, backs = (int)all.back, outs = (int)all.out;
  for (int k = me; k < backs; k += threads) {
    const int b = find<1>(sums, p.B, k);
    const Seq s = read_seq(p, b);
    p.free_pages[n_free + k] = p.table[(size_t)b * p.max_pages + s.need + (k - sums[b].y)];
  }
  // what the rows need of a sequence is read before the outputs may overwrite it
  meet();
  const int top = (int)n_free + backs;
  for (int k = me; k < outs; k += threads) {
    const int b = find<2>(sums, p.B, k);
    p.table[(size_t)b * p.max_pages + sums[b].w + (k - sums[b].z)] = p.free_pages[top - 1 - k];
  }
  for (int r = me; r < p.n_rows; r += threads) {
    int64_t at = -1;
    int pos = -1;
    if (r < rows) {
      const int b = find<0>(sums, p.B, r);
      const int4 x = sums[b];
      const int i = r - x.x;
      const int slot = p.lens[b] + i, page = slot >> p.page_shift;
      const int id = page < x.w ? p.table[(size_t)b * p.max_pages + page] : p.free_pages[top - 1 - (x.z + page - x.w)];
      at = ((int64_t)id << p.page_shift) + (slot & (p.page_size - 1));
      pos = p.qpos ? p.qpos[b] + 1 + i : slot;
    }
    if (p.slots) p.slots[r] = at;
    if (p.positions) p.positions[r] = pos;
  }
  meet();  // lens, held and qpos have been read by all
  for (int b = me; b < p.B; b += threads) {
    const Seq s = read_seq(p, b);
    const int n = p.n_new[b], q = p.qpos ? p.qpos[b] : 0;
    p.cu_new[b] = sums[b].x;
    p.lens_out[b] = s.len;
    p.held_out[b] = s.need;
    if (p.qpos) p.qpos_out[b] = n < 0 ? -1 : q + n;
  }
  if (me == 0) {
    p.cu_new[p.B] = rows;
    p.n_free_out[0] = top - outs;
  }
}

}  // namespace

cudaError_t launch_paged_plan(const PlanParams& p, cudaStream_t s) {
  const int seqs = p.B <= kSmemSeqs ? p.B : 0;
  const int bytes = seqs * (int)sizeof(int4);
  // A step whose rows a CTA's threads write in a few turns needs no cluster.
  const bool cluster = (int64_t)p.n_rows + p.B > 4 * kThreads;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster ? kCluster : 1);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  auto* k = cluster ? plan_kernel<true> : plan_kernel<false>;
  static std::atomic<uint64_t> done[2];
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), kSmemSeqs * (int)sizeof(int4), done[cluster ? 1 : 0]);
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, k, p);
}

}  // namespace capattn
