// The tables and slot maps of a step from request lengths, in one launch.
//
// Every CTA goes over all sequences by itself and sums up what they add, give back and need:
// new tokens, pages, pages.  Everything else is a function of those sums: the k-th page that
// goes out is the k-th from the top of the stack with this step's returns on it, which is an
// old entry or, found by the sums again, a page that comes back in this very step; so no CTA
// waits for another, and the result does not depend on scheduling.  The CTAs share out
// returning pages, outgoing pages and new rows, each finding its sequence by binary search.
// Lengths, held pages and the stack's height may be updated in place: the CTA that ends last
// writes them.  Bound by latency: a launch, the lengths, two scans, the searches in shared
// memory, the pages, the stores.  64 sequences of one new token: 4.8 us; 512 sequences and
// 66,000 rows: 7.5 (four rows a thread in flight at once 10.8, a cluster of eight CTAs that
// met twice 14.8); 400,000 rows: 10.9; 6000 sequences: 17.6 (81 with their sums in memory,
// where those of more than 8192 have to be).  256 threads instead of 512: 4.4, 7.4, but 144.
#include "paged_internal.h"
#include "tc_common.cuh"

namespace capattn {
namespace {

constexpr int kThreads = 512;
constexpr int kCtas = 152;
constexpr int kSmemSeqs = 8192;    // sequences whose sums fit shared memory
constexpr int kFewCtas = kPlanCopies;  // CTAs for more than those: their sums lie in the workspace

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
  // a sequence owns the pages of all its tokens: others would be taken for missing and replaced
  s.bad = s.bad || s.held < (int)(((int64_t)len + p.page_size - 1) >> p.page_shift);
  s.len = s.bad ? 0 : (int)after;
  s.need = (s.len + p.page_size - 1) >> p.page_shift;
  return s;
}

__device__ __forceinline__ int64_t scan64(int64_t x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// What comes before a sequence (rows, pages back, pages out), the pages that it held, its
// length behind the step and the pages of that.
struct Entry {
  int32_t rows, back, out, held, len, need;
};

// The entry that holds item x: the last one with at most x before it.
template <int PART>
__device__ __forceinline__ int find(const Entry* e, int B, int x) {
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    const int v = PART == 0 ? e[mid].rows : PART == 1 ? e[mid].back : e[mid].out;
    if (v <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads)
plan_kernel(PlanParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int64_t s_sum[3][kThreads / 32];
  __shared__ int s_bad, s_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Entry* e = p.B <= kSmemSeqs ? reinterpret_cast<Entry*>(smem) : reinterpret_cast<Entry*>(p.seqs) + (size_t)blockIdx.x * p.B;
  if (tid == 0) s_bad = 0;
  pdl_trigger();
  pdl_wait();
  __syncthreads();
  const int per = (p.B + kThreads - 1) / kThreads, b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  const int64_t n_free = p.n_free[0];
  int64_t add = 0, back = 0, out = 0;
  Seq only{};
  for (int b = b0; b < b1; ++b) {
    const Seq s = only = read_seq(p, b);
    if (s.bad) s_bad = 1;
    add += s.add;
    back += max(0, s.held - s.need);
    out += max(0, s.need - s.held);
  }
  int64_t sums[3] = {scan64(add, lane), scan64(back, lane), scan64(out, lane)}, all[3];
  if (lane == 31) {
#pragma unroll
    for (int x = 0; x < 3; ++x) s_sum[x][warp] = sums[x];
  }
  __syncthreads();
#pragma unroll
  for (int x = 0; x < 3; ++x) {
    const int64_t w = scan64(lane < kThreads / 32 ? s_sum[x][lane] : 0, lane);
    all[x] = __shfl_sync(0xFFFFFFFFu, w, 31);
    const int64_t before = __shfl_sync(0xFFFFFFFFu, w, max(0, warp - 1));
    if (warp > 0) sums[x] += before;
  }
  const bool ok = !s_bad && all[0] <= p.n_rows && n_free >= 0 && n_free + all[1] <= p.num_pages && all[2] <= n_free + all[1];
  const int threads = gridDim.x * kThreads, me = blockIdx.x * kThreads + tid;
  if (!ok) {
    // nothing changes: outputs of their own get what the inputs are
    if (me == 0) atomicOr(p.status, kStatusBadPlanBit);
    for (int b = me; b < p.B; b += threads) {
      if (p.lens_out != p.lens) p.lens_out[b] = p.lens[b];
      if (p.held_out != p.held) p.held_out[b] = p.held[b];
      if (p.qpos && p.qpos_out != p.qpos) p.qpos_out[b] = p.qpos[b];
    }
    for (int64_t b = me; b <= p.B; b += threads) p.cu_new[b] = 0;
    if (me == 0 && p.n_free_out != p.n_free) p.n_free_out[0] = (int)n_free;
    for (int64_t r = me; r < p.n_rows; r += threads) {
      if (p.slots) p.slots[r] = -1;
      if (p.positions) p.positions[r] = -1;
    }
    return;
  }
  int64_t at[3] = {sums[0] - add, sums[1] - back, sums[2] - out};
  for (int b = b0; b < b1; ++b) {
    const Seq s = per == 1 ? only : read_seq(p, b);
    e[b] = Entry{(int)at[0], (int)at[1], (int)at[2], s.held, s.len, s.need};
    at[0] += s.add;
    at[1] += max(0, s.held - s.need);
    at[2] += max(0, s.need - s.held);
  }
  __syncthreads();
  const int rows = (int)all[0], backs = (int)all[1], outs = (int)all[2], old = (int)n_free, top = old + backs;
  // The k-th page that comes back, the k-th that goes out.
  auto returned = [&](int k) -> int {
    const int b = find<1>(e, p.B, k);
    return p.table[(size_t)b * p.max_pages + e[b].need + (k - e[b].back)];
  };
  auto taken = [&](int k) -> int {
    const int i = top - 1 - k;
    return i >= old ? returned(i - old) : p.free_pages[i];
  };
  for (int64_t k = me; k < backs; k += threads) p.free_pages[old + k] = returned((int)k);
  for (int64_t k = me; k < outs; k += threads) {
    const int b = find<2>(e, p.B, (int)k);
    p.table[(size_t)b * p.max_pages + e[b].held + ((int)k - e[b].out)] = taken((int)k);
  }
  for (int64_t r = me; r < p.n_rows; r += threads) {
    int64_t place = -1;
    int pos = -1;
    if (r < rows) {
      const int b = find<0>(e, p.B, (int)r);
      const int left = (b + 1 < p.B ? e[b + 1].rows : rows) - (int)r;  // this row and those behind it
      const int slot = e[b].len - left, x = slot >> p.page_shift;
      const int page = x < e[b].held ? p.table[(size_t)b * p.max_pages + x] : taken(e[b].out + x - e[b].held);
      place = ((int64_t)page << p.page_shift) + (slot & (p.page_size - 1));
      pos = p.qpos ? p.qpos[b] + 1 + ((int)r - e[b].rows) : slot;
    }
    if (p.slots) p.slots[r] = place;
    if (p.positions) p.positions[r] = pos;
  }
  // What may replace its own input: by the CTA that ends last
  __syncthreads();
  if (tid == 0) {
    s_last = 1;
    if (gridDim.x > 1) {
      __threadfence();
      s_last = atomicAdd(p.ticket, 1u) == gridDim.x - 1;
      __threadfence();
    }
  }
  __syncthreads();
  if (!s_last) return;
  for (int b = tid; b < p.B; b += kThreads) {
    const int n = p.n_new[b], q = p.qpos ? p.qpos[b] : 0;
    p.cu_new[b] = e[b].rows;
    p.lens_out[b] = e[b].len;
    p.held_out[b] = e[b].need;
    if (p.qpos) p.qpos_out[b] = n < 0 ? -1 : q + n;
  }
  if (tid == 0) {
    p.cu_new[p.B] = rows;
    p.n_free_out[0] = top - outs;
    if (gridDim.x > 1) *p.ticket = 0u;
  }
}

}  // namespace

cudaError_t launch_paged_plan(const PlanParams& p, cudaStream_t s) {
  const bool small = p.B <= kSmemSeqs;
  const int bytes = small ? p.B * (int)sizeof(Entry) : 0;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(plan_kernel), kSmemSeqs * (int)sizeof(Entry), done);
  if (e != cudaSuccess) return e;
  // a row a thread where there are CTAs for it; one CTA needs no ticket
  const int64_t want = ((int64_t)p.n_rows + kThreads - 1) / kThreads;
  const int64_t most = small ? kCtas : kFewCtas;
  const int ctas = (int)(want < 1 ? 1 : want < most ? want : most);
  return launch_pdl(plan_kernel, dim3(ctas), dim3(kThreads), bytes, s, p);
}

}  // namespace capattn
