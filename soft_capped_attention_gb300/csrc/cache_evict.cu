// Eviction from the paged cache by accumulated weight.
//
// Per (sequence, KV head) with n > budget tokens: rank every slot by a 32-bit
// key (protected slots highest, then the weight's order, NaN lowest), find the
// budget-th largest key by radix selection, and keep the slots above it plus the
// lowest slots equal to it.  Slots that are kept and lie below the budget do not
// move; the i-th kept slot behind the budget goes to the i-th freed slot below
// it.  Their number is the least that any compaction has to copy, and a copy
// never reads what another writes (sources lie behind the budget, destinations
// below it), so all of them run at once.
//
// Selection is bound by latency (its 8 bytes a slot are little against the rows
// that move): a cluster of up to 8 CTAs takes a row, each CTA a run of slots whose
// keys it reads once and keeps in shared memory.  Three histogram passes (11, 11
// and 10 bits) find the threshold, each CTA adding up the cluster's histograms by
// distributed shared memory (four copies of a CTA's first one, since weights share
// few leading digits and equal bins serialise the atomics); three more passes over
// the keys count and list the slots.  What follows from the lists (the rows' pages,
// the copies, the moved tokens' weights and positions) is the second kernel's, over
// all SMs.
#include <cooperative_groups.h>

#include "cache_internal.h"

namespace capattn {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxParts = 8;
constexpr int kBins = 2048;
constexpr int kCachedKeys = 40 * 1024;  // keys a CTA keeps in shared memory (160 KB)

// Order of a weight as an unsigned key: larger weight, larger key; both zeros
// equal; NaN lowest.  Protected slots get 0xFFFFFFFF, above +inf's 0xFF800000.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 becomes +0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

struct RowKeys {
  const float* w;
  const int32_t* pos;
  int first, after;  // protected: position < first or > after
  __device__ __forceinline__ uint32_t of(float weight, int x) const {
    return x < first || x > after ? 0xFFFFFFFFu : weight_key(weight);
  }
  __device__ __forceinline__ uint32_t at(int j) const { return of(w[j], pos ? pos[j] : j); }
};

constexpr int kBatch = 8;   // slots a thread reads at once
constexpr int kCopies = 4;  // of the first digit's histogram
struct Shared {
  __align__(8) int hist[kCopies + 2][kBins];  // pass 0 (copies), 1, 2
  int warp_sum[3][kSelWarps];
  int totals[3];              // of this CTA: equal keys, movers, freed slots
  uint32_t digit;
  int above;
};

// Exclusive sum of x over the block's threads; *total the whole (buf: a word a warp).
__device__ __forceinline__ int block_scan(int x, int* buf, int warp, int lane, int* total) {
  int up = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, up, d);
    if (lane >= d) up += y;
  }
  if (lane == 31) buf[warp] = up;
  __syncthreads();
  const int w = buf[lane];  // 32 warps
  int all = w;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, all, d);
    if (lane >= d) all += y;
  }
  *total = __shfl_sync(0xFFFFFFFFu, all, 31);
  return up - x + __shfl_sync(0xFFFFFFFFu, all - w, warp);
}

__device__ __forceinline__ int cache_row(const CacheParams& p, int b, int g, int slot) {
  const int page = p.table[(size_t)b * p.max_pages + (slot >> p.page_shift)];
  if (page < 0 || page >= p.num_pages) {
    atomicOr(p.status, kStatusBadPageBit);
    return -1;
  }
  return ((page * p.Hkv + g) << p.page_shift) + (slot & (p.page_size - 1));
}

__global__ void __launch_bounds__(kSelThreads, 1)
select_kernel(CacheParams p, int parts) {
  extern __shared__ uint32_t s_keys[];
  __shared__ Shared s;
  cg::cluster_group cluster = cg::this_cluster();
  auto meet = [&] {
    if (parts > 1) cluster.sync(); else __syncthreads();
  };
  const int rank = blockIdx.x % parts, row = blockIdx.x / parts;
  const int b = row / p.Hkv, g = row % p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < (kCopies + 2) * kBins; i += kSelThreads) (&s.hist[0][0])[i] = 0;
  pdl_trigger();
  pdl_wait();
  int n = p.lens[b];
  if (n < 0 || n > p.max_len) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusBadLensBit);
    n = n < 0 ? 0 : p.max_len;
  }
  const size_t base = (size_t)row * p.max_len;
  RowKeys keys;
  keys.w = p.weights + base;
  keys.pos = p.pos ? p.pos + base : nullptr;
  const long long newest = p.pos ? p.qpos[b] : n - 1;
  keys.first = p.keep_first;
  keys.after = (int)max(newest - p.keep_last, -(1ll << 31));
  int32_t* src = p.src + (size_t)row * p.budget;
  int2* moves = reinterpret_cast<int2*>(p.moves + base);
  if (n <= p.budget) {  // nothing goes (every CTA of the cluster alike)
    for (int j = rank * kSelThreads + threadIdx.x; j < p.budget; j += parts * kSelThreads) {
      src[j] = j < n ? j : -1;
      if (j < n && p.weights_out != p.weights) p.weights_out[base + j] = keys.w[j];
      if (j < n && p.pos_out && p.pos_out != p.pos) p.pos_out[base + j] = keys.pos[j];
    }
    if (rank == 0 && threadIdx.x == 0) p.counts[row] = make_int2(0, n);
    return;
  }
  // this CTA's slots [c0, c1): equal runs of whole groups of 32, a run a warp
  const int run = (int)(((long long)n + (long long)parts * kSelThreads - 1) / ((long long)parts * kSelThreads)) * 32;
  const int c0 = (int)min((long long)n, (long long)rank * run * kSelWarps);
  const int c1 = (int)min((long long)n, (long long)c0 + (long long)run * kSelWarps);
  const bool cached = run * kSelWarps <= kCachedKeys;
  __syncthreads();  // the histograms are zero
  // First digit, with the keys on their way into shared memory.  Slots below the
  // budget are written as if they were kept; the moves overwrite those that go.
  const bool copy_w = p.weights_out != p.weights, copy_pos = p.pos_out && p.pos_out != p.pos;
  for (int j = c0 + threadIdx.x; j < c1; j += kBatch * kSelThreads) {
    float w[kBatch];
    int at[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int x = j + u * kSelThreads;
      w[u] = x < c1 ? keys.w[x] : 0.f;
      at[u] = x < c1 && keys.pos ? keys.pos[x] : x;
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int x = j + u * kSelThreads;
      if (x >= c1) break;
      const uint32_t k = keys.of(w[u], at[u]);
      if (cached) s_keys[x - c0] = k;
      atomicAdd(&s.hist[threadIdx.x % kCopies][k >> 21], 1);
      if (x < p.budget) {
        src[x] = x;
        if (copy_w) p.weights_out[base + x] = w[u];
        if (copy_pos) p.pos_out[base + x] = at[u];
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kBins; i += kSelThreads) {
    int sum = 0;
#pragma unroll
    for (int c = 0; c < kCopies; ++c) sum += s.hist[c][i];
    s.hist[0][i] = sum;
  }
  auto key = [&](int j) { return cached ? s_keys[j - c0] : keys.at(j); };
  // The budget-th largest key: its digits from the top; `left` is its rank among
  // the keys that share the digits so far.
  uint32_t prefix = 0;
  int left = p.budget;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    int* hist = s.hist[pass == 0 ? 0 : kCopies - 1 + pass];
    const int bins = pass == 2 ? 1024 : kBins;
    if (pass > 0) {
      const uint32_t mask = pass == 1 ? 0xFFFFFFFFu << 21 : 0xFFFFFFFFu << 10;
      for (int j = c0 + threadIdx.x; j < c1; j += kSelThreads) {
        const uint32_t k = key(j);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1);
      }
    }
    meet();  // the cluster's histograms of this pass are whole
    // a thread holds two bins, from the top
    int c[2] = {0, 0};
    const int top = bins - 1 - 2 * (int)threadIdx.x;
    if (top > 0) {
      int v[kMaxParts][2];  // all loads on their way before the first sum
#pragma unroll
      for (int x = 0; x < kMaxParts; ++x) {
        v[x][0] = v[x][1] = 0;
        if (x < parts) {
          const int2 h = *reinterpret_cast<const int2*>((parts > 1 ? cluster.map_shared_rank(hist, x) : hist) + top - 1);
          v[x][0] = h.y;
          v[x][1] = h.x;
        }
      }
#pragma unroll
      for (int x = 0; x < kMaxParts; ++x) {
        c[0] += v[x][0];
        c[1] += v[x][1];
      }
    }
    int total;
    const int above = block_scan(c[0] + c[1], s.warp_sum[pass], warp, lane, &total);
    if (above < left && left <= above + c[0]) {
      s.digit = (uint32_t)top;
      s.above = above;
    } else if (above + c[0] < left && left <= above + c[0] + c[1]) {
      s.digit = (uint32_t)(top - 1);
      s.above = above + c[0];
    }
    __syncthreads();
    prefix |= s.digit << shift;
    left -= s.above;
    __syncthreads();
  }
  // Places, in the order of the slots: warp by warp, CTA by CTA.
  const int j0 = min(c1, c0 + warp * run), j1 = min(c1, j0 + run);
  const uint32_t below = (1u << lane) - 1u;
  int equal = 0;
  for (int j = j0 + lane; j < j1; j += 32) equal += key(j) == prefix;
  equal = __reduce_add_sync(0xFFFFFFFFu, equal);
  // This warp's start in the cluster's order of one count a warp, after share()
  // has left it and the cluster has met; *total the cluster's.
  auto share = [&](int mine, int which) {
    if (lane == 0) s.warp_sum[which][warp] = mine;
    __syncthreads();
    const int x = s.warp_sum[which][lane];
    int up = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, up, d);
      if (lane >= d) up += y;
    }
    if (threadIdx.x == 31) s.totals[which] = up;
    return __shfl_sync(0xFFFFFFFFu, up - x, warp);
  };
  auto before = [&](int which, int* total) {
    int v = 0;  // a lane a CTA
    if (lane < parts) v = parts > 1 ? *cluster.map_shared_rank(&s.totals[which], lane) : s.totals[which];
    *total = __reduce_add_sync(0xFFFFFFFFu, v);
    return __reduce_add_sync(0xFFFFFFFFu, lane < rank ? v : 0);
  };
  int total;
  int eq0 = share(equal, 0);
  meet();
  eq0 += before(0, &total);
  // Kept: above the threshold, or among the first `left` equal ones.  All equal keys
  // of a warp are on one side of that, but for one warp of the cluster.
  const bool all_eq = eq0 + equal <= left, none_eq = eq0 >= left;
  auto kept_of = [&](int j, int& seen) {
    const uint32_t k = j < j1 ? key(j) : 0u;
    if (all_eq || none_eq) return j < j1 && (all_eq ? k >= prefix : k > prefix);
    const bool eq = j < j1 && k == prefix;
    const uint32_t eqs = __ballot_sync(0xFFFFFFFFu, eq);
    const bool kept = j < j1 && (k > prefix || (eq && seen + __popc(eqs & below) < left));
    seen += __popc(eqs);
    return kept;
  };
  int movers = 0, holes = 0, seen = eq0;
  for (int j = j0; j < j1; j += 32) {
    const int x = j + lane;
    const bool kept = kept_of(x, seen);
    movers += kept && x >= p.budget;
    holes += x < j1 && !kept && x < p.budget;
  }
  movers = __reduce_add_sync(0xFFFFFFFFu, movers);
  holes = __reduce_add_sync(0xFFFFFFFFu, holes);
  int n_moves, n_holes;
  int mover = share(movers, 1), hole = share(holes, 2);
  meet();
  mover += before(1, &n_moves);
  hole += before(2, &n_holes);
  seen = eq0;
  for (int j = j0; j < j1; j += 32) {
    const int x = j + lane;
    const bool kept = kept_of(x, seen);
    const bool moves_it = kept && x >= p.budget, freed = x < j1 && !kept && x < p.budget;
    const uint32_t who_moves = __ballot_sync(0xFFFFFFFFu, moves_it), who_goes = __ballot_sync(0xFFFFFFFFu, freed);
    if (moves_it) moves[mover + __popc(who_moves & below)].y = x;
    if (freed) moves[hole + __popc(who_goes & below)].x = x;
    mover += __popc(who_moves);
    hole += __popc(who_goes);
  }
  if (rank == 0 && threadIdx.x == 0) p.counts[row] = make_int2(n_moves, p.budget);
  if (parts > 1) cluster.sync();  // no CTA leaves while its counts may be read
}

// Carries out the moves: a group of vph threads a row, K and V together, two rows in
// flight a thread; the group's first thread takes the token's weight and position
// along.  (Moved tokens come from behind the budget and go below it, so none of
// this reads what another writes, in place too.)
constexpr int kMoveThreads = 256;
__global__ void __launch_bounds__(kMoveThreads)
move_kernel(CacheParams p, int vph_shift) {
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x, b = row / p.Hkv, g = row - b * p.Hkv;
  const int2 c = p.counts[row];
  if (g == 0 && blockIdx.y == 0 && threadIdx.x == 0) p.lens_out[b] = c.y;
  const size_t base = (size_t)row * p.max_len;
  const int2* moves = reinterpret_cast<const int2*>(p.moves + base);
  int32_t* src = p.src + (size_t)row * p.budget;
  const int per = kMoveThreads >> vph_shift;
  const int at = threadIdx.x & ((1 << vph_shift) - 1);
  uint4* k = static_cast<uint4*>(p.k);
  uint4* v = static_cast<uint4*>(p.v);
  const int stride = gridDim.y * per;
  for (int i = blockIdx.y * per + (threadIdx.x >> vph_shift); i < c.x; i += 2 * stride) {
    int2 m[2], r[2];
    uint4 a[2], d[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) m[u] = i + u * stride < c.x ? moves[i + u * stride] : make_int2(-1, -1);
#pragma unroll
    for (int u = 0; u < 2; ++u)
      r[u] = m[u].x >= 0 ? make_int2(cache_row(p, b, g, m[u].x), cache_row(p, b, g, m[u].y)) : make_int2(-1, -1);
#pragma unroll
    for (int u = 0; u < 2; ++u)
      if (r[u].x >= 0 && r[u].y >= 0) {
        a[u] = __ldcs(k + ((size_t)r[u].y << vph_shift) + at);
        d[u] = __ldcs(v + ((size_t)r[u].y << vph_shift) + at);
      }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (at == 0 && m[u].x >= 0) {
        src[m[u].x] = m[u].y;
        p.weights_out[base + m[u].x] = p.weights[base + m[u].y];
        if (p.pos_out) p.pos_out[base + m[u].x] = p.pos[base + m[u].y];
      }
      if (r[u].x >= 0 && r[u].y >= 0) {
        k[((size_t)r[u].x << vph_shift) + at] = a[u];
        v[((size_t)r[u].x << vph_shift) + at] = d[u];
      }
    }
  }
}

}  // namespace

cudaError_t launch_cache_evict(const CacheParams& p, int dtype, cudaStream_t s) {
  const int rows = p.B * p.Hkv;
  // CTAs of a row: while each still has 2048 slots and the rows leave SMs idle
  int parts = 1;
  while (parts < kMaxParts && p.max_len / parts > 2048 && rows * parts * 2 <= 152) parts *= 2;
  static std::atomic<uint64_t> done{0};
  const int keys = min((long long)kCachedKeys, ((long long)p.max_len + parts * kSelThreads - 1) / (parts * kSelThreads) * kSelThreads);
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(select_kernel), kCachedKeys * 4, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows * parts);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = keys * 4;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = parts;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, select_kernel, p, parts);
  if (e != cudaSuccess) return e;
  const int vph = p.D / (dtype == CAPATTN_BF16 ? 8 : 4);
  int shift = 0;
  while ((1 << shift) < vph) ++shift;
  const int per = kMoveThreads >> shift;
  const int most = min(p.budget, max(1, p.max_len - p.budget));  // rows that can move
  const int y = min(max(1, (152 * 8 + rows - 1) / rows), (most + 2 * per - 1) / (2 * per));
  return launch_pdl(move_kernel, dim3(rows, y), dim3(kMoveThreads), 0, s, p, shift);
}

}  // namespace capattn
