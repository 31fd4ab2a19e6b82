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
// keys it reads once and keeps in shared memory.  Four histogram passes of 8 bits
// find the threshold, each CTA adding up the cluster's histograms by distributed
// shared memory (of 11 bits, three passes: reading 8 KB from each of 8 CTAs took 7000
// cycles a pass, more than a pass of 8 bits altogether).  The third pass lists the few
// keys that share two digits, which is all the fourth has to look at, and counts the
// keys above them, so that one exchange of counts gives every warp its places; the
// last pass over the keys lists the slots.  What follows from the lists (the rows' pages,
// the copies, the moved tokens' weights and positions) is the second kernel's, over
// all SMs.
//   Measured: 8 rows of 130,977 tokens cut to 16,384 take 43 us (about 21 of them
// selection, 22 the 117 MB of rows that move), 128 rows of 2049 to 4096 cut to 2048
// take 28.5 us; 38.4 and 24.6 when the last call has left part of them in L2, as in what
// follows.  With the slots shared out in one run a CTA instead of two, the CTA
// below the budget had all the freed ones to list (and 44.6 us, with three exchanges
// of counts).  Clusters of 16 CTAs took 59 us against 46 (a GPC places few of them at
// once), one CTA a row 640 us.  1024 threads a CTA, copies of the first histogram and
// twice the loads in flight changed nothing.
#include <cooperative_groups.h>

#include "cache_internal.h"

namespace capattn {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxParts = 8;
constexpr int kBins = 256;
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
};

constexpr int kBatch = 4;       // vectors of four slots a thread reads at once
// The keys that share two digits are few as a rule: of a CTA's this many are listed.
constexpr int kListed = 2048;
constexpr int kFew = 256;       // so few are ranked against one another instead
// Slots of a warp or CTA with keys above and equal to the threshold, of those below
// the budget (lo) and behind it (hi).
struct Counts {
  int over_lo, equal_lo, over_hi, equal_hi;
};
struct Shared {
  __align__(16) int hist[4][kBins];  // of each pass
  __align__(16) int sum[2][kBins];   // the cluster's (two, for passes in turn)
  __align__(16) int warp_counts[kSelWarps][4];  // Counts
  __align__(16) uint32_t list[kListed];         // keys
  uint8_t list_of[kListed];   // and whose: 2 warp + (1: behind the budget)
  int listed;
  int4 counts;                // Counts of this CTA
  uint32_t threshold;
  int left;
};

// Inclusive sum over the lanes.
__device__ __forceinline__ int inclusive_sum(int x, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, d);
    if (lane >= d) x += y;
  }
  return x;
}

__device__ __forceinline__ int cache_row(const CacheParams& p, int b, int g, int slot) {
  const int page = p.table[(size_t)b * p.max_pages + (slot >> p.page_shift)];
  if (page < 0 || page >= p.num_pages) {
    atomicOr(p.status, kStatusBadPageBit);
    return -1;
  }
  return ((page * p.Hkv + g) << p.page_shift) + (slot & (p.page_size - 1));
}

// CACHED: a CTA's keys fit its shared memory (else they are computed anew in every
// pass).
template <bool CACHED>
__global__ void __launch_bounds__(kSelThreads, 1)
select_kernel(CacheParams p, int parts) {
  extern __shared__ __align__(16) uint32_t s_keys[];
  __shared__ Shared s;
  cg::cluster_group cluster = cg::this_cluster();
  auto meet = [&] {
    if (parts > 1) cluster.sync(); else __syncthreads();
  };
  const int rank = blockIdx.x % parts, row = blockIdx.x / parts;
  const int b = row / p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = threadIdx.x; i < 4 * kBins; i += kSelThreads) (&s.hist[0][0])[i] = 0;
  if (threadIdx.x == 0) s.listed = 0;
  pdl_trigger();
  pdl_wait();
  int n = p.lens[b];
  if (n < 0 || n > p.max_len) {
    if (threadIdx.x == 0) atomicOr(p.status, kStatusBadLensBit);
    n = n < 0 ? 0 : p.budget;  // nothing moves: the table behind the tokens may name anyone's pages
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
  // The slots below the budget (whole vectors of four) and those behind it are shared out
  // apart, so that no CTA has all that go or all that come: a run of each a warp, in
  // order, in steps of four consecutive slots a lane (rows of the weights are whole
  // 16-byte units).
  const int edge = p.budget & ~3;  // the vector at the edge of both is in both, each with its slots
  const int all_warps = parts * kSelWarps, at_warp = rank * kSelWarps + warp;  // (n is at most 2^30)
  const int run_lo = (p.budget + 128 * all_warps - 1) / (128 * all_warps) * 128;
  const int run_hi = (n - edge + 128 * all_warps - 1) / (128 * all_warps) * 128;
  const int lo0 = min(p.budget, at_warp * run_lo), lo1 = min(p.budget, lo0 + run_lo);
  const int hi0 = edge + min(n - edge, at_warp * run_hi), hi1 = min(n, hi0 + run_hi);
  const int steps_lo = (lo1 - lo0 + 127) / 128, steps = steps_lo + (hi1 - hi0 + 127) / 128;
  uint32_t* const cached = s_keys + warp * (run_lo + run_hi) + 4 * lane;
  // this lane's first slot of a step, and the end of its run
  auto slot_of = [&](int i) { return (i < steps_lo ? lo0 + 128 * i : hi0 + 128 * (i - steps_lo)) + 4 * lane; };
  auto end_of = [&](int i) { return i < steps_lo ? lo1 : hi1; };
  auto begin_of = [&](int i) { return i < steps_lo ? 0 : p.budget; };
  __syncthreads();  // the histograms are zero
  // First digit, with the keys on their way into shared memory.  Slots outside a run
  // have keys 0, the lowest: more of those change no digit of the budget-th largest
  // key.  Tokens below the budget are written as if they were kept; the moves overwrite
  // those that go.
  const bool copy_w = p.weights_out != p.weights, copy_pos = p.pos_out && p.pos_out != p.pos;
  auto make_keys = [&](int i, int x, const float4& w, const int4& at) {
    const int begin = begin_of(i), end = end_of(i);
    auto key = [&](int e, float weight, int place) {
      return x + e >= begin && x + e < end ? keys.of(weight, place) : 0u;
    };
    return make_uint4(key(0, w.x, at.x), key(1, w.y, at.y), key(2, w.z, at.z), key(3, w.w, at.w));
  };
  for (int i = 0; i < steps; i += kBatch) {
    float4 w[kBatch];
    int4 at[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (i + u >= steps) break;
      const int x = slot_of(i + u);
      at[u] = make_int4(x, x + 1, x + 2, x + 3);
      if (x < end_of(i + u)) {
        w[u] = *reinterpret_cast<const float4*>(keys.w + x);
        if (keys.pos) at[u] = *reinterpret_cast<const int4*>(keys.pos + x);
      }
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (i + u >= steps) break;
      const int x = slot_of(i + u);
      uint4 k = make_uint4(0u, 0u, 0u, 0u);
      if (x < end_of(i + u)) {
        k = make_keys(i + u, x, w[u], at[u]);
        atomicAdd(&s.hist[0][k.x >> 24], 1);
        atomicAdd(&s.hist[0][k.y >> 24], 1);
        atomicAdd(&s.hist[0][k.z >> 24], 1);
        atomicAdd(&s.hist[0][k.w >> 24], 1);
        if (i + u < steps_lo) {
          if (x < edge) {
            if (copy_w) *reinterpret_cast<float4*>(p.weights_out + base + x) = w[u];
            if (copy_pos) *reinterpret_cast<int4*>(p.pos_out + base + x) = at[u];
          } else {
            const float ws[3] = {w[u].x, w[u].y, w[u].z};
            const int as[3] = {at[u].x, at[u].y, at[u].z};
#pragma unroll
            for (int e = 0; e < 3; ++e) {
              if (x + e < p.budget && copy_w) p.weights_out[base + x + e] = ws[e];
              if (x + e < p.budget && copy_pos) p.pos_out[base + x + e] = as[e];
            }
          }
        }
      }
      if (CACHED) *reinterpret_cast<uint4*>(cached + 128 * (i + u)) = k;
    }
  }
  // this lane's keys of a step
  auto keys4 = [&](int i) {
    if (CACHED) return *reinterpret_cast<const uint4*>(cached + 128 * i);
    const int x = slot_of(i);
    if (x >= end_of(i)) return make_uint4(0u, 0u, 0u, 0u);
    const float4 w = *reinterpret_cast<const float4*>(keys.w + x);
    int4 at = make_int4(x, x + 1, x + 2, x + 3);
    if (keys.pos) at = *reinterpret_cast<const int4*>(keys.pos + x);
    return make_keys(i, x, w, at);
  };
  // The budget-th largest key: its digits from the top; `left` is its rank among
  // the keys that share the digits so far.
  uint32_t prefix = 0;
  int left = p.budget;
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    int* hist = s.hist[pass];
    const uint32_t mask = pass > 0 ? 0xFFFFFFFFu << (shift + 8) : 0u;
    if (pass == 3 && s.listed <= kListed) {
      for (int x = threadIdx.x; x < s.listed; x += kSelThreads) {
        const uint32_t k = s.list[x];
        if ((k & mask) == prefix) atomicAdd(&hist[k & (kBins - 1)], 1);
      }
    } else if (pass > 0) {
      int over = 0, over_lo = 0;  // keys above these digits
#pragma unroll 4
      for (int i = 0; i < steps; ++i) {
        if (i == steps_lo) {
          over_lo = over;
          over = 0;
        }
        const uint4 k4 = keys4(i);
        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t digits = k[e] & mask;
          over += digits > prefix;
          if (digits == prefix) {
            atomicAdd(&hist[(k[e] >> shift) & (kBins - 1)], 1);
            if (pass == 2) {
              const int x = atomicAdd(&s.listed, 1);
              if (x < kListed) {
                s.list[x] = k[e];
                s.list_of[x] = (uint8_t)(2 * warp + (i < steps_lo ? 0 : 1));
              }
            }
          }
        }
      }
      if (pass == 2) {
        if (steps == steps_lo) {
          over_lo = over;
          over = 0;
        }
        over_lo = __reduce_add_sync(0xFFFFFFFFu, over_lo);
        over = __reduce_add_sync(0xFFFFFFFFu, over);
        if (lane == 0) *reinterpret_cast<int4*>(s.warp_counts[warp]) = make_int4(over_lo, 0, over, 0);
        if (parts == 1) {
          __syncthreads();
          const int listed = s.listed;
          if (listed <= kFew) {
            if (threadIdx.x < listed) {
              const uint32_t k = s.list[threadIdx.x];
              int above = 0, same = 0;
              for (int x = 0; x < listed; ++x) {
                above += s.list[x] > k;
                same += s.list[x] == k;
              }
              if (above < left && left <= above + same) {
                s.threshold = k;
                s.left = left - above;
              }
            }
            __syncthreads();
            prefix = s.threshold;
            left = s.left;
            break;
          }
        }
      }
    }
    meet();  // the cluster's histograms of this pass are whole
    if (parts > 1) {
      if (threadIdx.x < kBins) {
        int v[kMaxParts], sum = 0;  // all loads on their way before the first sum
#pragma unroll
        for (int x = 0; x < kMaxParts; ++x) v[x] = x < parts ? cluster.map_shared_rank(hist, x)[threadIdx.x] : 0;
#pragma unroll
        for (int x = 0; x < kMaxParts; ++x) sum += v[x];
        s.sum[pass & 1][threadIdx.x] = sum;
      }
      __syncthreads();
    }
    // every warp finds the digit: a lane holds eight bins, from the top
    const int* all = parts > 1 ? s.sum[pass & 1] : hist;
    const int top = kBins - 1 - 8 * lane;
    const int4 c0123 = *reinterpret_cast<const int4*>(all + top - 3), c4567 = *reinterpret_cast<const int4*>(all + top - 7);
    const int c[8] = {c0123.w, c0123.z, c0123.y, c0123.x, c4567.w, c4567.z, c4567.y, c4567.x};
    int mine = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) mine += c[e];
    const int up = inclusive_sum(mine, lane);
    int above = up - mine, digit = 0, before = 0;
    const bool here = above < left && left <= up;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (above < left && left <= above + c[e]) {
        digit = top - e;
        before = above;
      }
      above += c[e];
    }
    const int from = __ffs(__ballot_sync(0xFFFFFFFFu, here)) - 1;
    prefix |= (uint32_t)__shfl_sync(0xFFFFFFFFu, digit, from) << shift;
    left -= __shfl_sync(0xFFFFFFFFu, before, from);
  }
  // Places, in the order of the slots.  Kept are the keys above the threshold and the
  // first `left` equal ones, so that of the first e equal ones min(e, left) are: one
  // round of counts gives every warp the number of freed slots and of movers before it.
  // The counts of the third pass lack the keys that share its digits.
  auto in_of = [&](int x, int end) { return x + 4 <= end ? 15u : x < end ? (1u << (end - x)) - 1u : 0u; };
  // bits of a step's slots x .. x + 3 that are this lane's
  auto mine_of = [&](int i, int x) { return in_of(x, end_of(i)) & ~in_of(x, begin_of(i)); };
  // bits of the slots above and equal to the threshold (key 0 is above none)
  auto compare = [&](int i, int x, uint32_t* over, uint32_t* same) {
    const uint4 k4 = keys4(i);
    const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
    *over = *same = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      *over |= (k[e] > prefix ? 1u : 0u) << e;
      *same |= (k[e] == prefix ? 1u : 0u) << e;
    }
    if (prefix == 0) *same &= mine_of(i, x);
  };
  if (prefix != 0 && s.listed <= kListed) {
    for (int x = threadIdx.x; x < s.listed; x += kSelThreads)
      if (s.list[x] >= prefix) {
        const int of = s.list_of[x];
        atomicAdd(&s.warp_counts[of >> 1][2 * (of & 1) + (s.list[x] == prefix)], 1);
      }
  } else {
    int4 c = make_int4(0, 0, 0, 0);
    for (int i = 0; i < steps; ++i) {
      uint32_t over, same;
      compare(i, slot_of(i), &over, &same);
      if (i < steps_lo) {
        c.x += __popc(over);
        c.y += __popc(same);
      } else {
        c.z += __popc(over);
        c.w += __popc(same);
      }
    }
    c = make_int4(__reduce_add_sync(0xFFFFFFFFu, c.x), __reduce_add_sync(0xFFFFFFFFu, c.y),
                  __reduce_add_sync(0xFFFFFFFFu, c.z), __reduce_add_sync(0xFFFFFFFFu, c.w));
    if (lane == 0) *reinterpret_cast<int4*>(s.warp_counts[warp]) = c;
  }
  __syncthreads();
  auto sum4 = [&](const int4& v, bool on) {
    return Counts{__reduce_add_sync(0xFFFFFFFFu, on ? v.x : 0), __reduce_add_sync(0xFFFFFFFFu, on ? v.y : 0),
                  __reduce_add_sync(0xFFFFFFFFu, on ? v.z : 0), __reduce_add_sync(0xFFFFFFFFu, on ? v.w : 0)};
  };
  const int4 of_warp = *reinterpret_cast<const int4*>(s.warp_counts[lane % kSelWarps]);
  const Counts in_cta = sum4(of_warp, lane < warp);
  if (warp == 0) {
    const Counts c = sum4(of_warp, lane < kSelWarps);
    if (lane == 0) s.counts = make_int4(c.over_lo, c.equal_lo, c.over_hi, c.equal_hi);
  }
  meet();
  int4 of_cta = make_int4(0, 0, 0, 0);  // a lane a CTA
  if (lane < parts) of_cta = parts > 1 ? *cluster.map_shared_rank(&s.counts, lane) : s.counts;
  const Counts in_cluster = sum4(of_cta, lane < rank), all = sum4(of_cta, true);
  // the cluster's counts are read: a CTA may leave once all have come here
  if (parts > 1) cluster.barrier_arrive();
  // equal keys before this warp's runs, freed slots, movers
  const int taken_lo = min(left, all.equal_lo);
  const int seen_hi = all.equal_lo + in_cluster.equal_hi + in_cta.equal_hi;
  int seen = in_cluster.equal_lo + in_cta.equal_lo;
  int hole = lo0 - (in_cluster.over_lo + in_cta.over_lo) - min(left, seen);
  int mover = in_cluster.over_hi + in_cta.over_hi + min(left, seen_hi) - taken_lo;
  for (int i = 0; i < steps; ++i) {
    const int x = slot_of(i);
    if (i == steps_lo) seen = seen_hi;
    uint32_t over, same;
    compare(i, x, &over, &same);
    uint32_t kept = over;
    if (__any_sync(0xFFFFFFFFu, same != 0)) {
      const int equal = __popc(same), up = inclusive_sum(equal, lane);
      int room = left - (seen + up - equal);  // of this lane's equal keys, the lowest `room` are kept
      seen += __shfl_sync(0xFFFFFFFFu, up, 31);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((same >> e) & 1u) {
          if (room > 0) kept |= 1u << e;
          --room;
        }
    }
    // the slots that are listed: freed ones below the budget, movers behind it
    const bool lo = i < steps_lo;
    const uint32_t out = lo ? mine_of(i, x) & ~kept : kept;
    const int count = __popc(out), up = inclusive_sum(count, lane);
    int* to = reinterpret_cast<int*>(moves) + (lo ? 2 * (hole + up - count) : 2 * (mover + up - count) + 1);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if ((out >> e) & 1u) {
        *to = x + e;
        to += 2;
      }
    const int sum = __shfl_sync(0xFFFFFFFFu, up, 31);
    if (lo) hole += sum;
    else mover += sum;
  }
  if (rank == 0 && threadIdx.x == 0)
    p.counts[row] = make_int2(all.over_hi + min(left, all.equal_lo + all.equal_hi) - taken_lo, p.budget);
  for (int j = rank * kSelThreads + threadIdx.x; j < p.budget; j += parts * kSelThreads) src[j] = j;
  if (parts > 1) cluster.barrier_wait();
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
  constexpr int N = 2;
  for (int i = blockIdx.y * per + (threadIdx.x >> vph_shift); i < c.x; i += N * stride) {
    int2 m[N];
    int to[N], from[N], x[N];
    float w[N];
    uint4 a[N], d[N];
#pragma unroll
    for (int u = 0; u < N; ++u) m[u] = i + u * stride < c.x ? moves[i + u * stride] : make_int2(-1, -1);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      to[u] = from[u] = -1;
      if (m[u].x < 0) continue;
      to[u] = cache_row(p, b, g, m[u].x);
      from[u] = cache_row(p, b, g, m[u].y);
      if (at == 0) {
        w[u] = p.weights[base + m[u].y];
        if (p.pos_out) x[u] = p.pos[base + m[u].y];
      }
    }
#pragma unroll
    for (int u = 0; u < N; ++u)
      if (to[u] >= 0 && from[u] >= 0) {
        a[u] = __ldcs(k + ((size_t)from[u] << vph_shift) + at);
        d[u] = __ldcs(v + ((size_t)from[u] << vph_shift) + at);
      }
#pragma unroll
    for (int u = 0; u < N; ++u) {
      if (at == 0 && m[u].x >= 0) {
        src[m[u].x] = m[u].y;
        p.weights_out[base + m[u].x] = w[u];
        if (p.pos_out) p.pos_out[base + m[u].x] = x[u];
      }
      if (to[u] >= 0 && from[u] >= 0) {
        k[((size_t)to[u] << vph_shift) + at] = a[u];
        v[((size_t)to[u] << vph_shift) + at] = d[u];
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
  const int64_t per_cta = (int64_t)4 * kSelThreads;
  // two runs a warp, of one vector more than the row
  const int64_t keys = ((p.max_len + 3 + parts * per_cta - 1) / (parts * per_cta) + 1) * per_cta;
  const bool cached = keys <= kCachedKeys;
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(select_kernel<true>), kCachedKeys * 4, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)rows * parts);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = cached ? keys * 4 : 0;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = parts;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cached ? cudaLaunchKernelEx(&cfg, select_kernel<true>, p, parts) : cudaLaunchKernelEx(&cfg, select_kernel<false>, p, parts);
  if (e != cudaSuccess) return e;
  const int vph = p.D / (dtype == CAPATTN_BF16 ? 8 : 4);
  int shift = 0;
  while ((1 << shift) < vph) ++shift;
  const int per = kMoveThreads >> shift;
  const int most = min(p.budget, max(1, p.max_len - p.budget));  // rows that can move
  // eight CTAs an SM, no more than there can be moves
  const int y = min(max(1, 152 * 8 / rows), (most + 2 * per - 1) / (2 * per));
  return launch_pdl(move_kernel, dim3(rows, y), dim3(kMoveThreads), 0, s, p, shift);
}

}  // namespace capattn
