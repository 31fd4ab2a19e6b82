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
#include "cache_internal.h"

namespace capattn {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;

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
  __device__ __forceinline__ uint32_t at(int j) const {
    const int x = pos ? pos[j] : j;
    return x < first || x > after ? 0xFFFFFFFFu : weight_key(w[j]);
  }
};

// Exclusive sum over the block's warps of one count a warp; *total the whole.
__device__ __forceinline__ int warp_offsets(int mine, int* buf, int warp, int lane, int* total) {
  __syncthreads();
  if (lane == 0) buf[warp] = mine;
  __syncthreads();
  int x = lane < kSelWarps ? buf[lane] : 0, up = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, up, d);
    if (lane >= d) up += y;
  }
  *total = __shfl_sync(0xFFFFFFFFu, up, 31);
  return __shfl_sync(0xFFFFFFFFu, up - x, warp);
}

__global__ void __launch_bounds__(kSelThreads)
select_kernel(CacheParams p) {
  __shared__ int hist[256];
  __shared__ int buf[kSelWarps];
  __shared__ uint32_t s_digit;
  __shared__ int s_above;
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x, b = row / p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
  if (n <= p.budget) {  // nothing goes
    for (int j = threadIdx.x; j < p.budget; j += kSelThreads) {
      src[j] = j < n ? j : -1;
      if (j < n && p.weights_out != p.weights) p.weights_out[base + j] = keys.w[j];
      if (j < n && p.pos_out && p.pos_out != p.pos) p.pos_out[base + j] = keys.pos[j];
    }
    if (threadIdx.x == 0) p.counts[row] = make_int2(0, n);
    return;
  }
  // the budget-th largest key: its digits from the top, `left` = its rank among
  // the keys that share the digits so far
  uint32_t prefix = 0;
  int left = p.budget;
  for (int shift = 24; shift >= 0; shift -= 8) {
    const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
    if (threadIdx.x < 256) hist[threadIdx.x] = 0;
    __syncthreads();
    for (int j = threadIdx.x; j < n; j += kSelThreads) {
      const uint32_t k = keys.at(j);
      if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1);
    }
    __syncthreads();
    if (warp == 0) {
      // lane l holds digits 255 - 8 l .. 248 - 8 l, from the top
      int c[8], sum = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[e] = hist[255 - 8 * lane - e];
        sum += c[e];
      }
      int up = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, up, d);
        if (lane >= d) up += y;
      }
      int above = up - sum;
      if (above < left && left <= up) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (above < left && left <= above + c[e]) {
            s_digit = (uint32_t)(255 - 8 * lane - e);
            s_above = above;
            above = left;  // found
          } else {
            above += c[e];
          }
        }
      }
    }
    __syncthreads();
    prefix |= s_digit << shift;
    left -= s_above;
  }
  // Slots in order: a warp takes a run of consecutive slots (whole groups of 32).
  const int run = ((n + kSelWarps * 32 - 1) / (kSelWarps * 32)) * 32;
  const int j0 = min(n, warp * run), j1 = min(n, j0 + run);
  int equal = 0;
  for (int j = j0; j < j1; j += 32) {
    const bool eq = j + lane < j1 && keys.at(j + lane) == prefix;
    equal += __popc(__ballot_sync(0xFFFFFFFFu, eq));
  }
  int total;
  const int eq0 = warp_offsets(equal, buf, warp, lane, &total);
  // kept: above the threshold, or among the first `left` equal ones
  const uint32_t below = (1u << lane) - 1u;
  auto kept_of = [&](int j, int& seen) {
    const uint32_t k = j < j1 ? keys.at(j) : 0u;
    const bool eq = j < j1 && k == prefix;
    const uint32_t eqs = __ballot_sync(0xFFFFFFFFu, eq);
    const bool kept = j < j1 && (k > prefix || (eq && seen + __popc(eqs & below) < left));
    seen += __popc(eqs);
    return kept;
  };
  int movers = 0, holes = 0, seen = eq0;
  for (int j = j0; j < j1; j += 32) {
    const bool in = j + lane < j1, kept = kept_of(j + lane, seen);
    movers += __popc(__ballot_sync(0xFFFFFFFFu, kept && j + lane >= p.budget));
    holes += __popc(__ballot_sync(0xFFFFFFFFu, in && !kept && j + lane < p.budget));
  }
  int n_moves, n_holes;
  int mover = warp_offsets(movers, buf, warp, lane, &n_moves);
  int hole = warp_offsets(holes, buf, warp, lane, &n_holes);
  seen = eq0;
  if (j1 > p.budget) {
    for (int j = j0; j < j1; j += 32) {
      const bool moves_it = kept_of(j + lane, seen) && j + lane >= p.budget;
      const uint32_t who = __ballot_sync(0xFFFFFFFFu, moves_it);
      if (moves_it) moves[mover + __popc(who & below)].y = j + lane;
      mover += __popc(who);
    }
  }
  __syncthreads();
  seen = eq0;
  for (int j = j0; j < min(j1, p.budget); j += 32) {
    const int x = j + lane;
    const bool kept = kept_of(x, seen), freed = x < j1 && x < p.budget && !kept;
    const uint32_t who = __ballot_sync(0xFFFFFFFFu, freed);
    if (freed) {
      const int i = hole + __popc(who & below), from = moves[i].y;
      moves[i].x = x;
      src[x] = from;
      p.weights_out[base + x] = keys.w[from];
      if (p.pos_out) p.pos_out[base + x] = keys.pos[from];
    } else if (x < j1 && x < p.budget) {
      src[x] = x;
      if (p.weights_out != p.weights) p.weights_out[base + x] = keys.w[x];
      if (p.pos_out && p.pos_out != p.pos) p.pos_out[base + x] = keys.pos[x];
    }
    hole += __popc(who);
  }
  if (threadIdx.x == 0) p.counts[row] = make_int2(n_moves, p.budget);
}

__device__ __forceinline__ long long cache_row(const CacheParams& p, int b, int g, int slot) {
  const int page = p.table[(size_t)b * p.max_pages + (slot >> p.page_shift)];
  if (page < 0 || page >= p.num_pages) {
    atomicOr(p.status, kStatusBadPageBit);
    return -1;
  }
  return (((long long)page * p.Hkv + g) << p.page_shift) + (slot & (p.page_size - 1));
}

// Copies the rows that move: a group of vph threads a row, K and V together.
constexpr int kMoveThreads = 256;
__global__ void __launch_bounds__(kMoveThreads)
move_kernel(CacheParams p, int vph_shift) {
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x, b = row / p.Hkv, g = row % p.Hkv;
  const int2 c = p.counts[row];
  if (g == 0 && blockIdx.y == 0 && threadIdx.x == 0) p.lens_out[b] = c.y;
  const int2* moves = reinterpret_cast<const int2*>(p.moves + (size_t)row * p.max_len);
  const int per = kMoveThreads >> vph_shift;
  const int at = threadIdx.x & ((1 << vph_shift) - 1);
  uint4* k = static_cast<uint4*>(p.k);
  uint4* v = static_cast<uint4*>(p.v);
  for (int i = blockIdx.y * per + (threadIdx.x >> vph_shift); i < c.x; i += gridDim.y * per) {
    const int2 m = moves[i];
    const long long to = cache_row(p, b, g, m.x), from = cache_row(p, b, g, m.y);
    if (to < 0 || from < 0) continue;
    const uint4 a = k[(from << vph_shift) + at], d = v[(from << vph_shift) + at];
    k[(to << vph_shift) + at] = a;
    v[(to << vph_shift) + at] = d;
  }
}

}  // namespace

cudaError_t launch_cache_evict(const CacheParams& p, int dtype, cudaStream_t s) {
  const int rows = p.B * p.Hkv;
  cudaError_t e = launch_pdl(select_kernel, dim3(rows), dim3(kSelThreads), 0, s, p);
  if (e != cudaSuccess) return e;
  const int vph = p.D / (dtype == CAPATTN_BF16 ? 8 : 4);
  int shift = 0;
  while ((1 << shift) < vph) ++shift;
  const int per = kMoveThreads >> shift;
  const int most = min(p.budget, max(1, p.max_len - p.budget));  // rows that can move
  const int y = min(max(1, (152 * 8 + rows - 1) / rows), (most + per - 1) / per);
  return launch_pdl(move_kernel, dim3(rows, y), dim3(kMoveThreads), 0, s, p, shift);
}

}  // namespace capattn
