// What attention of many new tokens leaves to be done: query tiles that several CTAs shared
// are added up, and rows whose result cannot be trusted are formed once more.
//
// A CTA takes 32 rows of a shared tile at a time.  Where few CTAs share it (prompts: two), its
// eight warps are the four quarters of the columns, twice: every other piece each.  Where many
// do (a long cache's few tokens), it takes one quarter, a warp every eighth piece.  The warps'
// sums are added in order, so the result does not depend on scheduling.  Bound by latency: it
// starts as attention ends, then records, partial results and the sums' exchange follow one
// another (4 to 6 us).  Joining in the attention kernel, by the CTA that ended last, left 151
// SMs idle meanwhile.
#include <cuda_bf16.h>

#include "cache_sched.cuh"
#include "paged_out.cuh"

namespace capattn {
namespace {

constexpr int kGroups = 8;  // warps
constexpr int kThreads = 32 * kGroups;
constexpr int kCtas = 304;
static_assert(kAttendSimtCtas <= 2 * kThreads, "two records a thread");

// One row, over its live slots alone, with a running maximum: a warp, D / 32 columns a lane.
template <typename T, int D, int METHOD>
__device__ __noinline__ void redo_row(const PagedParams& p, int row, int h, int lane) {
  constexpr int V = D / 32;
  const CacheParams& c = p.c;
  const int g = h / c.G;
  int lo = 0, hi = c.B;  // the first b with cu_new[b + 1] > row
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (p.cu_new[mid + 1] <= row) lo = mid + 1; else hi = mid;
  }
  if (lo >= c.B || p.cu_new[lo] > row) return;  // nobody's
  const SeqShape s = seq_shape(p, lo);
  const int i = row - s.row0;
  if (i < 0 || i >= s.n) return;
  const RowMask mask = row_mask(p, lo, g, s, i);
  const float temp = (c.temp ? c.temp[row] : 1.f) * kL2E;
  const T* q = static_cast<const T*>(c.q) + (size_t)row * c.q_stride + (size_t)h * D + lane * V;
  float qv[V], o[V], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    qv[e] = (float)q[e];
    o[e] = 0.f;
  }
  const int end = p.parents ? s.base + i + 1 : mask.hi;
  for (int c0 = mask.lo / 32 * 32; c0 < end; c0 += 32) {
    uint32_t bits = live_slots(p, mask, c0);
    while (bits) {
      // four slots at a time
      bool in[4];
      float kv[4][V], vv[4][V], t[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        in[u] = bits != 0u;
        size_t src = 0;
        if (in[u]) {
          src = cache_row(c, lo, g, c0 + __ffs(bits) - 1) * D + lane * V;
          bits &= bits - 1u;
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          kv[u][e] = in[u] ? (float)static_cast<const T*>(c.k)[src + e] : 0.f;
          vv[u][e] = in[u] ? (float)static_cast<const T*>(c.v)[src + e] : 0.f;
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        t[u] = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) t[u] = fmaf(qv[e], kv[u][e], t[u]);
      }
#pragma unroll
      for (int w = 16; w; w >>= 1)
#pragma unroll
        for (int u = 0; u < 4; ++u) t[u] += __shfl_xor_sync(0xFFFFFFFFu, t[u], w);
      float top = m;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        t[u] = in[u] ? any_cap<METHOD>(t[u], c.cap) * temp : -INFINITY;
        top = fmaxf(top, t[u]);
      }
      const float ref = top == -INFINITY ? 0.f : top, scale = top == -INFINITY ? 1.f : ex2_approx(m - top);
      m = top;
      l *= scale;
#pragma unroll
      for (int e = 0; e < V; ++e) o[e] *= scale;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (!in[u]) continue;
        const float w = ex2_approx(t[u] - ref);
        l += w;
#pragma unroll
        for (int e = 0; e < V; ++e) o[e] = fmaf(w, vv[u][e], o[e]);
      }
    }
  }
  const size_t at = (size_t)row * c.Hq + h;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < V; ++e) static_cast<T*>(c.o)[at * D + lane * V + e] = (T)(l == 0.f ? 0.f : o[e] * inv);
  if (lane == 0) c.lse[at] = l == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m) + log2f(l)) * kLn2;
}

// A sum of pieces of a row: reference, sum and N columns.
template <int N>
struct Sum {
  float m, l, o[N];
  bool bad;
  __device__ __forceinline__ Sum() : m(-INFINITY), l(0.f), bad(false) {
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = 0.f;
  }
  __device__ __forceinline__ void add(float m2, float l2, const float (&o2)[N], bool bad2) {
    if (l2 == 0.f) return;  // no live slot there
    bad = bad || bad2;
    const float top = fmaxf(m, m2);
    const float a = ex2_approx(m - top), f = ex2_approx(m2 - top);  // (m = -inf: a = 0)
    m = top;
    l = fmaf(l2, f, l * a);
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = fmaf(o2[e], f, o[e] * a);
  }
};

// From here on a quarter of the columns a CTA (never: a tree of 24 tokens 18.3 us instead of
// 15.0, one on 131,009 keys 100.6 instead of 93.8; from three pieces on: no different).
constexpr int kManyPieces = 5;

// What GROUPS warps left of columns [first, first + V) of a row, warps w0, w0 + stride, ..
template <int V, int GROUPS, int WIDTH>
__device__ __forceinline__ Sum<V> add_groups(const float (&part)[kGroups][WIDTH][32], int w0, int stride, int first, int lane) {
  Sum<V> sum;
#pragma unroll
  for (int k = 0; k < GROUPS; ++k) {
    const int w = w0 + k * stride;
    float v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = part[w][first + e][lane];
    sum.add(part[w][WIDTH - 3][lane], part[w][WIDTH - 2][lane], v, part[w][WIDTH - 1][lane] != 0.f);
  }
  return sum;
}

template <typename T, int D, int METHOD, int ROWS>
__global__ void __launch_bounds__(kThreads, 2)
paged_finish_kernel(PagedParams p) {
  constexpr int N = D / 4;
  __shared__ float part[kGroups][N + 3][32];
  __shared__ int s_sums[kGroups], s_record, s_in;
  const CacheParams& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  const bool redo_asked = *reinterpret_cast<volatile uint32_t*>(p.redo) != 0u;  // (by the attention kernel, not here)
  // The blocks of work of each record, two records a thread, and their sums.
  auto blocks_of = [&](int i) -> int {
    if (i >= p.ctas || p.records[i].steps < 0) return 0;
    const bool many = p.records[i].c1 - p.records[i].c0 + 1 >= kManyPieces;
    return (p.records[i].count * p.heads + 31) / 32 * (many ? 4 : 1);
  };
  const int n0 = blocks_of(2 * threadIdx.x), n1 = blocks_of(2 * threadIdx.x + 1);
  const int up = lane_scan(n0 + n1, lane);
  if (lane == 31) s_sums[warp] = up;
  __syncthreads();
  int before = up - n0 - n1, all = 0;
#pragma unroll
  for (int w = 0; w < kGroups; ++w) {
    if (w < warp) before += s_sums[w];
    all += s_sums[w];
  }
  for (int block = blockIdx.x; block < all; block += gridDim.x) {
    if (block >= before && block < before + n0 + n1) {
      const bool second = block >= before + n0;
      s_record = 2 * threadIdx.x + (second ? 1 : 0);
      s_in = block - before - (second ? n0 : 0);
    }
    __syncthreads();
    const Piece x = p.records[s_record];
    const bool many = x.c1 - x.c0 + 1 >= kManyPieces;
    const int cq = many ? s_in & 3 : warp & 3, r = 32 * (many ? s_in >> 2 : s_in) + lane;
    const int group = many ? warp : warp >> 2, groups = many ? kGroups : kGroups / 4;
    const int g = x.part / p.parts, h0 = (x.part - g * p.parts) * p.heads, heads = min(p.heads, c.G - h0);
    Sum<N> sum;
#pragma unroll 2
    for (int k = x.c0 + group; k <= x.c1; k += groups) {
      const int slot = piece_slot(x, k);
      const float2 ml = __ldcg(p.part_ml + (size_t)slot * ROWS + r);
      const bool bad = __ldcg(p.part_bad + (size_t)slot * ROWS + r) != 0u;
      float v[N];
#pragma unroll
      for (int e = 0; e < N / 4; ++e) {
        const float4 f = __ldcg(reinterpret_cast<const float4*>(p.part_o) + part_at<D, ROWS>(slot, r, cq, e));
        v[4 * e] = f.x; v[4 * e + 1] = f.y; v[4 * e + 2] = f.z; v[4 * e + 3] = f.w;
      }
      sum.add(ml.x, ml.y, v, bad);
    }
#pragma unroll
    for (int e = 0; e < N; ++e) part[warp][e][lane] = sum.o[e];
    part[warp][N][lane] = sum.m;
    part[warp][N + 1][lane] = sum.l;
    part[warp][N + 2][lane] = sum.bad ? 1.f : 0.f;
    __syncthreads();
    const int t = r / p.heads, hh = r - t * p.heads;
    const bool valid = t < x.count && hh < heads;
    const int tok = x.row0 + x.i0 + t, head = g * c.G + h0 + hh;
    const size_t row = (size_t)tok * c.Hq + head;
    uint32_t redo = 0u;
    // columns [at, at + V) of the row, done; the rows that cannot be trusted are left to one warp
    auto write = [&](const auto& y, int at, bool first) {
      constexpr int V = sizeof(y.o) / sizeof(float);
      const bool none = y.l == 0.f, bad = valid && !none && (y.bad || !(y.l < INFINITY));
      if (valid && !bad) {
        const float inv = none ? 0.f : 1.f / y.l;
        T* to = static_cast<T*>(c.o) + row * D + at;
#pragma unroll
        for (int e = 0; e < V; e += 2) {
          const float a = y.o[e] * inv, b = y.o[e + 1] * inv;
          if constexpr (sizeof(T) == 2) *reinterpret_cast<uint32_t*>(to + e) = pack_bf16x2(a, b);
          else *reinterpret_cast<float2*>(to + e) = make_float2(a, b);
        }
        if (first) c.lse[row] = none ? -INFINITY : (y.m + log2f(y.l)) * kLn2;
      }
      if (first) redo = __ballot_sync(0xFFFFFFFFu, bad);
    };
    if (many) {
      constexpr int V = N / kGroups;
      write(add_groups<V, kGroups>(part, 0, 1, V * warp, lane), cq * N + V * warp, cq == 0 && warp == 0);
    } else {
      constexpr int V = N / 2;
      write(add_groups<V, 2>(part, cq, 4, V * group, lane), cq * N + V * group, warp == 0);
    }
    for (; redo; redo &= redo - 1u) {
      const int l = __ffs(redo) - 1;
      redo_row<T, D, METHOD>(p, __shfl_sync(0xFFFFFFFFu, tok, l), __shfl_sync(0xFFFFFFFFu, head, l), lane);
    }
    __syncthreads();  // part, s_record and s_in have been read
  }
  // Rows of whole tiles: the flag says whether there are any (a shared tile's that come to NaN
  // meanwhile may be met here too, and give the same again).
  if (!redo_asked) return;
  const int64_t lses = (int64_t)p.n_rows * c.Hq, warps = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t at0 = ((int64_t)blockIdx.x * (kThreads / 32) + warp) * 32; at0 < lses; at0 += warps * 32) {
    const int64_t mine = at0 + lane;
    const bool asked = mine < lses && isnan(__ldcg(c.lse + mine));
    for (uint32_t left = __ballot_sync(0xFFFFFFFFu, asked); left; left &= left - 1u) {
      const int64_t at = at0 + __ffs(left) - 1;
      redo_row<T, D, METHOD>(p, (int)(at / c.Hq), (int)(at % c.Hq), lane);
    }
  }
  // the last CTA clears the flag for the next call
  __syncthreads();
  if (threadIdx.x == 0 && atomicAdd(p.redo + 1, 1u) == gridDim.x - 1) {
    p.redo[0] = 0u;
    p.redo[1] = 0u;
  }
}

template <typename T, int D, int METHOD, int ROWS>
cudaError_t launch(const PagedParams& p, cudaStream_t s) {
  return launch_pdl(paged_finish_kernel<T, D, METHOD, ROWS>, dim3(kCtas), dim3(kThreads), 0, s, p);
}

template <int METHOD>
struct PagedFinishLaunch {
  static cudaError_t run(const PagedParams& p, int dtype, cudaStream_t s) {
    if (dtype == CAPATTN_BF16)
      return p.c.D == 64 ? launch<__nv_bfloat16, 64, METHOD, kAttendRows>(p, s)
                         : launch<__nv_bfloat16, 128, METHOD, kAttendRows>(p, s);
    return p.c.D == 64 ? launch<float, 64, METHOD, kAttendSimtRows>(p, s) : launch<float, 128, METHOD, kAttendSimtRows>(p, s);
  }
};

}  // namespace

cudaError_t launch_paged_finish(const PagedParams& p, int dtype, cudaStream_t s) {
  return dispatch_cap<PagedFinishLaunch>(p.c.method, p, dtype, s);
}

}  // namespace capattn
