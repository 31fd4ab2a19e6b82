// What attention of many new tokens leaves to be done: query tiles that several CTAs shared
// are added up, and rows whose result cannot be trusted are formed once more.
//
// A CTA a (CTA of the attention, 32 rows): if a shared tile begins there, two groups of eight
// warps take every other piece each (a warp an eighth of the columns, a lane a row) and the
// groups are added in order, so the result does not depend on scheduling.  Joining in the
// attention kernel, by the CTA that ended last, left 151 SMs idle meanwhile.
#include <cuda_bf16.h>

#include "paged_out.cuh"

namespace capattn {
namespace {

constexpr int kThreads = 512;
constexpr int kGroups = 2;
constexpr int kParts = 8;  // of the columns, a warp each

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

template <int D>
constexpr int smem_bytes() { return (kGroups - 1) * 32 * kParts * (D / kParts + 3) * (int)sizeof(float); }

template <typename T, int D, int METHOD, int ROWS>
__global__ void __launch_bounds__(kThreads, 2)
paged_finish_kernel(PagedParams p) {
  constexpr int N = D / kParts, W = 32 * kParts;
  extern __shared__ float smem[];  // [group - 1][value][W threads]
  const CacheParams& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  pdl_wait();
  const int from = blockIdx.x / (ROWS / 32), block = blockIdx.x % (ROWS / 32);
  const Piece x = p.records[from];
  const int g = x.part / p.parts, h0 = (x.part - g * p.parts) * p.heads;
  const int heads = min(p.heads, c.G - h0);
  if (x.steps > 0 && 32 * block < x.count * heads) {  // (the same for all threads)
    const int part = warp & (kParts - 1), group = warp / kParts, at = threadIdx.x & (W - 1);
    const int r = 32 * block + lane;
    Sum<N> sum;
#pragma unroll 2
    for (int k = x.c0 + group; k <= x.c1; k += kGroups) {
      const int slot = piece_slot(x, k);
      const float2 ml = __ldcg(p.part_ml + (size_t)slot * ROWS + r);
      const bool bad = __ldcg(p.part_bad + (size_t)slot * ROWS + r) != 0u;
      float v[N];
#pragma unroll
      for (int e = 0; e < N / 4; ++e) {
        const float4 f = __ldcg(reinterpret_cast<const float4*>(p.part_o) + part_at<D, ROWS>(slot, r, part >> 1, (part & 1) * (N / 4) + e));
        v[4 * e] = f.x; v[4 * e + 1] = f.y; v[4 * e + 2] = f.z; v[4 * e + 3] = f.w;
      }
      sum.add(ml.x, ml.y, v, bad);
    }
    if (group > 0) {
      float* to = smem + (group - 1) * W * (N + 3) + at;
#pragma unroll
      for (int e = 0; e < N; ++e) to[e * W] = sum.o[e];
      to[N * W] = sum.m;
      to[(N + 1) * W] = sum.l;
      to[(N + 2) * W] = sum.bad ? 1.f : 0.f;
    }
    __syncthreads();
    if (group == 0) {
#pragma unroll 1
      for (int k = 0; k < kGroups - 1; ++k) {
        const float* src = smem + k * W * (N + 3) + at;
        float v[N];
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = src[e * W];
        sum.add(src[N * W], src[(N + 1) * W], v, src[(N + 2) * W] != 0.f);
      }
      const bool valid = r < x.count * heads;
      const int tok = x.row0 + x.i0 + r / heads, head = g * c.G + h0 + r % heads;
      const size_t row = (size_t)tok * c.Hq + head;
      const bool none = sum.l == 0.f, bad = valid && !none && (sum.bad || !(sum.l < INFINITY));
      if (valid && !bad) {
        const float inv = none ? 0.f : 1.f / sum.l;
#pragma unroll
        for (int e = 0; e < N; ++e) sum.o[e] *= inv;
        store_values(static_cast<T*>(c.o) + row * D + part * N, sum.o);
        if (part == 0) c.lse[row] = none ? -INFINITY : (sum.m + log2f(sum.l)) * kLn2;
      }
      if (part == 0)  // (the other warps know of the same rows and leave them alone)
        for (uint32_t left = __ballot_sync(0xFFFFFFFFu, bad); left; left &= left - 1u) {
          const int l = __ffs(left) - 1;
          redo_row<T, D, METHOD>(p, __shfl_sync(0xFFFFFFFFu, tok, l), __shfl_sync(0xFFFFFFFFu, head, l), lane);
        }
    }
  }
  // Rows of whole tiles: the flag says whether there are any (a shared tile's that come to NaN
  // meanwhile may be met here too, and give the same again).
  if (*reinterpret_cast<volatile uint32_t*>(p.redo) == 0u) return;
  const int64_t all = (int64_t)p.n_rows * c.Hq, warps = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t at0 = ((int64_t)blockIdx.x * (kThreads / 32) + warp) * 32; at0 < all; at0 += warps * 32) {
    const int64_t mine = at0 + lane;
    const bool asked = mine < all && isnan(__ldcg(c.lse + mine));
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
  auto* k = paged_finish_kernel<T, D, METHOD, ROWS>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem_bytes<D>(), done);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3(p.ctas * (ROWS / 32)), dim3(kThreads), smem_bytes<D>(), s, p);
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
