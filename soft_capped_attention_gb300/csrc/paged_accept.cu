// Acceptance of a drafted path: a CTA a sequence walks the tree (one warp, 32 candidates at
// a time) or checks the given path, looks up the pages of all rows that move, and moves the
// path's keys and values to the front of the new slots.  A row goes to a slot at or before its own and behind every earlier row's
// source, so a chunk of rows is loaded whole before any of it is stored, and chunks follow
// one another without more ado.  Bound by latency: the walk's dependent reads (from shared
// memory) and one round trip of the rows.  One tree of 25 tokens: 3.5 us; 128 of 33 (8 heads
// x 128, bf16, paths of up to 9): 5.3 us.
#include "paged_internal.h"
#include "tc_common.cuh"

namespace capattn {
namespace {

constexpr int kThreads = 512;
constexpr int kStaged = 1024;  // rows of a sequence whose tokens and parents are staged
constexpr int kVecs = 4;       // 16-byte vectors of K and of V a thread holds

__global__ void __launch_bounds__(kThreads)
accept_kernel(AcceptParams p, int vpr, int vph_shift) {
  __shared__ int s_parent[kStaged], s_token[kStaged], s_says[kStaged];
  __shared__ int s_from[kStaged], s_to[kStaged];  // cache rows of head 0; -1: the row is where it goes
  __shared__ int s_count, s_bad, s_bad_page;
  const CacheParams& c = p.c;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  pdl_trigger();
  pdl_wait();
  const int row0 = p.cu_new[b], end = p.cu_new[b + 1], len = c.lens[b];
  const int qpos = p.qpos_out ? c.qpos[b] : 0;
  uint32_t bad = 0;
  if (len < 0 || len > c.max_len) bad |= kStatusBadLensBit;
  if (row0 < 0 || end < row0 || end > p.n_rows || (!bad && end - row0 > len)) bad |= kStatusBadNewRowsBit;
  const int n = bad ? 0 : end - row0, base = len - n;
  int32_t* path = p.path + (size_t)b * p.width;
  if (tid == 0) {
    s_bad = s_bad_page = 0;
    s_count = 0;
  }
  if (p.tokens) {
    for (int i = tid; i < min(n, kStaged); i += kThreads) {
      s_parent[i] = p.parents[row0 + i];
      s_token[i] = p.tokens[row0 + i];
      s_says[i] = p.predicted[row0 + i];
    }
    __syncthreads();
    if (tid < 32) {
      int at = n > 0 ? 0 : -1, count = 0, says = -1;
      while (at >= 0) {
        if (lane == 0) path[count] = at;
        ++count;
        says = at < kStaged ? s_says[at] : p.predicted[row0 + at];
        int next = -1;
        for (int x0 = at + 1; count < p.width && x0 < n && next < 0; x0 += 32) {
          const int x = x0 + lane;
          bool hit = false;
          if (x < min(n, kStaged)) hit = s_parent[x] == at && s_token[x] == says;
          else if (x < n) hit = p.parents[row0 + x] == at && p.tokens[row0 + x] == says;
          const uint32_t some = __ballot_sync(0xFFFFFFFFu, hit);
          if (some) next = x0 + __ffs(some) - 1;
        }
        at = next;
      }
      for (int i = count + lane; i < p.width; i += 32) path[i] = -1;
      if (lane == 0) {
        s_count = count;
        p.count[b] = count;
        if (p.next) p.next[b] = says;
      }
    }
    __syncthreads();  // path too: written and read by this CTA
  } else {
    __syncthreads();
    const int count = p.count[b];
    if (count < 0 || count > p.width || count > n) {
      if (tid == 0 && !bad) s_bad = 1;
    } else {
      for (int i = tid; i < count; i += kThreads) {
        const int x = path[i];
        if (x < 0 || x >= n || (i > 0 && x <= path[i - 1])) s_bad = 1;
      }
      if (tid == 0) s_count = count;
    }
    __syncthreads();
  }
  if (s_bad) bad |= kStatusBadPathBit;
  const int count = bad ? 0 : s_count;
  // cache row of a slot below len (fewer than 2^31 rows), -1: its page is out of range
  auto row_of = [&](int slot) -> int {
    const int page = c.table[(size_t)b * c.max_pages + (slot >> c.page_shift)];
    if (page < 0 || page >= c.num_pages) return -1;
    return (page * c.Hkv << c.page_shift) + (slot & (c.page_size - 1));
  };
  // every page that the move needs, before anything moves
  for (int i = tid; i < count; i += kThreads) {
    const int x = path[i], from = x == i ? -1 : row_of(base + x), to = x == i ? -1 : row_of(base + i);
    if (x != i && (from < 0 || to < 0)) s_bad_page = 1;
    if (i < kStaged) {
      s_from[i] = from;
      s_to[i] = to;
    }
  }
  __syncthreads();
  if (s_bad_page) {
    bad |= kStatusBadPageBit;
    if (p.tokens) {  // nothing is accepted
      for (int i = tid; i < p.width; i += kThreads) path[i] = -1;
      if (tid == 0) {
        p.count[b] = 0;
        if (p.next) p.next[b] = -1;
      }
    }
  }
  if (bad) {
    // the sequence stays as it is
    if (tid == 0) {
      atomicOr(c.status, bad);
      p.lens_out[b] = len;
      if (p.qpos_out) p.qpos_out[b] = qpos;
    }
    return;
  }
  uint4* kc = static_cast<uint4*>(c.k);
  uint4* vc = static_cast<uint4*>(c.v);
  const long long total = (long long)count * vpr;
  for (long long i0 = tid; i0 - tid < total; i0 += kThreads * kVecs) {
    uint4 a[kVecs], v[kVecs];
    long long dst[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      const long long i = i0 + u * kThreads;
      dst[u] = -1;
      if (i >= total) continue;
      const int r = (int)(i / vpr), w = (int)(i - (long long)r * vpr);
      long long from, to;
      if (r < kStaged) {
        from = s_from[r];
        to = s_to[r];
      } else {
        const int x = path[r];
        from = x == r ? -1 : row_of(base + x);
        to = row_of(base + r);
      }
      if (from < 0) continue;  // is there already
      const long long h = (long long)(w >> vph_shift) << c.page_shift;
      const int at = w & ((1 << vph_shift) - 1);
      a[u] = kc[((from + h) << vph_shift) + at];
      v[u] = vc[((from + h) << vph_shift) + at];
      dst[u] = ((to + h) << vph_shift) + at;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kVecs; ++u)
      if (dst[u] >= 0) {
        kc[dst[u]] = a[u];
        vc[dst[u]] = v[u];
      }
  }
  if (c.weights || c.pos) {
    const long long values = (long long)count * c.Hkv;
    for (long long i0 = tid; i0 - tid < values; i0 += kThreads) {  // tokens in order, heads inside
      const int r = (int)(i0 / c.Hkv), g = (int)(i0 - (long long)r * c.Hkv);
      const size_t row = ((size_t)b * c.Hkv + g) * c.max_len + base;
      float w = 0.f;
      if (i0 < values && c.weights) w = c.weights[row + path[r]];
      __syncthreads();
      if (i0 < values) {
        if (c.weights) c.weights[row + r] = w;
        if (c.pos) c.pos[row + r] = qpos - n + 1 + r;
      }
    }
  }
  if (tid == 0) {
    p.lens_out[b] = base + count;
    if (p.qpos_out) p.qpos_out[b] = qpos - n + count;
  }
}

}  // namespace

cudaError_t launch_paged_accept(const AcceptParams& p, int dtype, cudaStream_t s) {
  const int vph = p.c.D / (dtype == CAPATTN_BF16 ? 8 : 4);  // 16-byte vectors of a head's row
  int shift = 0;
  while ((1 << shift) < vph) ++shift;
  return launch_pdl(accept_kernel, dim3(p.c.B), dim3(kThreads), 0, s, p, p.c.Hkv * vph, shift);
}

}  // namespace capattn
