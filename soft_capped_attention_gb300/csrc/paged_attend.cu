// Attention of many new tokens per sequence over the paged cache on the CUDA cores (fp32), and
// the rows that are formed once more (both types).
//
// Per query tile (tokens x query heads of one KV head, 64 rows) and 64 slots, with a
// running reference m (log2 units):
//   S = Q K^T, x = log2(e) temp cap(sm_scale S), P = 2^(x - m), l += sum P, O += P V.
// fp32 stays on the CUDA cores: a TF32 product keeps 11 bits of q and k.  256 threads, 4 x 4
// scores each (16 products for two vectors of shared memory) and 4 x D / 16 outputs; Q and K
// lie transposed, so that both products read vectors along rows or keys.
#include <cuda_bf16.h>

#include "cache_math.cuh"
#include "cap_math.cuh"
#include "paged_out.cuh"

namespace capattn {
namespace {

constexpr int BM = 64;
constexpr int TK = 64;
constexpr int kThreads = 256;

template <int D>
struct SimtSmem {
  float q[D][BM];      // transposed
  union {
    float k[D][TK];    // transposed
    float p[TK * BM];  // once the scores are there: key-major; a key's rows in blocks of 4, rotated by key / 4
  };
  float v[TK][D];
  RowMask mask[BM];
  float temp[BM];
  uint32_t live[BM][TK / 32];
  Piece piece;
  ScheduleMem sched;
  int last;
};

__device__ __forceinline__ float4 load4(const float* x) { return *reinterpret_cast<const float4*>(x); }

// Row of the cache that holds a slot of sequence b (a bad page is flagged and read as page 0).
__device__ __forceinline__ size_t cache_row(const CacheParams& c, int b, int g, int slot) {
  int page = c.table[(size_t)b * c.max_pages + (slot >> c.page_shift)];
  if (page < 0 || page >= c.num_pages) {
    atomicOr(c.status, kStatusBadPageBit);
    page = 0;
  }
  return (((size_t)page * c.Hkv + g) << c.page_shift) + (slot & (c.page_size - 1));
}

template <typename T, int D, int METHOD>
__global__ void __launch_bounds__(kThreads, 2)
paged_simt_kernel(PagedParams p) {
  extern __shared__ __align__(16) uint8_t raw[];
  using S = SimtSmem<D>;
  S& s = *reinterpret_cast<S*>(raw);
  constexpr int OC = D / 16;  // output columns of a thread: 4 tx + 64 x
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  pdl_trigger();
  pdl_wait();
  schedule<TK>(p, kThreads, s.sched);
  PieceWalk<TK> walk(p, s.sched, lane);
  const CacheParams& c = p.c;
  const T* kc = static_cast<const T*>(c.k);
  const T* vc = static_cast<const T*>(c.v);
  for (;;) {
    if (warp == 0) {
      const Piece x = walk.next(p);
      if (lane == 0) s.piece = x;
    }
    __syncthreads();
    const Piece x = s.piece;
    if (x.steps < 0) break;
    const int g = x.part / p.parts, h0 = (x.part - g * p.parts) * p.heads;
    const int heads = min(p.heads, c.G - h0), rows = x.count * heads;
    const int head0 = g * c.G + h0;
    if (threadIdx.x < BM) {
      const int r = threadIdx.x;
      const SeqShape sh = {x.row0, x.n, x.len, x.base};
      s.mask[r] = r < rows ? row_mask(p, x.b, g, sh, x.i0 + r / heads) : dead_row();
      s.temp[r] = (r < rows && c.temp ? c.temp[x.row0 + x.i0 + r / heads] : 1.f) * kL2E;
    }
    for (int i = threadIdx.x; i < BM * (D / 4); i += kThreads) {
      const int r = i % BM, d = i / BM * 4;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows)
        a = load4(static_cast<const T*>(c.q) + (size_t)(x.row0 + x.i0 + r / heads) * c.q_stride +
                  (size_t)(head0 + r % heads) * D + d);
      s.q[d][r] = a.x;
      s.q[d + 1][r] = a.y;
      s.q[d + 2][r] = a.z;
      s.q[d + 3][r] = a.w;
    }
    float m[4], l[4], o[4][OC];
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      m[a] = -INFINITY;
      l[a] = 0.f;
#pragma unroll
      for (int e = 0; e < OC; ++e) o[a][e] = 0.f;
    }
    for (int step = 0; step < x.steps; ++step) {
      const int j0 = (x.tile0 + step) * TK;
      __syncthreads();  // the last step's products, the row masks
      for (int i = threadIdx.x; i < TK * (D / 4); i += kThreads) {
        const int r = i % TK, d = i / TK * 4, j = j0 + r;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
        if (j >= x.first && j < x.len) {
          const size_t at = cache_row(c, x.b, g, j) * D + d;
          a = load4(kc + at);
          b = load4(vc + at);
        }
        s.k[d][r] = a.x;
        s.k[d + 1][r] = a.y;
        s.k[d + 2][r] = a.z;
        s.k[d + 3][r] = a.w;
        *reinterpret_cast<float4*>(&s.v[r][d]) = b;
      }
      if (threadIdx.x < 2 * BM) {
        const int r = threadIdx.x >> 1, half = threadIdx.x & 1, c0 = j0 + 32 * half;
        s.live[r][half] = all_live(s.mask[r], c0, 32) ? 0xFFFFFFFFu : live_slots(p, s.mask[r], c0);
      }
      __syncthreads();
      float acc[4][4] = {};
#pragma unroll 8
      for (int d = 0; d < D; ++d) {
        const float4 a = *reinterpret_cast<const float4*>(&s.q[d][4 * ty]), b = *reinterpret_cast<const float4*>(&s.k[d][4 * tx]);
        const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int y = 0; y < 4; ++y)
#pragma unroll
          for (int z = 0; z < 4; ++z) acc[y][z] = fmaf(av[y], bv[z], acc[y][z]);
      }
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const uint32_t live = s.live[4 * ty + y][tx >> 3] >> (4 * (tx & 7));
        const float temp = s.temp[4 * ty + y];
        float top = -INFINITY;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          acc[y][z] = (live >> z) & 1u ? any_cap<METHOD>(acc[y][z], c.cap) * temp : -INFINITY;
          top = fmaxf(top, acc[y][z]);
        }
#pragma unroll
        for (int w = 1; w < 16; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, w));
        top = fmaxf(top, m[y]);
        const float scale = top == -INFINITY ? 1.f : ex2_approx(m[y] - top), ref = top == -INFINITY ? 0.f : top;
        m[y] = top;
        l[y] *= scale;
#pragma unroll
        for (int e = 0; e < OC; ++e) o[y][e] *= scale;
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          acc[y][z] = ex2_approx(acc[y][z] - ref);
          l[y] += acc[y][z];
        }
      }
      __syncthreads();  // P takes the place of K
#pragma unroll
      for (int z = 0; z < 4; ++z)
        *reinterpret_cast<float4*>(&s.p[(4 * tx + z) * BM + 4 * ((ty + tx) & 15)]) =
            make_float4(acc[0][z], acc[1][z], acc[2][z], acc[3][z]);
      __syncthreads();
#pragma unroll 4
      for (int j = 0; j < TK; ++j) {
        const float4 a = *reinterpret_cast<const float4*>(&s.p[j * BM + 4 * ((ty + (j >> 2)) & 15)]);
        const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int w = 0; w < OC / 4; ++w) {
          const float4 b = *reinterpret_cast<const float4*>(&s.v[j][64 * w + 4 * tx]);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            o[y][4 * w] = fmaf(av[y], b.x, o[y][4 * w]);
            o[y][4 * w + 1] = fmaf(av[y], b.y, o[y][4 * w + 1]);
            o[y][4 * w + 2] = fmaf(av[y], b.z, o[y][4 * w + 2]);
            o[y][4 * w + 3] = fmaf(av[y], b.w, o[y][4 * w + 3]);
          }
        }
      }
    }
    // ---------------------------------------------------------- end of a piece
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      const int r = 4 * ty + y;
      float zero = 0.f;  // NaN once an output is not finite
#pragma unroll
      for (int e = 0; e < OC; ++e) zero = fmaf(o[y][e], 0.f, zero);
#pragma unroll
      for (int w = 1; w < 16; w <<= 1) {
        l[y] += __shfl_xor_sync(0xFFFFFFFFu, l[y], w);
        zero += __shfl_xor_sync(0xFFFFFFFFu, zero, w);
      }
      // a row without live slots in this piece has l = 0 (and 0 times anything in O)
      const bool none = m[y] == -INFINITY && l[y] == 0.f, bad = !none && (zero != 0.f || !(l[y] < INFINITY));
      if (r >= rows) continue;
      if (x.whole) {
        const size_t row = (size_t)(x.row0 + x.i0 + r / heads) * c.Hq + head0 + r % heads;
        const float inv = none ? 0.f : 1.f / l[y];
#pragma unroll
        for (int w = 0; w < OC / 4; ++w) {
          const float v[4] = {none ? 0.f : o[y][4 * w] * inv, none ? 0.f : o[y][4 * w + 1] * inv,
                              none ? 0.f : o[y][4 * w + 2] * inv, none ? 0.f : o[y][4 * w + 3] * inv};
          store_values(static_cast<T*>(c.o) + row * D + 64 * w + 4 * tx, v);
        }
        if (tx == 0) {
          if (bad) ask_redo(p);
          c.lse[row] = bad ? kNaN32 : none ? -INFINITY : (m[y] + log2f(l[y])) * kLn2;
        }
      } else {
        const size_t at = (size_t)x.slot * BM + r;
#pragma unroll
        for (int w = 0; w < OC / 4; ++w)
          *reinterpret_cast<float4*>(p.part_o + at * D + 64 * w + 4 * tx) =
              make_float4(o[y][4 * w], o[y][4 * w + 1], o[y][4 * w + 2], o[y][4 * w + 3]);
        if (tx == 0) {
          p.part_ml[at] = make_float2(m[y], none ? 0.f : l[y]);
          reinterpret_cast<uint32_t*>(p.part_bad)[at] = bad ? 1u : 0u;
        }
      }
    }
    __syncthreads();
    if (!x.whole) {
      if (threadIdx.x == 0) s.last = count_tile_piece(p, x);
      __syncthreads();
      const int r = threadIdx.x >> 2;
      if (s.last && r < rows)
        join_row<T, D, BM>(p, x, r, threadIdx.x & 3, (size_t)(x.row0 + x.i0 + r / heads) * c.Hq + head0 + r % heads);
    }
  }
}

// ---------------------------------------------------------------- rows formed once more
// A row whose lse is NaN: its sums overflowed or vanished, or something that is not live
// for it met it in a tile's product (0 times NaN or infinity).  A warp goes over the row's
// live slots one by one with a running maximum and touches no other; four columns of D a
// lane.  Most calls have no such row and end at the flag.
template <typename T, int D, int METHOD>
__global__ void __launch_bounds__(128)
paged_redo_kernel(PagedParams p) {
  constexpr int V = D / 32;
  pdl_trigger();
  pdl_wait();
  if (*reinterpret_cast<volatile uint32_t*>(p.redo) == 0u) return;
  const CacheParams& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t all = (int64_t)p.n_rows * c.Hq, warps = (int64_t)gridDim.x * 4;
  for (int64_t at0 = ((int64_t)blockIdx.x * 4 + warp) * 32; at0 < all; at0 += warps * 32) {
    const int64_t mine = at0 + lane;
    const bool asked = mine < all && isnan(__ldcg(c.lse + mine));
    for (uint32_t left = __ballot_sync(0xFFFFFFFFu, asked); left; left &= left - 1u) {
      const int64_t at = at0 + __ffs(left) - 1;
      const int row = (int)(at / c.Hq), h = (int)(at % c.Hq), g = h / c.G;
      int lo = 0, hi = c.B;  // the first b with cu_new[b + 1] > row
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p.cu_new[mid + 1] <= row) lo = mid + 1; else hi = mid;
      }
      if (lo >= c.B || p.cu_new[lo] > row) continue;  // nobody's
      const SeqShape s = seq_shape(p, lo);
      const int i = row - s.row0;
      if (i < 0 || i >= s.n) continue;
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
          size_t src[4];
          bool in[4];
          float kv[4][V], vv[4][V], t[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            in[u] = bits != 0u;
            src[u] = 0;
            if (in[u]) {
              src[u] = cache_row(c, lo, g, c0 + __ffs(bits) - 1) * D + lane * V;
              bits &= bits - 1u;
            }
#pragma unroll
            for (int e = 0; e < V; ++e) {
              kv[u][e] = in[u] ? (float)static_cast<const T*>(c.k)[src[u] + e] : 0.f;
              vv[u][e] = in[u] ? (float)static_cast<const T*>(c.v)[src[u] + e] : 0.f;
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
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int e = 0; e < V; ++e) static_cast<T*>(c.o)[(size_t)at * D + lane * V + e] = (T)(l == 0.f ? 0.f : o[e] * inv);
      if (lane == 0) c.lse[at] = l == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m) + log2f(l)) * kLn2;
    }
  }
  // the last CTA clears the flag for the next call
  __syncthreads();
  if (threadIdx.x == 0 && atomicAdd(p.redo + 1, 1u) == gridDim.x - 1) {
    p.redo[0] = 0u;
    p.redo[1] = 0u;
  }
}

template <typename T, int D, int METHOD>
cudaError_t run_simt(const PagedParams& p, cudaStream_t s) {
  auto* k = paged_simt_kernel<T, D, METHOD>;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), sizeof(SimtSmem<D>), done);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3(p.ctas), dim3(kThreads), sizeof(SimtSmem<D>), s, p);
}

template <typename T, int D, int METHOD>
cudaError_t run_redo(const PagedParams& p, cudaStream_t s) {
  return launch_pdl(paged_redo_kernel<T, D, METHOD>, dim3(kAttendCtas), dim3(128), 0, s, p);
}

template <typename T, int D, int METHOD>
cudaError_t run(const PagedParams& p, bool redo, cudaStream_t s) {
  if constexpr (sizeof(T) == 4) {
    if (!redo) return run_simt<T, D, METHOD>(p, s);
  }
  return run_redo<T, D, METHOD>(p, s);
}

template <typename T, int D>
cudaError_t run_cap(const PagedParams& p, bool redo, cudaStream_t s) {
  switch (p.c.method) {
    case CAPATTN_CAP_TANH: return run<T, D, CAPATTN_CAP_TANH>(p, redo, s);
    case CAPATTN_CAP_SOFT_SIGN: return run<T, D, CAPATTN_CAP_SOFT_SIGN>(p, redo, s);
    case CAPATTN_CAP_ALSC: return run<T, D, CAPATTN_CAP_ALSC>(p, redo, s);
    default: return run<T, D, CAPATTN_CAP_NONE>(p, redo, s);
  }
}

template <typename T>
cudaError_t run_dim(const PagedParams& p, bool redo, cudaStream_t s) {
  return p.c.D == 64 ? run_cap<T, 64>(p, redo, s) : run_cap<T, 128>(p, redo, s);
}

}  // namespace

cudaError_t launch_paged_attend_simt(const PagedParams& p0, cudaStream_t s) {
  PagedParams p = p0;
  p.parts = (p.c.G + BM - 1) / BM;
  p.heads = (p.c.G + p.parts - 1) / p.parts;
  p.tokens = BM / p.heads;
  p.ctas = kAttendSimtCtas;
  p.min_units = 4;
  return run_dim<float>(p, false, s);
}

cudaError_t launch_paged_redo(const PagedParams& p, int dtype, cudaStream_t s) {
  return dtype == CAPATTN_BF16 ? run_dim<__nv_bfloat16>(p, true, s) : run_dim<float>(p, true, s);
}

}  // namespace capattn
