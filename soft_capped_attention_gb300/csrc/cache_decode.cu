// Attention of one new token per sequence over the paged cache: the CUDA-core
// kernel (fp32) and the weights pass.
//
// Per (sequence b, group of up to 16 query heads of one KV head), over live
// slots j:  t_j = temp cap(sm_scale <q, k_j>),  m = max t, l = sum e^(t - m),
// O = sum e^(t - m) v_j, kept as a running triple; o = O / l, lse = m + log l.
// Pieces (m_i, l_i, O_i) of a split join as M = max m_i, l = sum l_i e^(m_i - M),
// O likewise.
//   fp32 stays on the CUDA cores (a TF32 product keeps 11 bits of q and k).  Memory
// bounds a group of one head (4 sequences of 16,000 keys x 8 heads, D = 128, 524 MB:
// 95 us, 5.5 TB/s); a larger one is bound by reading the tile from shared memory once a
// head, by eight warps an SM (4 heads: 125 us, 16 heads: 356 us, of which the products
// alone would take 56: the shared-memory pipe is 66 % busy, the FMA pipe 20 %).
#include "cache_internal.h"
#include "cache_math.cuh"
#include "cache_sched.cuh"

namespace capattn {
namespace {

constexpr int TK = 32;         // keys of a tile: one a lane
constexpr int kThreads = 128;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
  const int bytes = live ? 16 : 0;  // 0: the 16 bytes are filled with zeros
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Dot product of 16 bytes of a key row with q in shared memory.
__device__ __forceinline__ void dot16(float& acc, const float* k, const float* q) {
  const float4 a = *reinterpret_cast<const float4*>(k), b = *reinterpret_cast<const float4*>(q);
  acc = fmaf(a.x, b.x, acc);
  acc = fmaf(a.y, b.y, acc);
  acc = fmaf(a.z, b.z, acc);
  acc = fmaf(a.w, b.w, acc);
}
template <typename T, int D, int GM>
struct Smem {
  static constexpr int PER = 16 / sizeof(T);
  static constexpr int ROW = D + PER;  // a row's stride: 16 bytes of padding against bank conflicts
  static constexpr int PARTS = kThreads / D;
  T k[2][TK][ROW];
  T v[2][TK][ROW];
  float q[GM][D];
  float p[GM][TK];
  float scale[GM], m[GM], l[GM];
  float half[PARTS > 1 ? GM : 1][64];  // D = 64: outputs of the second half of the threads
  float lsum[32];
  int flag;
  // the join's 4 x 4 x D floats: no tile is in flight at a piece's end (every copy that a
  // piece starts belongs to one of its tiles, and the last one waits for all)
  __device__ float* join() { return reinterpret_cast<float*>(&k[0][0][0]); }
  static_assert(2 * TK * ROW * sizeof(T) >= 16 * D * sizeof(float), "the join's buffer");
};

// Tiles of 32 keys come in by cp.async, two stages.  Scores: warp w takes heads
// w, w + 4, .., a lane a key (its row in 16-byte pieces; the padding spreads the
// lanes over the banks, q is a broadcast).  Outputs: a thread takes a column d
// (D = 64: and half of the keys) of every head.
template <typename T, int D, int METHOD, int GM>
__global__ void __launch_bounds__(kThreads)
decode_simt_kernel(CacheParams p) {
  extern __shared__ __align__(16) uint8_t raw[];
  using S = Smem<T, D, GM>;
  S& s = *reinterpret_cast<S*>(raw);
  constexpr int CH = D / S::PER;            // 16-byte pieces of a row
  constexpr int NH = (GM + 3) / 4;          // heads of a warp
  constexpr int PARTS = kThreads / D;       // threads of a column
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int d = threadIdx.x % D, part = threadIdx.x / D;
  const T* kc = static_cast<const T*>(p.k);
  const T* vc = static_cast<const T*>(p.v);
  __shared__ int s_sums[kSchedSums + 32];
  PieceIter<TK> it(p, warp, lane, kThreads / 32, s_sums);
  int b, vh, tile;
  SeqSpan sp;
  while (it.next(p, &b, &vh, &tile, &sp)) {
    const HeadGroup hg = head_group(p, vh);
    const int n = it.n;
    for (int i = threadIdx.x; i < GM * D; i += kThreads) {
      const int g = i / D;
      s.q[g][i % D] = g < hg.count
          ? static_cast<const T*>(p.q)[(size_t)b * p.q_stride + (size_t)(hg.h0 + g) * D + i % D] : 0.f;
    }
    const float temp = p.temp ? p.temp[b] : 1.f;
    const int qpos = p.pos ? p.qpos[b] : 0;
    const int32_t* pos = p.pos ? p.pos + ((size_t)b * p.Hkv + hg.g) * p.max_len : nullptr;
    auto load = [&](int i) {
      const int st = i & 1, j0 = (tile + i) * TK;
      for (int c = threadIdx.x; c < TK * CH; c += kThreads) {
        const int r = c / CH, x = c % CH, j = j0 + r;
        const bool live = j >= sp.first && j < sp.len;
        size_t at = 0;
        if (live) {
          const size_t row = (((size_t)page_of(p, b, j) * p.Hkv + hg.g) << p.page_shift) + (j & (p.page_size - 1));
          at = row * D + x * S::PER;
        }
        cp_async16(smem_u32(&s.k[st][r][x * S::PER]), kc + at, live);
        cp_async16(smem_u32(&s.v[st][r][x * S::PER]), vc + at, live);
      }
      cp_commit();
    };
    float m[NH], l[NH], acc[GM];
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
#pragma unroll
    for (int g = 0; g < GM; ++g) acc[g] = 0.f;
    if (n > 0) load(0);  // a piece may be a group's first unit alone, or an empty sequence
    for (int i = 0; i < n; ++i) {
      const int st = i & 1;
      if (i + 1 < n) {
        load(i + 1);
        cp_wait<1>();
      } else {
        cp_wait<0>();
      }
      __syncthreads();
      const int j = (tile + i) * TK + lane;
      bool live = j >= sp.first && j < sp.len;
      if (pos && p.window_len > 0 && live && pos[j] <= qpos - p.window_len) {
        live = false;
        if (warp == 0)  // a masked row must not reach the sum, whatever it holds
          for (int x = 0; x < D; ++x) s.v[st][lane][x] = (T)0.f;
      }
#pragma unroll
      for (int u = 0; u < NH; ++u) {
        const int g = warp + 4 * u;
        if (g < hg.count) {
          float dot = 0.f;
#pragma unroll 8
          for (int x = 0; x < CH; ++x) dot16(dot, &s.k[st][lane][x * S::PER], &s.q[g][x * S::PER]);
          float t = exact_cap<METHOD>(dot * p.sm_scale, p.cap) * temp;
          t = live ? t : -INFINITY;
          if (p.scores && j < sp.len)
            p.scores[((size_t)b * p.Hq + hg.h0 + g) * p.max_len + j] = t;
          float mx = t;
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, x));
          mx = fmaxf(mx, m[u]);
          const float ref = mx == -INFINITY ? 0.f : mx;
          const float scale = __expf(m[u] - ref);
          const float e = __expf(t - ref);
          float sum = e;
#pragma unroll
          for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, x);
          m[u] = mx;
          l[u] = l[u] * scale + sum;
          s.p[g][lane] = e;
          if (lane == 0) s.scale[g] = scale;
        }
      }
      __syncthreads();
      constexpr int KEYS = TK / PARTS;
#pragma unroll
      for (int g = 0; g < GM; ++g)
        if (g < hg.count) acc[g] *= s.scale[g];
#pragma unroll 4
      for (int k4 = 0; k4 < KEYS; k4 += 4) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = s.v[st][part * KEYS + k4 + e][d];
#pragma unroll
        for (int g = 0; g < GM; ++g) {
          if (g < hg.count) {
            const float4 w = *reinterpret_cast<const float4*>(&s.p[g][part * KEYS + k4]);
            acc[g] = fmaf(w.x, v[0], fmaf(w.y, v[1], fmaf(w.z, v[2], fmaf(w.w, v[3], acc[g]))));
          }
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < NH; ++u) {
      const int g = warp + 4 * u;
      if (lane == 0 && g < hg.count) {
        s.m[g] = m[u];
        s.l[g] = l[u];
      }
    }
    if (PARTS > 1 && part == 1) {
#pragma unroll
      for (int g = 0; g < GM; ++g) s.half[g][d & 63] = acc[g];
    }
    __syncthreads();
    if (part == 0) {
#pragma unroll
      for (int g = 0; g < GM; ++g) {
        if (g >= hg.count) continue;
        float o = acc[g];
        if (PARTS > 1) o += s.half[g][d & 63];
        if (it.whole) {
          const float lg = s.l[g];
          const size_t row = (size_t)b * p.Hq + hg.h0 + g;
          static_cast<T*>(p.o)[row * D + d] = (T)(lg == 0.f ? 0.f : o / lg);
          if (d == 0) p.lse[row] = lg == 0.f ? -INFINITY : s.m[g] + logf(lg);
        } else {
          p.part_o[((size_t)it.slot * kDecodeHeads + g) * D + d] = o;
          if (d == 0) p.part_ml[(size_t)it.slot * kDecodeHeads + g] = make_float2(s.m[g], s.l[g]);
        }
      }
    }
    __syncthreads();
    if (!it.whole) {
      const Pieces pc(it);
      if (threadIdx.x == 0) s.flag = count_piece(p, pc);
      __syncthreads();
      if (s.flag) join_pieces<T, D, 4>(p, pc, b, hg, warp, lane, 1, s.join(), s.lsum);
      __syncthreads();
    }
  }
}

// weights[b, g, j] += sum over the group's heads of exp(t - lse): a thread four
// consecutive slots (rows are whole 16-byte units: max_len is a multiple of 8).
__global__ void __launch_bounds__(128)
decode_weights_kernel(CacheParams p) {
  pdl_trigger();
  pdl_wait();
  const int row = blockIdx.x, b = row / p.Hkv, g = row - b * p.Hkv;
  const SeqSpan sp = seq_span<64>(p, b);
  const float* lse = p.lse + (size_t)b * p.Hq + (size_t)g * p.G;
  const float* sc = p.scores + ((size_t)b * p.Hq + (size_t)g * p.G) * p.max_len;
  float* out = p.weights + (size_t)row * p.max_len;
  for (int j = (sp.first & ~3) + 4 * (blockIdx.y * 128 + threadIdx.x); j < sp.len; j += gridDim.y * 512) {
    float4 w = *reinterpret_cast<const float4*>(out + j);
    float4 add = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int h = 0; h < p.G; ++h) {
      const float4 t = __ldcs(reinterpret_cast<const float4*>(sc + (size_t)h * p.max_len + j));
      const float n = lse[h];
      // a dead score is -inf (and the norm of a head without live keys too)
      add.x += t.x == -INFINITY ? 0.f : __expf(t.x - n);
      add.y += t.y == -INFINITY ? 0.f : __expf(t.y - n);
      add.z += t.z == -INFINITY ? 0.f : __expf(t.z - n);
      add.w += t.w == -INFINITY ? 0.f : __expf(t.w - n);
    }
    if (j >= sp.first && j + 4 <= sp.len) {
      *reinterpret_cast<float4*>(out + j) = make_float4(w.x + add.x, w.y + add.y, w.z + add.z, w.w + add.w);
    } else {
      const float a[4] = {w.x + add.x, w.y + add.y, w.z + add.z, w.w + add.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (j + e >= sp.first && j + e < sp.len) out[j + e] = a[e];
    }
  }
}

template <int D, int METHOD, int GM>
cudaError_t run_simt(const CacheParams& p0, cudaStream_t s) {
  auto* k = decode_simt_kernel<float, D, METHOD, GM>;
  static std::atomic<uint64_t> done{0};
  const int smem = sizeof(Smem<float, D, GM>);
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem, done);
  if (e != cudaSuccess) return e;
  // as many CTAs as the SMs hold at once (three by their registers), no more than
  // there can be tiles
  CacheParams p = p0;
  const int per_sm = 227 * 1024 / (smem + 1024) < 3 ? 227 * 1024 / (smem + 1024) : 3;
  const int64_t most = (int64_t)p.B * p.VH * ((p.max_len + TK - 1) / TK);
  p.ctas = (int)(most < 152 * per_sm ? most : 152 * per_sm);
  p.min_tiles = 2;
  return launch_pdl(k, dim3(p.ctas), dim3(kThreads), smem, s, p);
}

template <int D, int METHOD>
cudaError_t run_heads(const CacheParams& p, cudaStream_t s) {
  const int n = p.G < kDecodeHeads ? p.G : kDecodeHeads;
  if (n <= 1) return run_simt<D, METHOD, 1>(p, s);
  if (n <= 4) return run_simt<D, METHOD, 4>(p, s);
  return run_simt<D, METHOD, 16>(p, s);
}

template <int D>
cudaError_t run_cap(const CacheParams& p, cudaStream_t s) {
  switch (p.method) {
    case CAPATTN_CAP_TANH: return run_heads<D, CAPATTN_CAP_TANH>(p, s);
    case CAPATTN_CAP_SOFT_SIGN: return run_heads<D, CAPATTN_CAP_SOFT_SIGN>(p, s);
    case CAPATTN_CAP_ALSC: return run_heads<D, CAPATTN_CAP_ALSC>(p, s);
    default: return run_heads<D, CAPATTN_CAP_NONE>(p, s);
  }
}

cudaError_t launch_decode_fp32(const CacheParams& p, cudaStream_t s) {
  return p.D == 64 ? run_cap<64>(p, s) : run_cap<128>(p, s);
}

}  // namespace

cudaError_t launch_cache_decode(const CacheParams& p, int dtype, cudaStream_t s) {
  const cudaError_t e = dtype == CAPATTN_BF16 ? launch_decode_tc(p, s) : launch_decode_fp32(p, s);
  if (e != cudaSuccess || !p.scores) return e;
  const int live = p.window_len > 0 && !p.pos ? min(p.max_len, p.window_len) : p.max_len;
  const dim3 grid(p.B * p.Hkv, min((live + 511) / 512, 1024));
  return launch_pdl(decode_weights_kernel, grid, dim3(128), 0, s, p);
}

}  // namespace capattn
