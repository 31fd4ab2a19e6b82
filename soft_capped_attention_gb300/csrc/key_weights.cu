// Attention weight that each key of a prompt received (capattn_key_weights):
//   w[b, g, j] = sum over heads h of group g, counted rows i of exp(t_ij - lse_i)
// with t and the masks of the forward; here the fp32 kernel.  One CTA per (b, g, 64 keys) walks the
// group's heads and the query tiles that its key tile's visit map names, so the
// sums need no atomics and keep their order.
#include "cache_internal.h"
#include "cache_math.cuh"

namespace capattn {
namespace {

constexpr int kT = 64;   // keys and queries of a step

// CUDA cores: 256 threads, 4 keys x 4 queries each; rows staged in shared memory.
template <int D, int METHOD>
__global__ void __launch_bounds__(256)
key_weights_simt_kernel(Params p, KeyWeightsParams kw) {
  constexpr int PAD = D + 4;
  extern __shared__ __align__(16) float sm[];
  float* sk = sm;              // [64][PAD]
  float* sq = sm + kT * PAD;   // [64][PAD]
  __shared__ float s_lse[kT], s_temp[kT];
  __shared__ int4 s_row[kT];
  __shared__ float s_sum[16][kT];
  pdl_trigger();
  pdl_wait();
  const int bg = blockIdx.x % (p.B * p.Hkv), g = bg % p.Hkv, b = bg / p.Hkv;
  const int k0 = blockIdx.x / (p.B * p.Hkv) * kT;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;  // keys tx + 16 e, queries ty + 16 f
  int lo = 0, hi = p.L;
  if (kw.rows) {
    lo = kw.rows[2 * b];
    hi = kw.rows[2 * b + 1];
    if (!(lo >= 0 && lo <= hi && hi <= p.L)) {
      if (threadIdx.x == 0) atomicOr(p.status, kStatusBadRowsBit);
      lo = max(lo, 0);
      hi = min(hi, p.L);
    }
  }
  const float* q = static_cast<const float*>(p.q);
  const float* k = static_cast<const float*>(p.k);
  for (int i = threadIdx.x; i < kT * D; i += 256) {
    const int r = i / D, x = i % D;
    sk[r * PAD + x] = k0 + r < p.Lk ? k[(((size_t)b * p.Lk + k0 + r) * p.Hkv + g) * D + x] : 0.f;
  }
  const uint32_t* map = p.kmap + ((size_t)b * p.nk + k0 / p.block_kv) * p.wq;
  float sum[4] = {0.f, 0.f, 0.f, 0.f}, comp[4] = {0.f, 0.f, 0.f, 0.f};  // compensated (Kahan)
  for (int hh = 0; hh < p.G; ++hh) {
    const int h = g * p.G + hh;
    TileIter it(map, p.wq);
    int qt;
    while (it.next(qt)) {
      for (int q0 = qt * p.block_q; q0 < min(p.L, (qt + 1) * p.block_q); q0 += kT) {
        if (q0 >= hi || q0 + kT <= lo) continue;
        __syncthreads();
        for (int i = threadIdx.x; i < kT * D; i += 256) {
          const int r = i / D, x = i % D;
          sq[r * PAD + x] = q0 + r < p.L ? q[(((size_t)b * p.L + q0 + r) * p.Hq + h) * D + x] : 0.f;
        }
        if (threadIdx.x < kT) {
          const int i = q0 + threadIdx.x;
          const bool in = i >= lo && i < hi;
          s_lse[threadIdx.x] = in ? p.lse[((size_t)b * p.Hq + h) * p.L + i] : -INFINITY;
          s_temp[threadIdx.x] = in && p.temp ? p.temp[(size_t)b * p.L + i] : 1.f;
          s_row[threadIdx.x] = in ? p.rowinfo[(size_t)b * p.L + i] : make_int4(0, 0, -1, 0);
        }
        __syncthreads();
        float acc[4][4] = {};
#pragma unroll 4
        for (int x = 0; x < D; x += 4) {
          float4 a[4], c[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            a[e] = *reinterpret_cast<const float4*>(&sk[(tx + 16 * e) * PAD + x]);
            c[e] = *reinterpret_cast<const float4*>(&sq[(ty + 16 * e) * PAD + x]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
#pragma unroll
            for (int f = 0; f < 4; ++f)
              acc[e][f] = fmaf(a[e].x, c[f].x, fmaf(a[e].y, c[f].y, fmaf(a[e].z, c[f].z, fmaf(a[e].w, c[f].w, acc[e][f]))));
        }
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const int4 r = s_row[ty + 16 * f];
          const float lse = s_lse[ty + 16 * f], temp = s_temp[ty + 16 * f];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = k0 + tx + 16 * e;
            const bool live = (j >= r.x && j < r.y) || j == r.z;
            const float t = exact_cap<METHOD>(acc[e][f] * p.sm_scale, kw.cap) * temp;
            part[e] += live ? __expf(t - lse) : 0.f;
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float y = part[e] - comp[e], t = sum[e] + y;
          comp[e] = (t - sum[e]) - y;
          sum[e] = t;
        }
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int e = 0; e < 4; ++e) s_sum[ty][tx + 16 * e] = sum[e];
  __syncthreads();
  if (threadIdx.x < kT && k0 + threadIdx.x < p.Lk) {
    float x = 0.f;
    for (int y = 0; y < 16; ++y) x += s_sum[y][threadIdx.x];
    kw.w[((size_t)b * p.Hkv + g) * kw.w_stride + k0 + threadIdx.x] = x;
  }
}

template <int D, int METHOD>
cudaError_t run_simt(const Params& p, const KeyWeightsParams& kw, cudaStream_t s) {
  auto* k = key_weights_simt_kernel<D, METHOD>;
  static std::atomic<uint64_t> done{0};
  const int smem = 2 * kT * (D + 4) * sizeof(float);
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3((unsigned)p.B * p.Hkv * ((p.Lk + kT - 1) / kT)), dim3(256), smem, s, p, kw);
}

template <int D>
cudaError_t run_cap(const Params& p, const KeyWeightsParams& kw, cudaStream_t s) {
  switch (p.cap.method) {
    case CAPATTN_CAP_TANH: return run_simt<D, CAPATTN_CAP_TANH>(p, kw, s);
    case CAPATTN_CAP_SOFT_SIGN: return run_simt<D, CAPATTN_CAP_SOFT_SIGN>(p, kw, s);
    case CAPATTN_CAP_ALSC: return run_simt<D, CAPATTN_CAP_ALSC>(p, kw, s);
    default: return run_simt<D, CAPATTN_CAP_NONE>(p, kw, s);
  }
}

}  // namespace

cudaError_t launch_key_weights(const Params& p, const KeyWeightsParams& kw, int dtype, cudaStream_t s) {
  if (dtype == CAPATTN_BF16) return launch_key_weights_tc(p, kw, s);
  return p.D == 64 ? run_cap<64>(p, kw, s) : run_cap<128>(p, kw, s);
}

}  // namespace capattn
