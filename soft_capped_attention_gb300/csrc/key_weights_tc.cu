// capattn_key_weights on the 5th-generation tensor cores (bf16).
//
// w_j = sum over heads h of the group and counted rows i of 2^(x_ij),
//   x_ij = temp_i log2(e) cap(sm_scale <q_i, k_j>) - log2(e) lse_i.
// One CTA owns 128 keys of one (batch, KV head): K stays in shared memory, Q tiles
// of the group's heads stream through a ring by TMA, and tcgen05 forms S^T = K
// Q^T (128 keys x 128 queries, two TMEM buffers) with a key per TMEM lane, so that
// the sum over queries is a sum within a thread: no transposition, no atomics.
// Eight warps (two warpgroups of 64 query columns each) read 32 columns at a
// time, cap them, exponentiate and add.
//
// What bounds it: one exp2 per pair on the MUFU pipe (16 a clock and SM, against
// about 26 pairs a clock that the tensor cores deliver at D = 128), then the
// issue slots of the cap's polynomial; there is no second product and nothing is
// stored.  Two CTAs an SM hide each other's waits.  The steps (head x visited
// query tile) of a key tile are cut into equal parts over a cluster of up to 8
// CTAs when there are too few key tiles to fill the SMs; the parts are summed
// through distributed shared memory in rank order.
//
// Sums: 32 columns in fp32, then compensated (Kahan) over the chunks: a prompt of
// 131072 rows adds as exactly as a short one.
#include <cooperative_groups.h>

#include "cache_internal.h"
#include "cache_math.cuh"
#include "tc_common.cuh"
#include "tma_maps.h"

namespace capattn {
namespace {

namespace cg = cooperative_groups;

constexpr int BT = 128;
constexpr int SLAB = 128 * 64 * 2;
constexpr int NSTAGE = 2;
constexpr int NBUF = 2;
constexpr int kThreads = 320;  // TMA warp, MMA warp, 8 elementwise warps
template <int HD>
constexpr int tile_bytes() { return (HD / 64) * SLAB; }
template <int HD>
constexpr int smem_bytes() { return (1 + NSTAGE) * tile_bytes<HD>() + 1024; }

// The visited query tiles of a key tile within [qlo, qhi], in order.
struct MapRow {
  const uint32_t* map;
  int qlo, qhi;  // inclusive
  __device__ __forceinline__ uint32_t word(int w) const {
    uint32_t x = map[w];
    if (w == (qlo >> 5)) x &= 0xFFFFFFFFu << (qlo & 31);
    if (w == (qhi >> 5)) x &= 0xFFFFFFFFu >> (31 - (qhi & 31));
    return x;
  }
  __device__ int count() const {
    int n = 0;
    for (int w = qlo >> 5; w <= (qhi >> 5); ++w) n += __popc(word(w));
    return n;
  }
};

// Steps [s0, s1) of head-major (head, visited tile).
struct Steps {
  MapRow row;
  int hh, w, left;
  uint32_t bits;
  __device__ Steps(const MapRow& r, int ntiles, int s0, int s1) : row(r), left(s1 - s0) {
    hh = ntiles > 0 ? s0 / ntiles : 0;
    int skip = s0 - hh * ntiles;
    w = r.qlo >> 5;
    bits = left > 0 ? r.word(w) : 0u;
    while (left > 0) {
      const int c = __popc(bits);
      if (skip < c) break;
      skip -= c;
      bits = r.word(++w);
    }
    while (skip-- > 0) bits &= bits - 1u;
  }
  __device__ __forceinline__ bool next(int& h, int& qt) {
    if (left <= 0) return false;
    --left;
    while (bits == 0u) {
      if (w >= (row.qhi >> 5)) {
        ++hh;
        w = row.qlo >> 5;
      } else {
        ++w;
      }
      bits = row.word(w);
    }
    h = hh;
    qt = w * 32 + __ffs(bits) - 1;
    bits &= bits - 1u;
    return true;
  }
};

// A query column's inputs, loaded two steps ahead of use.
struct ColRaw {
  float lse, temp;
  int4 span;
  int2 full;  // key tiles that the query tile covers whole
};

template <int METHOD>
__device__ __forceinline__ float chunk_sum(const uint32_t (&x)[32], const float4* cc, const int4* spans, int j,
                                           bool masked, bool poly, const ExactCap& k) {
  F2 acc = f2(0.f, 0.f);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float4 c = cc[e];  // mul, mul', add, add'
    const float X0 = __uint_as_float(x[2 * e]), X1 = __uint_as_float(x[2 * e + 1]);
    F2 f;
    if constexpr (METHOD == CAPATTN_CAP_NONE) {
      f = f2(X0, X1);  // sm_scale is in mul
    } else if constexpr (has_poly(METHOD)) {
      f = poly ? poly_cap2<METHOD>(f2(X0, X1), k) : f2(any_cap<METHOD>(X0, k), any_cap<METHOD>(X1, k));
    } else {
      f = f2(any_cap<METHOD>(X0, k), any_cap<METHOD>(X1, k));
    }
    float a, b;
    f2_split(f2_fma(f2(c.x, c.y), f, f2(c.z, c.w)), a, b);
    a = ex2_approx(a);
    b = ex2_approx(b);
    if (masked) {
      const int4 r0 = spans[2 * e], r1 = spans[2 * e + 1];
      a = (j >= r0.x && j < r0.y) || j == r0.z ? a : 0.f;
      b = (j >= r1.x && j < r1.y) || j == r1.z ? b : 0.f;
    }
    acc = f2_add(acc, f2(a, b));
  }
  float a, b;
  f2_split(acc, a, b);
  return a + b;
}

template <int METHOD, int HD>
__global__ void __launch_bounds__(kThreads, 2)
key_weights_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const Params p,
                      const KeyWeightsParams kw, const int parts) {
  constexpr int TILE = tile_bytes<HD>();
  constexpr int NSLAB = HD / 64;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[1 + 2 * NSTAGE + 2 * NBUF];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ __align__(16) float4 colc[2][BT / 2];
  __shared__ __align__(16) int4 cols[2][BT];
  __shared__ float s_sum[2][BT], s_out[BT];

  const int rank = blockIdx.x % parts, unit = blockIdx.x / parts;
  const int bg = unit % (p.B * p.Hkv), g = bg % p.Hkv, b = bg / p.Hkv;
  const int kt = unit / (p.B * p.Hkv), k0 = kt * BT;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sK = base, sQ = base + TILE;
  const uint32_t bar_k = smem_u32(&bars[0]);
  const uint32_t bar_full = smem_u32(&bars[1]);                        // + 8 s: Q of stage s landed
  const uint32_t bar_empty = smem_u32(&bars[1 + NSTAGE]);              // + 8 s: its MMAs are done
  const uint32_t bar_s = smem_u32(&bars[1 + 2 * NSTAGE]);              // + 8 u: S^T in buffer u
  const uint32_t bar_free = smem_u32(&bars[1 + 2 * NSTAGE + NBUF]);    // + 8 u: buffer u read (8 warps)
  if (threadIdx.x == 0) {
    abort_flag = 0;
    mbar_init(bar_k, 1);
    for (int s = 0; s < NSTAGE; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int u = 0; u < NBUF; ++u) {
      mbar_init(bar_s + 8 * u, 1);
      mbar_init(bar_free + 8 * u, 8);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), NBUF * BT);
    tmem_relinquish();
  }
  pdl_trigger();
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  int lo = 0, hi = p.L;  // counted rows
  if (kw.rows) {
    lo = kw.rows[2 * b];
    hi = kw.rows[2 * b + 1];
    if (!(lo >= 0 && lo <= hi && hi <= p.L)) {
      if (threadIdx.x == 0) atomicOr(p.status, kStatusBadRowsBit);
      lo = max(lo, 0);
      hi = min(hi, p.L);
    }
  }
  MapRow row{p.kmap + ((size_t)b * p.nk + kt) * p.wq, lo / BT, (hi - 1) / BT};
  const int ntiles = lo < hi ? row.count() : 0;
  const int all = ntiles * p.G;
  const int s0 = (int)((int64_t)all * rank / parts), s1 = (int)((int64_t)all * (rank + 1) / parts);
  const int n = s1 - s0;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (n > 0) {
      const bool leader = elect_one_sync();
      if (leader) {
        mbar_expect_tx(bar_k, TILE);
        for (int sl = 0; sl < NSLAB; ++sl) tma_load_4d(sK + sl * SLAB, &mk, bar_k, 64 * sl, g, k0, b);
      }
      __syncwarp();
      Steps st(row, ntiles, s0, s1);
      int hh, qt, j = 0;
      while (st.next(hh, qt)) {
        const int s = j % NSTAGE, u = j / NSTAGE;
        if (u > 0 && !mbar_wait_warp(bar_empty + 8 * s, (u - 1) & 1, p.status, &abort_flag)) break;
        if (leader) {
          mbar_expect_tx(bar_full + 8 * s, TILE);
          for (int sl = 0; sl < NSLAB; ++sl)
            tma_load_4d(sQ + s * TILE + sl * SLAB, &mq, bar_full + 8 * s, 64 * sl, g * p.G + hh, qt * BT, b);
        }
        __syncwarp();
        ++j;
      }
      if (leader) {
        drain_wait(bar_k, 0);
        for (int x = (j > NSTAGE ? j - NSTAGE : 0); x < j; ++x) drain_wait(bar_full + 8 * (x % NSTAGE), (x / NSTAGE) & 1);
      }
      __syncwarp();
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (n > 0) {
      const bool leader = elect_one_sync();
      constexpr uint32_t idesc = idesc_bf16(BT, BT, 0, 0);
      const uint64_t dK = smem_desc(sK, 16, 1024), dQ = smem_desc(sQ, 16, 1024);
      bool ok = mbar_wait_warp(bar_k, 0, p.status, &abort_flag);
      int j = 0;
      for (; ok && j < n; ++j) {
        const int s = j % NSTAGE, u = j % NBUF, r = j / NBUF;
        if (r > 0) ok = mbar_wait_warp(bar_free + 8 * u, (r - 1) & 1, p.status, &abort_flag);
        ok = ok && mbar_wait_warp(bar_full + 8 * s, (j / NSTAGE) & 1, p.status, &abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < HD / 16; ++ks) {
            const uint32_t off = (ks >> 2) * SLAB + (ks & 3) * 32;
            mma_ss(tmem + u * BT, desc_add(dK, off), desc_add(dQ, s * TILE + off), idesc, ks > 0 ? 1u : 0u);
          }
          mma_commit(bar_empty + 8 * s);
          mma_commit(bar_s + 8 * u);
        }
        __syncwarp();
      }
      // every MMA has completed before TMEM is freed
      if (leader)
        for (int x = (j > NBUF ? j - NBUF : 0); x < j; ++x) mbar_poll(bar_s + 8 * (x % NBUF), (x / NBUF) & 1);
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ elementwise
    const int wg = (warp - 2) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;                   // key of the tile
    const int tid = (warp - 2 - 4 * wg) * 32 + lane;     // within the warpgroup
    const int j = k0 + r;
    const uint32_t cols_t = tmem + ((uint32_t)(quarter * 32) << 16) + 64u * wg;
    const int my_col = 64 * wg + tid;                    // the column whose constants this thread writes (tid < 64)
    Steps nx(row, ntiles, s0, s1);
    auto load = [&](bool have, int hh, int qt) {
      ColRaw c;
      c.lse = -INFINITY;
      c.temp = 1.f;
      c.span = make_int4(0, 0, -1, 0);
      c.full = make_int2(0, 0);
      if (!have) return c;
      // whole: the tile's rows are all counted
      if (qt * BT >= lo && (qt + 1) * BT <= hi) c.full = p.qfull[(size_t)b * p.nq + qt];
      const int i = qt * BT + my_col;
      if (tid < 64 && i >= lo && i < hi) {
        c.lse = p.lse[((size_t)b * p.Hq + g * p.G + hh) * p.L + i];
        if (p.temp) c.temp = p.temp[(size_t)b * p.L + i];
        c.span = p.rowinfo[(size_t)b * p.L + i];
      }
      return c;
    };
    auto put = [&](int buf, const ColRaw& c) {
      if (tid < 64) {
        float* f = reinterpret_cast<float*>(&colc[buf][my_col >> 1]) + (my_col & 1);
        f[0] = c.temp * kL2E * (METHOD == CAPATTN_CAP_NONE ? p.sm_scale : 1.f);
        f[2] = c.lse == -INFINITY ? 0.f : -c.lse * kL2E;
        cols[buf][my_col] = c.span;
      }
    };
    int hh, qt;
    bool have = nx.next(hh, qt);
    ColRaw cur = load(have, hh, qt);
    have = nx.next(hh, qt);
    ColRaw nxt = load(have, hh, qt);
    float sum = 0.f, comp = 0.f;
    put(0, cur);
    bool ok = true;
    for (int step = 0; step < n; ++step) {
      const int cb = step & 1, u = step % NBUF;
      named_bar_sync(1 + wg, 128);  // this step's constants are written, the last step's read
      if (step + 1 < n) put(cb ^ 1, nxt);
      have = nx.next(hh, qt);
      const ColRaw far = load(have, hh, qt);
      const bool masked = !(kt >= cur.full.x && kt < cur.full.y);
      ok = ok && mbar_wait_warp(bar_s + 8 * u, (step / NBUF) & 1, p.status, &abort_flag);
      if (ok) {
        tc_fence_after();
        uint32_t x[2][32];
        tmem_ld32(cols_t + u * BT, x[0]);
        tmem_ld32(cols_t + u * BT + 32, x[1]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_free + 8 * u);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          bool poly = false;
          if constexpr (has_poly(METHOD)) {
            float am = 0.f;
#pragma unroll
            for (int e = 0; e < 32; e += 2) am = fmax3_abs(am, __uint_as_float(x[c][e]), __uint_as_float(x[c][e + 1]));
            poly = __all_sync(0xFFFFFFFFu, am <= kw.cap.xmax && kw.cap.xmax > 0.f);
          }
          const float4* cc = &colc[cb][32 * wg + 16 * c];
          const int4* sp = &cols[cb][64 * wg + 32 * c];
          float part;
          if (masked)
            part = poly ? chunk_sum<METHOD>(x[c], cc, sp, j, true, true, kw.cap)
                        : chunk_sum<METHOD>(x[c], cc, sp, j, true, false, kw.cap);
          else
            part = poly ? chunk_sum<METHOD>(x[c], cc, sp, j, false, true, kw.cap)
                        : chunk_sum<METHOD>(x[c], cc, sp, j, false, false, kw.cap);
          const float y = part - comp, t = sum + y;
          comp = (t - sum) - y;
          sum = t;
        }
      }
      cur = nxt;
      nxt = far;
    }
    s_sum[wg][r] = sum;
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, NBUF * BT);
  }
  if (threadIdx.x < BT) s_out[threadIdx.x] = s_sum[0][threadIdx.x] + s_sum[1][threadIdx.x];
  float* w = kw.w + ((size_t)b * p.Hkv + g) * kw.w_stride + k0;
  if (parts == 1) {
    if (threadIdx.x < BT && k0 + (int)threadIdx.x < p.Lk) w[threadIdx.x] = s_out[threadIdx.x];
    return;
  }
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();
  if (rank == 0 && threadIdx.x < BT && k0 + (int)threadIdx.x < p.Lk) {
    float x = 0.f;
    for (int c = 0; c < parts; ++c) x += cluster.map_shared_rank(s_out, c)[threadIdx.x];
    w[threadIdx.x] = x;
  }
  cluster.sync();  // no CTA leaves while its sums may be read
}

template <int METHOD, int HD>
cudaError_t run(const Params& p, const KeyWeightsParams& kw, cudaStream_t s) {
  auto* k = key_weights_tc_kernel<METHOD, HD>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem_bytes<HD>(), done);
  CUtensorMap mq, mk;
  if (e == cudaSuccess) e = make_bhld_map(&mq, p.q, p.B, p.L, p.Hq, HD, BT);
  if (e == cudaSuccess) e = make_bhld_map(&mk, p.k, p.B, p.Lk, p.Hkv, HD, BT);
  if (e != cudaSuccess) return e;
  // Parts of a key tile's steps: until two CTAs an SM have several turns each.
  const int64_t units = (int64_t)p.B * p.Hkv * p.nk;
  int parts = 1;
  while (parts < 8 && units * parts < 152 * 2 * 4 && parts * 2 <= p.G * p.nq) parts *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * parts));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem_bytes<HD>();
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = parts;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k, mq, mk, p, kw, parts);
}

template <int HD>
cudaError_t run_cap(const Params& p, const KeyWeightsParams& kw, cudaStream_t s) {
  switch (p.cap.method) {
    case CAPATTN_CAP_TANH: return run<CAPATTN_CAP_TANH, HD>(p, kw, s);
    case CAPATTN_CAP_SOFT_SIGN: return run<CAPATTN_CAP_SOFT_SIGN, HD>(p, kw, s);
    case CAPATTN_CAP_ALSC: return run<CAPATTN_CAP_ALSC, HD>(p, kw, s);
    default: return run<CAPATTN_CAP_NONE, HD>(p, kw, s);
  }
}

}  // namespace

cudaError_t launch_key_weights_tc(const Params& p, const KeyWeightsParams& kw, cudaStream_t s) {
  return p.D == 64 ? run_cap<64>(p, kw, s) : run_cap<128>(p, kw, s);
}

}  // namespace capattn
