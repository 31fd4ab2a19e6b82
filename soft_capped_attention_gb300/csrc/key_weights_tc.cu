// capattn_key_weights on the 5th-generation tensor cores (bf16).
//
// w_j = sum over heads h of the group and counted rows i of 2^(x_ij),
//   x_ij = temp_i log2(e) cap(sm_scale <q_i, k_j>) - log2(e) lse_i.
// A unit is 128 keys of one (batch, KV head), a step one query tile of one of the
// group's heads that the keys' visit map names.  A persistent grid, one CTA an SM,
// takes equal shares of all steps (as decode does of its tiles, cache_sched.cuh):
// K stays in shared memory for a unit (two buffers), Q tiles stream through a ring
// by TMA, and tcgen05 forms S^T = K Q^T (128 keys x 128 queries, four TMEM buffers)
// with a key per TMEM lane, so that the sum over queries is a sum within a thread:
// no transposition, no atomics.  Sixteen warps read it, cap, exponentiate and add:
// four warpgroups, two for the even steps and two for the odd ones, 64 query columns
// each.  A unit that two CTAs share leaves
// partial sums, which the last of them adds in order.
//
// What bounds it: the elementwise pass.  There is no second product and nothing is
// stored; the tensor cores need 260 cycles for a step of 128 x 128 pairs, the exp2s
// 512 on the MUFU pipe (32 a clock and SM), the cap's polynomial and the sums 640
// (tanh near zero; 5 products a pair at 128 a clock) to 1150 (alsc with
// temperatures).  Measured are about 1400 cycles a step on a long prompt (8192 rows,
// 32 heads, tanh: 322 us, 854 TFLOP/s at 2 D a live pair), with about half of the issue
// slots used (the elementwise warps wait for tensor memory and for one another at a
// piece's end), and about 12 us of launches and first loads (two prompts of 2048 x 16
// heads: 32.6 us in all; 4096 rows x 32 heads in a window of 1024 with alsc and
// temperatures: 72.3 us; 32.1 and 70.3 with inputs in L2, as in what follows).
//   Tried: the steps of a key tile cut over clusters of up to 8 CTAs instead of the
// persistent shares (58 us for the two prompts: two steps a CTA, mostly prologue);
// constants loaded by the TMA warp (40 us: the MMAs waited for it); one step for all
// sixteen warps, 32 columns each (38 -> 40 us: the waits are paid per 32 columns);
// 16-column chunks (41 us); both chunks of a step unrolled (42 us: more code than the
// instruction caches like); a piece's sums written by the TMA warp between its loads
// (37.5 us against 32.1).
//
// Sums: 32 columns in fp32, then compensated (Kahan) over those: a prompt of
// 131072 rows adds as exactly as a short one.
#include <limits.h>

#include "cache_internal.h"
#include "cache_math.cuh"
#include "tc_common.cuh"
#include "tma_maps.h"

namespace capattn {
namespace {

constexpr int BT = 128;
constexpr int SLAB = 128 * 64 * 2;
constexpr int NSTAGE = 4;              // Q tiles in flight
constexpr int NBUF = 4;                // S^T buffers
constexpr int NK = 2;                  // K buffers
constexpr int kElem = 16;              // elementwise warps
constexpr int kConst = 2;              // warps that load the columns' constants, 64 columns each
constexpr int kThreads = 64 + 32 * (kElem + kConst);
template <int HD>
constexpr int tile_bytes() { return (HD / 64) * SLAB; }
template <int HD>
constexpr int smem_bytes() { return (NK + NSTAGE) * tile_bytes<HD>() + 1024; }

// Key-tile map (the transpose of the query-tile map, counted rows only) and the
// steps of each (batch, key tile): a warp each.  The first one clears the counters.
__global__ void __launch_bounds__(128)
key_plan_kernel(Params p, KeyWeightsParams kw) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t e = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < kWeightCtas; i += 128) kw.counters[i] = 0u;
  if (e >= (int64_t)p.B * p.nk) return;
  const int b = (int)(e / p.nk), kt = (int)(e % p.nk);
  int lo = 0, hi = p.L;
  if (kw.rows) {
    lo = kw.rows[2 * b];
    hi = kw.rows[2 * b + 1];
    if (!(lo >= 0 && lo <= hi && hi <= p.L)) {
      if (lane == 0 && kt == 0) atomicOr(p.status, kStatusBadRowsBit);
      lo = max(lo, 0);
      hi = min(hi, p.L);
    }
  }
  int count = 0;
  for (int w = 0; w < p.wq; ++w) {
    const int qt = 32 * w + lane;
    bool on = qt < p.nq && qt * BT < hi && (qt + 1) * BT > lo && lo < hi;
    if (on) on = (p.qmap[((size_t)b * p.nq + qt) * p.wk + (kt >> 5)] >> (kt & 31)) & 1u;
    const uint32_t word = __ballot_sync(0xFFFFFFFFu, on);
    if (lane == 0) p.kmap[(size_t)e * p.wq + w] = word;
    count += __popc(word);
  }
  if (lane == 0) kw.steps[e] = count * p.G;
}

// The units' steps, shared out: CTA c of n takes steps [U c / n, U (c + 1) / n) of
// all U, numbered by (batch, key tile), KV head, step.  A unit counts kUnitCost steps
// more than it has (its first ones), about what starting and ending it costs: the
// last key tiles of a causal prompt have one step a head (two prompts of 2048: 37 us
// with 1, 39 with 2, 40 with 4).  At least 1: a unit without steps has zeros to write.
constexpr int kUnitCost = 1;
static_assert(kUnitCost >= 1, "every unit has to belong to a CTA");
struct Share {
  uint64_t total;
  uint32_t ctas;
  __device__ __forceinline__ uint64_t begin_of(uint32_t c) const { return c >= ctas ? total : total * c / ctas; }
  __device__ __forceinline__ int cta_of(uint64_t x) const { return (int)(((x + 1) * ctas - 1) / total); }
};

struct Start {  // where a CTA's range begins
  uint64_t total, before;  // all steps; those before entry e
  int e;
};

// Walks a CTA's pieces (warp-uniform).
struct PieceWalk {
  Share sh;
  uint64_t u, end, begin;
  int e, g, t0;
  // of the piece that next() gave
  int n;        // its steps (maybe none)
  int first;    // the first of them within the unit
  bool whole;
  int slot;
  uint64_t s0, s1;

  __device__ PieceWalk(const Params& p, const KeyWeightsParams& kw, const Start& st) {
    sh.total = st.total;
    sh.ctas = (uint32_t)min((uint64_t)gridDim.x, st.total);
    begin = u = sh.begin_of(blockIdx.x);
    end = sh.begin_of(blockIdx.x + 1);
    e = st.e;
    g = t0 = 0;
    if (u >= end) return;
    const uint32_t m = (uint32_t)(kw.steps[e] + kUnitCost);
    const uint64_t in = u - st.before;
    g = (int)(in / m);
    t0 = (int)(in % m);
  }
  __device__ bool next(const Params& p, const KeyWeightsParams& kw, int* e_out, int* g_out) {
    if (u >= end) return false;
    const int m = kw.steps[e] + kUnitCost;
    const int take = (int)min((uint64_t)(m - t0), end - u);
    first = max(0, t0 - kUnitCost);
    n = max(0, t0 + take - kUnitCost) - first;
    whole = t0 == 0 && take == m;
    slot = 2 * (int)blockIdx.x + (u == begin ? 0 : 1);
    s0 = u - (uint64_t)t0;
    s1 = s0 + (uint64_t)m;
    *e_out = e;
    *g_out = g;
    u += (uint64_t)take;
    t0 = 0;
    if (++g == p.Hkv) {
      g = 0;
      ++e;
    }
    return true;
  }
};

// Steps [first, first + n) of a unit, head-major: (head, visited tile).
struct Steps {
  const uint32_t* map;
  int words, hh, w, left;
  uint32_t bits;
  __device__ Steps(const uint32_t* m, int wq, int per_head, int first, int n) : map(m), words(wq), left(n) {
    hh = n > 0 ? first / per_head : 0;
    int skip = first - hh * per_head;
    w = 0;
    bits = n > 0 ? map[0] : 0u;
    while (left > 0) {
      const int c = __popc(bits);
      if (skip < c) break;
      skip -= c;
      bits = map[++w];
    }
    while (left > 0 && skip-- > 0) bits &= bits - 1u;
  }
  __device__ __forceinline__ bool next(int& h, int& qt) {
    if (left <= 0) return false;
    --left;
    while (bits == 0u) {
      if (++w == words) {
        ++hh;
        w = 0;
      }
      bits = map[w];
    }
    h = hh;
    qt = w * 32 + __ffs(bits) - 1;
    bits &= bits - 1u;
    return true;
  }
};

constexpr int NCONST = NBUF;  // column constants go with the S^T buffers
constexpr int kAhead = 2;     // steps by which their inputs are asked for ahead

// Asynchronous copies of 4, 8 and 16 bytes into shared memory; zeros where !in.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool in) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES), "r"(in ? BYTES : 0)
               : "memory");
}

// Per-method constants of the log2-domain logit:
//   x = log2(e) temp cap(sm_scale X) - log2(e) lse = (temp X) Q(X) + add
// with Q the cap's polynomial times log2(e) (in z = X^2 for tanh, in X for alsc;
// the constant sm_scale log2(e) without a cap).  tanh has one of three terms for
// scores near zero, kept in registers (two products a pair less: 34.4 us for the two
// prompts against 36.8), and one of five.
template <int METHOD, bool WIDE>
struct Poly {
  static constexpr int N = METHOD == CAPATTN_CAP_TANH ? (WIDE ? 5 : 3) : METHOD == CAPATTN_CAP_ALSC ? 7 : 1;
  F2 c[N];
  __device__ __forceinline__ explicit Poly(const ExactCap& k) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float x = 1.f;
      if (METHOD == CAPATTN_CAP_NONE) x = k.sm_scale;
      else if (METHOD == CAPATTN_CAP_TANH && !WIDE) x = k.near.c[i];
      else if (has_poly(METHOD)) x = k.poly[i];
      c[i] = f2(x * kL2E, x * kL2E);
    }
  }
  __device__ __forceinline__ F2 eval(F2 X) const {
    const F2 z = METHOD == CAPATTN_CAP_TANH ? f2_mul(X, X) : X;
    F2 q = c[N - 1];
#pragma unroll
    for (int i = N - 2; i >= 0; --i) q = f2_fma(q, z, c[i]);
    return q;
  }
};
// How a chunk's scores are capped: by the polynomial in registers, by tanh's longer
// one, one by one.
enum { kNear, kWide, kOneByOne };

// Sum of 2^x over 32 query columns of this thread's key.  LEVEL: every raw score of
// the warp is in that polynomial's range (or the cap has none to leave).
// MASK: 0 every pair is live; 1 a column's live keys are [lo, lo + len); 2 and one more.
template <int METHOD, bool TEMP, int MASK, int LEVEL, class P>
__device__ __forceinline__ float chunk_sum(const uint32_t (&x)[32], const float* add, const float* temp,
                                           const int2* spans, const int* extra, int j, const P& poly, const ExactCap& k) {
  F2 acc = f2(0.f, 0.f);
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    const float4 ad = *reinterpret_cast<const float4*>(add + e);
    float4 tp = make_float4(1.f, 1.f, 1.f, 1.f);
    if (TEMP) tp = *reinterpret_cast<const float4*>(temp + e);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float X0 = __uint_as_float(x[e + 2 * h]), X1 = __uint_as_float(x[e + 2 * h + 1]);
      const F2 a2 = h == 0 ? f2(ad.x, ad.y) : f2(ad.z, ad.w), t2 = h == 0 ? f2(tp.x, tp.y) : f2(tp.z, tp.w);
      F2 y;
      if constexpr (LEVEL != kOneByOne && METHOD != CAPATTN_CAP_SOFT_SIGN) {
        const F2 X = f2(X0, X1);
        y = f2_fma(TEMP ? f2_mul(X, t2) : X, poly.eval(X), a2);
      } else {
        F2 t = f2_mul(f2(any_cap<METHOD>(X0, k), any_cap<METHOD>(X1, k)), f2(kL2E, kL2E));
        y = TEMP ? f2_fma(t, t2, a2) : f2_add(t, a2);
      }
      float a, b;
      f2_split(y, a, b);
      a = ex2_approx(a);
      b = ex2_approx(b);
      if (MASK > 0) {
        const int4 r = *reinterpret_cast<const int4*>(spans + e + 2 * h);  // (lo, len) of two columns
        bool la = (uint32_t)(j - r.x) < (uint32_t)r.y, lb = (uint32_t)(j - r.z) < (uint32_t)r.w;
        if (MASK > 1) {
          la = la || j == extra[e + 2 * h];
          lb = lb || j == extra[e + 2 * h + 1];
        }
        a = la ? a : 0.f;
        b = lb ? b : 0.f;
      }
      acc = f2_add(acc, f2(a, b));
    }
  }
  float a, b;
  f2_split(acc, a, b);
  return a + b;
}

template <int METHOD, int HD, bool TEMP>
__global__ void __launch_bounds__(kThreads, 1)
key_weights_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const Params p,
                      const KeyWeightsParams kw) {
  constexpr int TILE = tile_bytes<HD>();
  constexpr int NSLAB = HD / 64;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * (NK + NSTAGE + NBUF)];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag, join_flag;
  __shared__ __align__(16) float col_add[NCONST][BT], col_temp[TEMP ? NCONST : 1][BT];
  __shared__ __align__(16) int2 col_span[NCONST][BT];
  __shared__ int col_extra[NCONST][BT];
  // (least and largest lo, least and largest hi) over the live spans of 32 columns;
  // a column without live keys makes the largest lo and the least hi impossible
  __shared__ __align__(16) int4 col_range[NCONST][BT / 32];
  __shared__ int col_masked[NCONST];  // whether any pair of the step is dead
  // the constants' inputs on their way
  __shared__ __align__(16) int4 raw_span[kAhead + 1][BT];
  __shared__ float raw_lse[kAhead + 1][BT], raw_temp[TEMP ? kAhead + 1 : 1][BT];
  __shared__ __align__(8) int2 raw_full[kAhead + 1][kConst];
  __shared__ float s_sum[2][kElem / 4][BT];
  __shared__ Start s_start;
  __shared__ uint64_t s_scan[kThreads / 32];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sK = base, sQ = base + NK * TILE;
  const uint32_t bar_kfull = smem_u32(&bars[0]);          // + 8 x: K of buffer x landed
  const uint32_t bar_kempty = bar_kfull + 8 * NK;         // + 8 x: its unit's MMAs are done
  const uint32_t bar_full = bar_kempty + 8 * NK;          // + 8 s: Q of stage s landed
  const uint32_t bar_empty = bar_full + 8 * NSTAGE;       // + 8 s: its MMAs are done
  const uint32_t bar_s = bar_empty + 8 * NSTAGE;          // + 8 u: S^T and constants in buffer u (commit, constants' lanes)
  const uint32_t bar_free = bar_s + 8 * NBUF;             // + 8 u: buffer u read (elementwise warps)
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int x = 0; x < NK; ++x) {
      mbar_init(bar_kfull + 8 * x, 1);
      mbar_init(bar_kempty + 8 * x, 1);
    }
    for (int s = 0; s < NSTAGE; ++s) {
      mbar_init(bar_full + 8 * s, 1);
      mbar_init(bar_empty + 8 * s, 1);
    }
    for (int u = 0; u < NBUF; ++u) {
      mbar_init(bar_s + 8 * u, 1 + 32 * kConst);
      mbar_init(bar_free + 8 * u, kElem / 2);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), NBUF * BT);
    tmem_relinquish();
  }
  pdl_trigger();
  pdl_wait();
  // all steps, and the entry where this CTA's range begins: a thread takes a run of
  // entries
  {
    const int64_t E = (int64_t)p.B * p.nk;
    const int64_t run = (E + kThreads - 1) / kThreads;
    const int64_t e0 = min(E, run * (int64_t)threadIdx.x), e1 = min(E, e0 + run);
    uint64_t mine = 0;
    for (int64_t e = e0; e < e1; ++e) mine += (uint64_t)(kw.steps[e] + kUnitCost) * p.Hkv;
    uint64_t up = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint64_t y = __shfl_up_sync(0xFFFFFFFFu, up, d);
      if (lane >= d) up += y;
    }
    if (lane == 31) s_scan[warp] = up;
    __syncthreads();
    uint64_t before = up - mine, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += s_scan[w];
      total += s_scan[w];
    }
    Share sh;
    sh.total = total;
    sh.ctas = (uint32_t)min((uint64_t)gridDim.x, total);
    const uint64_t begin = sh.begin_of(blockIdx.x);
    if (threadIdx.x == 0) s_start.total = total;
    if (begin >= before && begin < before + mine) {
      for (int64_t e = e0; e < e1; ++e) {
        const uint64_t m = (uint64_t)(kw.steps[e] + kUnitCost) * p.Hkv;
        if (begin < before + m) {
          s_start.e = (int)e;
          s_start.before = before;
          break;
        }
        before += m;
      }
    } else if (begin >= total && threadIdx.x == 0) {  // an empty range
      s_start.e = 0;
      s_start.before = 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  PieceWalk it(p, kw, s_start);
  int e, g;
  uint32_t step = 0, unit = 0;  // steps and units with steps so far

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    const bool leader = elect_one_sync();
    bool ok = true;
    while (ok && it.next(p, kw, &e, &g)) {
      if (it.n == 0) continue;
      const int b = e / p.nk, kt = e % p.nk;
      const int x = unit % NK, ux = unit / NK;
      if (ux > 0 && !mbar_wait_warp(bar_kempty + 8 * x, (ux - 1) & 1, p.status, &abort_flag)) break;
      if (leader) {
        mbar_expect_tx(bar_kfull + 8 * x, TILE);
        for (int sl = 0; sl < NSLAB; ++sl)
          tma_load_4d(sK + x * TILE + sl * SLAB, &mk, bar_kfull + 8 * x, 64 * sl, g, kt * BT, b);
      }
      __syncwarp();
      ++unit;
      Steps st(p.kmap + (size_t)e * p.wq, p.wq, kw.steps[e] / p.G, it.first, it.n);
      int hh, qt;
      while (st.next(hh, qt)) {
        const int s = step % NSTAGE, us = step / NSTAGE;
        if (us > 0 && !mbar_wait_warp(bar_empty + 8 * s, (us - 1) & 1, p.status, &abort_flag)) {
          ok = false;
          break;
        }
        if (leader) {
          mbar_expect_tx(bar_full + 8 * s, TILE);
          for (int sl = 0; sl < NSLAB; ++sl)
            tma_load_4d(sQ + s * TILE + sl * SLAB, &mq, bar_full + 8 * s, 64 * sl, g * p.G + hh, qt * BT, b);
        }
        __syncwarp();
        ++step;
      }
    }
    if (leader) {
      for (uint32_t x = unit > NK ? unit - NK : 0; x < unit; ++x) drain_wait(bar_kfull + 8 * (x % NK), (x / NK) & 1);
      for (uint32_t x = step > NSTAGE ? step - NSTAGE : 0; x < step; ++x)
        drain_wait(bar_full + 8 * (x % NSTAGE), (x / NSTAGE) & 1);
    }
    __syncwarp();
  } else if (warp >= 2 + kElem) {
    // ------------------------------------------------------------ column constants
    // Each lane copies its columns' inputs into shared memory two steps ahead and takes
    // them from there itself.  (Loads into registers that the loop hands on were waited
    // for in every step: 352 us for 8192 rows against 324.)
    const int part = warp - 2 - kElem, c0 = 64 * part + lane;  // and c0 + 32
    bool ok = true;
    while (ok && it.next(p, kw, &e, &g)) {
      if (it.n == 0) continue;
      const int b = e / p.nk, kt = e % p.nk;
      const int lo = kw.rows ? max(kw.rows[2 * b], 0) : 0, hi = kw.rows ? min(kw.rows[2 * b + 1], p.L) : p.L;
      Steps st(p.kmap + (size_t)e * p.wq, p.wq, kw.steps[e] / p.G, it.first, it.n);
      const float* lse = p.lse + ((size_t)b * p.Hq + g * p.G) * p.L;
      const float* temp = TEMP ? p.temp + (size_t)b * p.L : nullptr;
      const int4* spans = p.rowinfo + (size_t)b * p.L;
      const int2* full = p.qfull + (size_t)b * p.nq;
      int tiles[kAhead + 1];  // query tiles of the steps on their way
      int to = 0;
      auto ask = [&] {  // for the next step's inputs, if there is one
        int hh = 0, qt = 0;
        if (st.next(hh, qt)) {
          if (lane == 0) copy_async<8>(&raw_full[to][part], full + qt, true);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int col = c0 + 32 * y, i = qt * BT + col;
            const bool in = i < p.L;
            const int row = in ? i : 0;
            copy_async<4>(&raw_lse[to][col], lse + (size_t)hh * p.L + row, in);
            if (TEMP) copy_async<4>(&raw_temp[to][col], temp + row, in);
            copy_async<16>(&raw_span[to][col], spans + row, in);
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        to = to == kAhead ? 0 : to + 1;
        return qt;
      };
      tiles[0] = ask();
      tiles[1] = ask();
      int from = 0;
      for (int i = 0; i < it.n; ++i) {
        tiles[2] = ask();
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
        __syncwarp();  // lane 0's copy too
        const int2 f = raw_full[from][part];
        const int q0 = tiles[0] * BT;
        const int c = step % NCONST, uc = step / NCONST;
        if (uc > 0 && !mbar_wait_warp(bar_free + 8 * c, (uc - 1) & 1, p.status, &abort_flag)) {
          ok = false;
          break;
        }
        // whole: every pair of the step is live
        const bool step_masked = !(q0 >= lo && q0 + BT <= hi && kt >= f.x && kt < f.y);
        if (c0 == 0) col_masked[c] = step_masked;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int col = c0 + 32 * y;
          const float l = raw_lse[from][col];
          col_add[c][col] = l == -INFINITY ? 0.f : -l * kL2E;
          if (TEMP) col_temp[c][col] = raw_temp[from][col];
        }
        if (step_masked) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int col = c0 + 32 * y;
            int4 span = raw_span[from][col];
            if (q0 + col < lo || q0 + col >= hi) span = make_int4(0, 0, -1, 0);
            col_span[c][col] = make_int2(span.x, span.y - span.x);
            if (p.bounds) col_extra[c][col] = span.z;
            const bool some = span.y > span.x;
            int4 range;
            range.x = __reduce_min_sync(0xFFFFFFFFu, some ? span.x : INT_MAX);
            range.y = __reduce_max_sync(0xFFFFFFFFu, some ? span.x : INT_MAX);
            range.z = __reduce_min_sync(0xFFFFFFFFu, some ? span.y : INT_MIN);
            range.w = __reduce_max_sync(0xFFFFFFFFu, some ? span.y : INT_MIN);
            if (lane == 0) col_range[c][col >> 5] = range;
          }
        }
        mbar_arrive(bar_s + 8 * c);
        ++step;
        tiles[0] = tiles[1];
        tiles[1] = tiles[2];
        from = from == kAhead ? 0 : from + 1;
        __syncwarp();  // raw_full is read
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();  // the rings are free for the next piece
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const bool leader = elect_one_sync();
    constexpr uint32_t idesc = idesc_bf16(BT, BT, 0, 0);
    const uint64_t dK = smem_desc(sK, 16, 1024), dQ = smem_desc(sQ, 16, 1024);
    bool ok = true;
    while (ok && it.next(p, kw, &e, &g)) {
      if (it.n == 0) continue;
      const int x = unit % NK;
      ok = mbar_wait_warp(bar_kfull + 8 * x, (unit / NK) & 1, p.status, &abort_flag);
      for (int i = 0; ok && i < it.n; ++i) {
        const int s = step % NSTAGE, u = step % NBUF, r = step / NBUF;
        if (r > 0) ok = mbar_wait_warp(bar_free + 8 * u, (r - 1) & 1, p.status, &abort_flag);
        ok = ok && mbar_wait_warp(bar_full + 8 * s, (step / NSTAGE) & 1, p.status, &abort_flag);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < HD / 16; ++ks) {
            const uint32_t off = (ks >> 2) * SLAB + (ks & 3) * 32;
            mma_ss(tmem + u * BT, desc_add(dK, x * TILE + off), desc_add(dQ, s * TILE + off), idesc, ks > 0 ? 1u : 0u);
          }
          mma_commit(bar_empty + 8 * s);
          mma_commit(bar_s + 8 * u);
          if (i == it.n - 1) mma_commit(bar_kempty + 8 * x);
        }
        __syncwarp();
        ++step;
      }
      ++unit;
    }
    // every MMA has completed before TMEM is freed
    if (leader)
      for (uint32_t x = step > NSTAGE ? step - NSTAGE : 0; x < step; ++x)
        mbar_poll(bar_empty + 8 * (x % NSTAGE), (x / NSTAGE) & 1);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ elementwise
    const int wg = (warp - 2) >> 2, quarter = warp & 3;
    const int r = quarter * 32 + lane;                   // key of the tile
    const uint32_t mine = wg >> 1;                       // the steps it takes: even or odd ones
    const int half = 64 * (wg & 1);                      // its columns of them
    const uint32_t cols_t = tmem + ((uint32_t)(quarter * 32) << 16) + half;
    const Poly<METHOD, false> near(kw.cap);
    int parity = 0;
    bool ok = true;  // after a timeout the warp still meets the others at every unit's barriers
    while (it.next(p, kw, &e, &g)) {
      const int b = e / p.nk, k0 = (e % p.nk) * BT, j = k0 + r;
      float sum = 0.f, comp = 0.f;
      const uint32_t end = step + it.n;
      for (step += (step & 1) ^ mine; step < end; step += 2) {
        const int u = step % NBUF;
        ok = ok && mbar_wait_warp(bar_s + 8 * u, (step / NBUF) & 1, p.status, &abort_flag);
        if (!ok) break;
        tc_fence_after();
        const bool step_masked = col_masked[u] != 0;
#pragma unroll 1
        for (int c = 0; c < 64; c += 32) {
          bool masked = step_masked;
          if (step_masked) {
            // this warp's keys [j - lane, j - lane + 32) against the columns' spans: all
            // live, none (skipped), or a test a pair
            const int4 range = col_range[u][(half + c) >> 5];
            const int first = j - lane;
            if (!p.bounds && (first + 31 < range.x || first >= range.w)) continue;
            masked = first < range.y || first + 32 > range.z;
          }
          uint32_t x[32];
          int level = kNear;
          if constexpr (!has_poly(METHOD)) {
            tmem_ld32(cols_t + u * BT + c, x);
            tmem_wait_ld();
          } else {
            float am = tmem_ld32_absmax(cols_t + u * BT + c, x);
            asm volatile("tcgen05.wait::ld.sync.aligned;" : "+f"(am)::"memory");
            const bool wide = __all_sync(0xFFFFFFFFu, am <= kw.cap.xmax && kw.cap.xmax > 0.f);
            if constexpr (METHOD == CAPATTN_CAP_TANH) {
              const bool close = __all_sync(0xFFFFFFFFu, am <= kw.cap.near.xmax && kw.cap.near.xmax > 0.f);
              level = close ? kNear : wide ? kWide : kOneByOne;
            } else {
              level = wide ? kNear : kOneByOne;
            }
          }
          const float* ad = &col_add[u][half + c];
          const float* tp = &col_temp[TEMP ? u : 0][half + c];
          const int2* sp = &col_span[u][half + c];
          const int* ex = &col_extra[u][half + c];
          float part;
#define CAPATTN_CHUNK(MASK)                                                                              \
  if (level == kNear) {                                                                                  \
    part = chunk_sum<METHOD, TEMP, MASK, kNear>(x, ad, tp, sp, ex, j, near, kw.cap);                     \
  } else if (METHOD == CAPATTN_CAP_TANH && level == kWide) {                                             \
    const Poly<METHOD, true> wide(kw.cap);                                                               \
    part = chunk_sum<METHOD, TEMP, MASK, METHOD == CAPATTN_CAP_TANH ? kWide : kNear>(x, ad, tp, sp, ex, j, wide, kw.cap); \
  } else {                                                                                               \
    part = chunk_sum<METHOD, TEMP, MASK, kOneByOne>(x, ad, tp, sp, ex, j, near, kw.cap);                 \
  }
          if (!masked) {
            CAPATTN_CHUNK(0)
          } else if (!p.bounds) {
            CAPATTN_CHUNK(1)
          } else {
            CAPATTN_CHUNK(2)
          }
#undef CAPATTN_CHUNK
          const float y = part - comp, t = sum + y;
          comp = (t - sum) - y;
          sum = t;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_free + 8 * u);
      }
      step = end;
      // ------------------------------------------------------ end of a piece
      // The first warpgroup adds the four up and writes; the others go on.  (s_sum
      // alternates: it is written again only after the next piece's barrier.)
      float(*sums)[BT] = s_sum[parity];
      parity ^= 1;
      sums[wg][r] = sum;
      named_bar_sync(1, 32 * kElem);
      if (wg != 0) continue;
      float* w = kw.w + ((size_t)b * p.Hkv + g) * kw.w_stride + k0;
      const float all = (sums[0][r] + sums[1][r]) + (sums[2][r] + sums[3][r]);
      if (it.whole) {
        if (j < p.Lk) w[r] = all;
        continue;
      }
      kw.partial[(size_t)it.slot * BT + r] = all;
      __threadfence();
      named_bar_sync(2, BT);
      const int c0 = it.sh.cta_of(it.s0), c1 = it.sh.cta_of(it.s1 - 1);
      if (threadIdx.x == 64) {
        const bool last = atomicAdd(&kw.counters[c0], 1u) == (uint32_t)(c1 - c0);
        __threadfence();
        join_flag = last;
      }
      named_bar_sync(2, BT);
      if (join_flag && j < p.Lk) {
        const int late = it.s0 != it.sh.begin_of(c0) ? 1 : 0;
        float x = 0.f;
        for (int c = c0; c <= c1; ++c) x += __ldcg(&kw.partial[(size_t)(2 * c + (c == c0 ? late : 0)) * BT + r]);
        w[r] = x;
      }
      named_bar_sync(2, BT);  // join_flag is read
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, NBUF * BT);
  }
}

template <int METHOD, int HD, bool TEMP>
cudaError_t run_temp(const Params& p, const KeyWeightsParams& kw, cudaStream_t s) {
  auto* k = key_weights_tc_kernel<METHOD, HD, TEMP>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), smem_bytes<HD>(), done);
  CUtensorMap mq, mk;
  if (e == cudaSuccess) e = make_bhld_map(&mq, p.q, p.B, p.L, p.Hq, HD, BT);
  if (e == cudaSuccess) e = make_bhld_map(&mk, p.k, p.B, p.Lk, p.Hkv, HD, BT);
  if (e != cudaSuccess) return e;
  const int64_t entries = (int64_t)p.B * p.nk;
  e = launch_pdl(key_plan_kernel, dim3((unsigned)((entries + 3) / 4)), dim3(128), 0, s, p, kw);
  if (e != cudaSuccess) return e;
  // no more CTAs than there can be steps
  const int64_t most = entries * p.Hkv * p.nq * p.G;
  return launch_pdl(k, dim3((unsigned)(most < kWeightCtas ? most : kWeightCtas)), dim3(kThreads), smem_bytes<HD>(), s, mq,
                    mk, p, kw);
}

template <int METHOD, int HD>
cudaError_t run(const Params& p, const KeyWeightsParams& kw, cudaStream_t s) {
  return p.temp ? run_temp<METHOD, HD, true>(p, kw, s) : run_temp<METHOD, HD, false>(p, kw, s);
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
