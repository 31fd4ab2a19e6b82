// Attention of many new tokens per sequence over the paged cache on the 5th-generation
// tensor cores (bf16).
//
// Per query tile (tokens x query heads of one KV head, up to 128 rows) and 128 slots:
//   S = Q K^T, x = log2(e) temp cap(sm_scale S), P = 2^(x - m), l += sum P, O += P V.
// One CTA per SM takes an equal share of all steps (paged_sched.cuh); the query heads of a
// group lie in one tile, so a key is read once for all of them, and a tile of a prompt
// spans few tokens, which wastes little of its causal edge.
//
// The reference m of a row's exponentials is fixed before its scores are seen, so no step
// looks for a maximum and a row's threads exchange nothing but l at the end:
//   with a cap, |x| is bounded and m = min(max(0, bound - 100), 40) (0 for all usual caps,
//   which also makes x - m exact), which serves rows whose largest x is between -40 and 160;
//   without one, and with one so wide that rows may lie elsewhere (is_wide_cap), m comes from
//   the live scores of the piece's first step (0 while the largest is within 2^+-40).  Wide
//   caps have a kernel of their own, since the exchange of a row's largest score among its warps
//   costs 2 to 3 us a piece: tanh 300 and 50 take 155 and 137 us (a prompt of 4096 tokens, 32 / 8
//   heads), 418 and 268 (64 of 512); in the ordinary kernel, not used, it cost 1 to 10 %.
// That holds for logits within about 2^100 above m; a row whose sum leaves [2^-80, inf),
// and one that met NaN or infinity in a slot that is not live for it (0 times them), gets
// NaN for its lse and is formed once more by paged_finish_kernel, a warp a row: some 1500
// times as long (a prompt of 4096 tokens under tanh 300 with m = bound - 100: 213 ms).
//
// Warp roles (20 warps):
//   warp 19      walks the CTA's pieces into a ring of eight slots and loads their Q by TMA;
//                warps 0 and 18 follow and load K and V, a page (or 128 rows of one) a box,
//                into rings; V's rows without a token are zeroed (0 times what they hold must
//                be 0);
//   warp 1       TMEM allocator and MMA issuer: S_0 S_1 S_2 | PV_0 S_3 | PV_1 S_4 | ... over
//                the steps of all pieces, so that a piece's first scores are there when the
//                last one's end;
//   warps 2..17  softmax, eight for the even steps and eight for the odd ones, two threads a
//                row, 64 slots each: loads of 32 columns (which give the largest |S| too, for
//                the choice of the cap's polynomial), P stored over the scores.  With three
//                score buffers a group finds its next scores ready when it has written P.
//                Around a piece's first step they write the last piece's O.
// TMEM (512 columns): S / P [0, 128), [128, 256), [256, 384), O [384, 384 + D).
// P is rounded to bf16 (at most half a step of o's own type, and the sum l is of the
// unrounded values): a second product for its low half would cost as much as the first.
// o's error against 64 bits is 2.3e-3 of its size, 1.7e-3 of it its own rounding.  A row of one
// live slot, whose o is its value, divides by the rounded P (l has its sign set on the way);
// rounded sums for every row cost the windowed prompts 12 us and gain nothing from some ten
// slots on.
//
// What bounds it: long prompts, the softmax (issue slots 57-59 % used, tensor pipe 40-60 % of
// the active cycles; no pipe is full, the two groups wait for tensor memory and the issuer in
// turn); trees and long caches, memory; single small sequences, the chain of lengths, pages,
// tiles and the join.  A chunk of 4096 tokens behind 12,288, 32 / 8 heads x 128, tanh: 702 us
// (1370 TFLOP/s; 660 without a cap, 850 soft_sign, 837 alsc); nine prompts of 128 to 3969
// tokens, 16 / 16 heads, soft_sign: 258 us; four of 4096, 32 / 8 heads, window 1024, alsc,
// temperatures: 308 us; 64 of 512, 32 / 8 heads, tanh: 272 us; 32 trees of 16 tokens on 916 to
// 4016, 32 / 8 heads, alsc: 71 us (4.7 TB/s); one of 32 on 131,009: 93 us (5.8 TB/s).
//
// What was tried and lost (the chunk's, the nine prompts' or the windowed ones' us): one group
// of 16 warps for every step (705, 307, 337), with P in tensor memory of its own (876, 353,
// 394); separate issuers of S and of P V (spills at 80 registers); K and V by one warp (898),
// pieces by K's warp (645, but 64 short prompts 343) or the issuer's (670, 302); waits for the
// last P V before P is written (730); 16 columns at a time (alsc 966, 334); the two 32-column
// halves unrolled (355: the loop outgrows the instruction cache); masked columns out of line
// (584); MMAs issued in a loop (863) or under a branch of one lane (730); 104 registers for
// the softmax warps and 64 for the others (spills: 980, 411, 486).
#include <float.h>

#include "fwd_common.cuh"
#include "paged_out.cuh"
#include "tma_maps.h"

namespace capattn {
namespace {

using fwdtc::BN;
using fwdtc::SLAB;
using fwdtc::tile_bytes;

constexpr int BM = kAttendRows;
// K and V stages
template <int HD>
constexpr int kst() { return HD == 64 ? 4 : 2; }
template <int HD>
constexpr int vst() { return HD == 64 ? 4 : 2; }
constexpr uint32_t NSB = 3;       // score buffers
constexpr uint32_t kOCol = 384;   // TMEM column of O
constexpr int NSLOT = 8;  // pieces known ahead
constexpr int kSoftmaxWarps = 16;
constexpr int NTHREADS = 640;
constexpr float kLeastSum = 0x1p-80f;
// two Q tiles, the K and V tiles, the sums [2][4][128] and the first step's maxima
template <int HD>
constexpr int smem_bytes() { return (2 + kst<HD>() + vst<HD>()) * tile_bytes<HD>() + 2 * 4096 + 1024; }

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// mbar_wait_warp with all but the first try out of line: the roles' loops run once a step
// each and fetch their instructions anew, so a wait of 40 of them costs more than a call.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, uint32_t* status, volatile int* abort_flag) {
  return mbar_wait(bar, parity, status, abort_flag);
}
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, uint32_t* status, volatile int* abort_flag) {
  const bool ok = mbar_try_wait(bar, parity) || wait_long(bar, parity, status, abort_flag);
  return __all_sync(0xFFFFFFFFu, ok);
}

// Values that an asynchronous TMEM load delivers: nothing that uses them moves before the
// wait that this follows.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
__device__ __forceinline__ void tmem_st4(uint32_t taddr, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
template <int N>
__device__ __forceinline__ void settled(uint32_t (&v)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) asm volatile("" : "+r"(v[e]));
}

// Matrix descriptors whose high word is a constant (128-byte swizzle, rows of 8 x 128 bytes):
// only the low one, the address, is computed.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lbo_bytes) { return ((addr >> 4) & 0x3FFFu) | (lbo_bytes >> 4) << 16; }

__device__ __forceinline__ void mma_ts_low(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc, uint32_t go) {
  asm volatile(
      "{ .reg .pred p, q; .reg .b64 y; setp.ne.b32 p, %5, 0; setp.ne.b32 q, %6, 0; mov.b64 y, {%2, %3};"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p; }" ::"r"(d), "r"(a), "r"(b), "n"(kDescHigh), "r"(idesc), "r"(acc), "r"(go)
      : "memory");
}
__device__ __forceinline__ void mma_ss_low(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc, uint32_t go) {
  asm volatile(
      "{ .reg .pred p, q; .reg .b64 x, y; setp.ne.b32 p, %5, 0; setp.ne.b32 q, %6, 0; mov.b64 x, {%1, %3}; mov.b64 y, {%2, %3};"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p; }" ::"r"(d), "r"(a), "r"(b), "n"(kDescHigh), "r"(idesc), "r"(acc), "r"(go)
      : "memory");
}
// S = Q K^T, O += P V (P packed at the start of each 32 columns of its score buffer).
template <int HD>
__device__ __forceinline__ void issue_s(uint32_t d, uint32_t dQ, uint32_t dK, uint32_t go) {
  constexpr uint32_t idesc = idesc_bf16(BM, BN, 0, 0);
#pragma unroll
  for (int ks = 0; ks < HD / 16; ++ks) {
    const uint32_t off = ((ks >> 2) * SLAB + (ks & 3) * 32) >> 4;
    mma_ss_low(d, dQ + off, dK + off, idesc, ks > 0 ? 1u : 0u, go);
  }
}
template <int HD>
__device__ __forceinline__ void issue_pv(uint32_t d, uint32_t pt, uint32_t dV, uint32_t acc0, uint32_t go) {
  constexpr uint32_t idesc = idesc_bf16(BM, HD, 0, 1);
#pragma unroll
  for (int ks = 0; ks < BN / 16; ++ks)
    mma_ts_low(d, pt + 32 * (ks >> 1) + 8 * (ks & 1), dV + ((ks * 2048) >> 4), idesc, ks > 0 ? 1u : acc0, go);
}
__device__ __forceinline__ void commit_if(uint32_t bar, uint32_t go) {
  asm volatile("{ .reg .pred q; setp.ne.b32 q, %1, 0; @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0]; }" ::"r"(bar), "r"(go) : "memory");
}

// x = log2(e) temp cap(sm_scale X) of one row as X Q: the cap's polynomial near zero times
// the row's factor.
template <int METHOD>
struct RowPoly {
  static constexpr int N = METHOD == CAPATTN_CAP_TANH ? 3 : METHOD == CAPATTN_CAP_NONE ? 1 : 7;
  F2 c[N];
  __device__ __forceinline__ void set(const ExactCap& k, float mul) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float x = METHOD == CAPATTN_CAP_TANH ? k.near.c[i] : METHOD == CAPATTN_CAP_NONE ? k.sm_scale : k.poly[i];
      c[i] = f2(x * mul, x * mul);
    }
  }
  __device__ __forceinline__ F2 eval(F2 X) const {
    F2 z = METHOD == CAPATTN_CAP_TANH ? f2_mul(X, X) : X;
    if constexpr (METHOD == CAPATTN_CAP_SOFT_SIGN) z.v &= 0x7FFFFFFF7FFFFFFFull;  // |X|
    F2 q = c[N - 1];
#pragma unroll
    for (int i = N - 2; i >= 0; --i) q = f2_fma(q, z, c[i]);
    return q;
  }
};

// How a step's scores are capped: by the row's polynomial, by tanh's longer one, one by one.
enum { kNear, kWide, kOneByOne };

// N columns of P, packed to bf16; adds their sums (of the even and the odd ones) to acc.
template <int METHOD, int LEVEL, bool MASKED, int N>
__device__ __forceinline__ void p_columns(F2& acc, const uint32_t (&v)[N], uint32_t (&pk)[N / 2], const RowPoly<METHOD>& poly,
                                          float mul, float add, uint32_t live, const ExactCap& k) {
  const F2 add2 = f2(add, add), mul2 = f2(mul, mul);
#pragma unroll
  for (int e = 0; e < N / 2; ++e) {
    const F2 X = f2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
    F2 y;
    if constexpr (LEVEL == kNear) {
      y = f2_fma(X, poly.eval(X), add2);
    } else if constexpr (LEVEL == kWide) {
      y = f2_fma(poly_cap2<METHOD>(X, k), mul2, add2);
    } else {
      y = f2_fma(f2(any_cap<METHOD>(__uint_as_float(v[2 * e]), k), any_cap<METHOD>(__uint_as_float(v[2 * e + 1]), k)),
                 mul2, add2);
    }
    float a, b;
    f2_split(y, a, b);
    a = ex2_approx(a);
    b = ex2_approx(b);
    if constexpr (MASKED) {
      if (!(live & (1u << (2 * e)))) a = 0.f;
      if (!(live & (2u << (2 * e)))) b = 0.f;
    }
    acc = f2_add(acc, f2(a, b));
    pk[e] = pack_bf16x2(a, b);
  }
}
__device__ __forceinline__ float total(F2 acc) {
  float a, b;
  f2_split(acc, a, b);
  return a + b;
}

template <int METHOD>
__device__ __forceinline__ bool is_near(float top, const ExactCap& k) {
  if constexpr (METHOD == CAPATTN_CAP_NONE) return true;
  return __all_sync(0xFFFFFFFFu, top <= (METHOD == CAPATTN_CAP_TANH ? k.near.xmax : k.xmax));
}

// 32 columns whose scores leave the row's polynomial, from tensor memory to P in their place;
// returns their sum.  Out of line, so that the loop that runs without it stays small; it loads
// the scores once more (handed over, they went through local memory, which the little L1 beside
// the tiles does not hold: a step took 6 us).  The scores of slots without a token are of
// whatever lies there, so the choice is made once more from the live ones, for eight columns at
// a time, and the sum goes in the inline forms' order: a result's last bit would show either.
// With queries that make scores of sigma 4, 12 and 12 at caps of 50 (tanh), 20 (soft_sign) and 30
// (alsc), a prompt of 4096 tokens, 32 / 8 heads, takes 276, 247 and 834 us instead of 143 (near);
// inline these were 231, 232 and 506 but 64 short prompts of small scores 291 instead of 272.
template <int METHOD>
__device__ __noinline__ float p_far(uint32_t at, float mul, float add, uint32_t live, const ExactCap& k) {
  RowPoly<METHOD> poly;
  poly.set(k, mul);
  F2 acc = f2(0.f, 0.f);
#pragma unroll 1
  for (int e0 = 0; e0 < 32; e0 += 8) {
    uint32_t v[8], pk[4];
    tmem_ld8(at + e0, v);
    tmem_wait_ld();
    settled(v);
    const uint32_t mine = live >> e0;
    float top = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if ((mine >> e) & 1u) top = fmaxf(top, fabsf(__uint_as_float(v[e])));
    if (is_near<METHOD>(top, k)) {
      p_columns<METHOD, kNear, true>(acc, v, pk, poly, mul, add, mine, k);
    } else if (METHOD == CAPATTN_CAP_TANH && __all_sync(0xFFFFFFFFu, top <= k.xmax)) {
      p_columns<METHOD, METHOD == CAPATTN_CAP_TANH ? kWide : kOneByOne, true>(acc, v, pk, poly, mul, add, mine, k);
    } else {
      p_columns<METHOD, kOneByOne, true>(acc, v, pk, poly, mul, add, mine, k);
    }
    __syncwarp();
    tmem_st4(at + e0 / 2, pk);
    tmem_wait_st();
  }
  return total(acc);
}

// The largest live score (sign 1) or the smallest one's negative (-1) of 64 columns of a row.
__device__ __noinline__ float live_top(uint32_t at, float sign, uint64_t live) {
  float top = -INFINITY;
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    uint32_t v[32];
    tmem_ld32(at + 32u * h, v);
    const uint32_t mine = (uint32_t)(live >> (32 * h));
    tmem_wait_ld();
    settled(v);
#pragma unroll
    for (int e = 0; e < 32; ++e)
      if ((mine >> e) & 1u) top = fmaxf(top, sign * __uint_as_float(v[e]));
  }
  return top;
}

// The largest x of a row: |cap| times its factor's size.
template <int METHOD>
__device__ __forceinline__ float largest_x(const ExactCap& k, float mul) {
  if constexpr (METHOD == CAPATTN_CAP_ALSC) return fmaxf(mul * k.alsc.out * k.alsc.one_minus_sb, -mul * k.alsc.out * k.alsc.sb);
  return fabsf(mul * k.cap);
}

template <int METHOD, int HD, bool WIDE>
__global__ void __launch_bounds__(NTHREADS, 1)
paged_tc_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                const __grid_constant__ CUtensorMap mv, const PagedParams p) {
  constexpr int TILE = tile_bytes<HD>();
  constexpr int NSLAB = HD / 64;
  constexpr int KST = kst<HD>(), VST = vst<HD>();
  constexpr int OQ = HD / 4;  // O columns of a thread
  constexpr bool LOOK = METHOD == CAPATTN_CAP_NONE || WIDE;  // the first step's scores give the reference
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * 2 + 2 * KST + 2 * VST + 2 * NSB + 2 + 2 * NSLOT + 4 + 8 + 2];
  __shared__ Piece items[NSLOT];
  __shared__ ScheduleMem s_sched;
  __shared__ uint32_t s_bad[2][4][4];  // piece parity, quarter, rows / 32
  __shared__ int s_drained[2][4];      // piece parity, rows / 32: warps that have read their part of O
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const CacheParams& c = p.c;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = base;                     // buffer x at + x * TILE
  const uint32_t sK = base + 2 * TILE;          // stage s at + s * TILE
  const uint32_t sV = base + (2 + KST) * TILE;  // stage s at + s * TILE
  float* sums = reinterpret_cast<float*>(smem_raw + (base - smem_u32(smem_raw)) + (2 + KST + VST) * TILE);
  float* tops = sums + 2 * 4 * BM;

  const uint32_t bar_qfull = smem_u32(&bars[0]);     // + 8 x
  const uint32_t bar_qempty = bar_qfull + 16;        // + 8 x: the piece's last S complete
  const uint32_t bar_kfull = bar_qempty + 16;        // + 8 s
  const uint32_t bar_kempty = bar_kfull + 8 * KST;   // + 8 s
  const uint32_t bar_vfull = bar_kempty + 8 * KST;   // + 8 s
  const uint32_t bar_vempty = bar_vfull + 8 * VST;   // + 8 s
  const uint32_t bar_sfull = bar_vempty + 8 * VST;   // + 8 x: S in buffer x complete
  const uint32_t bar_pfull = bar_sfull + 8 * NSB;    // + 8 x: P in buffer x written (8 warps)
  const uint32_t bar_ofull = bar_pfull + 8 * NSB;        // the piece's last P V complete
  const uint32_t bar_oempty = bar_ofull + 8;         // O read by the 16 softmax warps
  const uint32_t bar_ifull = bar_oempty + 8;         // + 8 s: piece slot written
  const uint32_t bar_iempty = bar_ifull + 8 * NSLOT; // + 8 s: piece done with (19 warps)
  const uint32_t bar_sums = bar_iempty + 8 * NSLOT;  // + 8 x: the sums of rows 32 x .. written (4 warps)
  const uint32_t bar_tops = bar_sums + 32;           // + 8 (2 x + piece parity): first step's maxima (2 warps)
  const uint32_t bar_vfix = bar_tops + 64;           // V rows that get zeros have landed
  const uint32_t bar_final = bar_vfix + 8;

  if (threadIdx.x < 8) s_drained[threadIdx.x >> 2][threadIdx.x & 3] = 0;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar_qfull + 8 * x, 1);
      mbar_init(bar_qempty + 8 * x, 1);
    }
    for (uint32_t x = 0; x < NSB; ++x) {
      mbar_init(bar_sfull + 8 * x, 1);
      mbar_init(bar_pfull + 8 * x, kSoftmaxWarps / 2);
    }
    mbar_init(bar_ofull, 1);
    mbar_init(bar_oempty, kSoftmaxWarps);
    for (int s = 0; s < KST; ++s) {
      mbar_init(bar_kfull + 8 * s, 1);
      mbar_init(bar_kempty + 8 * s, 1);
    }
    for (int s = 0; s < VST; ++s) {
      mbar_init(bar_vfull + 8 * s, 1);
      mbar_init(bar_vempty + 8 * s, 1);
    }
    for (int s = 0; s < NSLOT; ++s) {
      mbar_init(bar_ifull + 8 * s, 1);
      mbar_init(bar_iempty + 8 * s, 3 + kSoftmaxWarps);
    }
    for (int x = 0; x < 4; ++x) mbar_init(bar_sums + 8 * x, 4);
    for (int x = 0; x < 8; ++x) mbar_init(bar_tops + 8 * x, 2);
    mbar_init(bar_vfix, 1);
    mbar_init(bar_final, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), 512);
    tmem_relinquish();
  }
  // the setup above overlaps the previous kernel's tail; global memory only after it
  pdl_trigger();
  pdl_wait();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const bool few = c.B <= kWarpSeqs;
  if (!few) schedule_by_cta<BN>(p, NTHREADS, s_sched);

  // The next piece (k-th) as every role but the walker reads it.
  auto wait_piece = [&](int k) -> bool {
    return wait_warp(bar_ifull + 8 * (k % NSLOT), (k / NSLOT) & 1, c.status, &abort_flag) && items[k % NSLOT].steps > 0;
  };
  auto done_with = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_iempty + 8 * (k % NSLOT));
  };

  if (warp == 19) {
    // ------------------------------------------------------------ pieces and Q
    const bool leader = elect_one_sync();
    if (leader) tma_prefetch_desc(&mq);
    __syncwarp();
    const uint32_t bytes = (uint32_t)(p.heads * p.tokens) * 128u * NSLAB;
    PieceWalk<BN> walk(p, few ? schedule_by_warp<BN>(p, lane) : s_sched.out, lane);
    int k = 0, loaded = 0;
    bool shared = false;
    for (;; ++k) {
      const Piece x = walk.next(p);
      if (x.steps > 0 && !x.whole && x.c0 == (int)blockIdx.x) {
        if (lane == 0) leave_record(p, x);
        shared = true;
      }
      if (k >= NSLOT && !wait_warp(bar_iempty + 8 * (k % NSLOT), (k / NSLOT - 1) & 1, c.status, &abort_flag)) break;
      if (lane == 0) {
        items[k % NSLOT] = x;
        mbar_arrive(bar_ifull + 8 * (k % NSLOT));
      }
      __syncwarp();
      if (x.steps < 0) break;
      const int y = k & 1;
      if (k >= 2 && !wait_warp(bar_qempty + 8 * y, ((k >> 1) - 1) & 1, c.status, &abort_flag)) break;
      if (leader) {
        const int g = x.part / p.parts, head0 = g * c.G + (x.part - g * p.parts) * p.heads;
        mbar_expect_tx(bar_qfull + 8 * y, bytes);
        for (int sl = 0; sl < NSLAB; ++sl)
          tma_load_3d(sQ + y * TILE + sl * SLAB, &mq, bar_qfull + 8 * y, 64 * sl, head0, x.row0 + x.i0);
      }
      loaded = k + 1;
      __syncwarp();
    }
    if (!shared && lane == 0) leave_no_record(p);
    // (on an early exit the copies in flight land before the CTA ends)
    if (leader)
      for (int x = loaded > 2 ? loaded - 2 : 0; x < loaded; ++x) drain_wait(bar_qfull + 8 * (x & 1), (x >> 1) & 1);
    __syncwarp();
  } else if (warp == 0 || warp == 18) {
    // ------------------------------------------------------------ K (warp 0) and V (warp 18)
    const bool values = warp == 18;
    const CUtensorMap* map = values ? &mv : &mk;
    const int rows = min(BN, c.page_size), boxes = BN / rows;  // rows of a box, boxes of a step (one a lane)
    const uint32_t box_bytes = (uint32_t)rows * 128u * NSLAB;
    const uint32_t tiles = values ? sV : sK, full0 = values ? bar_vfull : bar_kfull, empty0 = values ? bar_vempty : bar_kempty;
    const int stages = values ? VST : KST;
    if (lane == 0) tma_prefetch_desc(map);
    int j = 0, fixes = 0;
    bool ok = true, landing = false;  // landing: copies that bar_vfix counts may be on their way
    for (int k = 0; ok && wait_piece(k); ++k) {
      const Piece& x = items[k % NSLOT];
      const int g = x.part / p.parts, len = x.len, first = x.first, tile0 = x.tile0, steps = x.steps;
      const int32_t* table = c.table + (size_t)x.b * c.max_pages;
      done_with(k);
      // The page of this lane's box of a step, as read; looked at a step later.
      constexpr int kNoBox = INT_MIN;
      auto page_at = [&](int t) {
        const int slot = t * BN + lane * rows;
        return lane >= boxes || slot >= len || slot + rows <= first ? kNoBox : table[slot >> c.page_shift];
      };
      int page = page_at(tile0);
      for (int i = 0; i < steps; ++i, ++j) {
        const int t = tile0 + i, next = i + 1 < steps ? page_at(t + 1) : kNoBox;
        const int s = j % stages, u = j / stages;
        if (u > 0 && !wait_warp(empty0 + 8 * s, (u - 1) & 1, c.status, &abort_flag)) {
          ok = false;
          break;
        }
        // rows without a token: [0, lo) and [hi, 128)
        const int lo = first > t * BN ? (first - t * BN) / rows * rows : 0, hi = min(BN, len - t * BN);
        const bool fix = values && (lo > 0 || hi < BN);
        const uint32_t bar = fix ? bar_vfix : full0 + 8 * s, dst = tiles + s * TILE;
        const int n = __popc(__ballot_sync(0xFFFFFFFFu, page != kNoBox));
        if (lane == 0) mbar_expect_tx(bar, n * box_bytes);
        __syncwarp();
        if (page != kNoBox) {
          if (page < 0 || page >= c.num_pages) {  // flagged, and read as page 0
            atomicOr(c.status, kStatusBadPageBit);
            page = 0;
          }
          const int row = (page * c.Hkv + g) * c.page_size + ((t * BN + lane * rows) & (c.page_size - 1));
#pragma unroll
          for (int sl = 0; sl < NSLAB; ++sl) tma_load_2d(dst + sl * SLAB + lane * rows * 128, map, bar, 64 * sl, row);
        }
        __syncwarp();
        if (fix) {
          if (!wait_warp(bar_vfix, fixes & 1, c.status, &abort_flag)) {
            ok = false;
            landing = true;
            break;
          }
          ++fixes;
          for (int r = lane >> 3; r < BN; r += 4) {
            if (r >= lo && r < hi) continue;
#pragma unroll
            for (int sl = 0; sl < NSLAB; ++sl)
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst + sl * SLAB + r * 128 + (lane & 7) * 16), "r"(0)
                           : "memory");
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(full0 + 8 * s);
        }
        page = next;
      }
    }
    if (lane == 0) {
      if (landing) drain_wait(bar_vfix, fixes & 1);
      for (int x = j > stages ? j - stages : 0; x < j; ++x) drain_wait(full0 + 8 * (x % stages), (x / stages) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t leader = elect_one_sync() ? 1u : 0u;
    const uint32_t dQ = desc_low(sQ, 16);
    const uint32_t dK = desc_low(sK, 16);
    const uint32_t dV = desc_low(sV, SLAB);
    int sk = 0, left = 0;                // next S: its piece, the piece's steps still to come (0: not known yet)
    uint32_t sg = 0, ks = 0, kp = 0;     // next S: its buffer; K stage and its phase
    // 1: issued, 0: there are no more steps, -1: a wait gave up
    auto issue_scores = [&]() -> int {
      if (left == 0) {
        if (!wait_warp(bar_ifull + 8 * (sk % NSLOT), (sk / NSLOT) & 1, c.status, &abort_flag)) return -1;
        left = __reduce_max_sync(0xFFFFFFFFu, items[sk % NSLOT].steps);
        if (left < 0) return 0;
        if (!wait_warp(bar_qfull + 8 * (sk & 1), (sk >> 1) & 1, c.status, &abort_flag)) return -1;
      }
      if (!wait_warp(bar_kfull + 8 * ks, kp, c.status, &abort_flag)) return -1;
      tc_fence_after();
      issue_s<HD>(tmem + 128u * sg, dQ + (uint32_t)(sk & 1) * (TILE >> 4), dK + ks * (TILE >> 4), leader);
      commit_if(bar_sfull + 8 * sg, leader);
      commit_if(bar_kempty + 8 * ks, leader);
      if (left == 1) commit_if(bar_qempty + 8 * (sk & 1), leader);  // its Q is no longer read
      __syncwarp();
      sg = sg + 1 == NSB ? 0 : sg + 1;
      if (++ks == KST) {
        ks = 0;
        kp ^= 1u;
      }
      if (--left == 0) ++sk;
      return 1;
    };
    int ahead = 1;
    for (uint32_t x = 0; x < NSB && ahead > 0; ++x) ahead = issue_scores();
    uint32_t g = 0, gp = 0, vs = 0, vp = 0;  // next P V: P's buffer, its phase; V stage, its phase
    for (int k = 0; ahead >= 0 && wait_piece(k); ++k) {
      const int n = __reduce_max_sync(0xFFFFFFFFu, items[k % NSLOT].steps);
      bool ok = true;
      for (int i = 0; i < n; ++i) {
        ok = wait_warp(bar_pfull + 8 * g, gp, c.status, &abort_flag) && wait_warp(bar_vfull + 8 * vs, vp, c.status, &abort_flag);
        // O has been read out since the last piece
        if (ok && i == 0 && k > 0) ok = wait_warp(bar_oempty, (k - 1) & 1, c.status, &abort_flag);
        if (!ok) break;
        tc_fence_after();
        issue_pv<HD>(tmem + kOCol, tmem + 128u * g, dV + vs * (TILE >> 4), i > 0 ? 1u : 0u, leader);
        commit_if(bar_vempty + 8 * vs, leader);
        if (i + 1 == n) commit_if(bar_ofull, leader);  // the piece's O is complete
        __syncwarp();
        if (++g == NSB) {
          g = 0;
          gp ^= 1u;
        }
        if (++vs == VST) {
          vs = 0;
          vp ^= 1u;
        }
        // S of the step three on overwrites this P after its P V (in-order MMAs)
        if (ahead > 0) ahead = issue_scores();
        ok = ahead >= 0;
        if (!ok) break;
      }
      done_with(k);
      if (!ok) break;
    }
    // (warp 1 re-checks this commit before it frees TMEM)
    commit_if(bar_final, leader);
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax and results
    const int cq = (warp - 2) >> 2;   // quarter of Q's and O's columns
    const int group = cq >> 1;        // takes the even or the odd steps,
    const int half = cq & 1;          // slots [64 half, 64 half + 64) of each
    const int quad = warp & 3;        // rows [32 quad, 32 quad + 32): the TMEM lanes it may access
    const int r = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t s_half = tmem + lane_off + 64u * (uint32_t)half;  // + 128 x: score buffer x
    uint32_t sb = (uint32_t)group, sp = 0;  // this group's next score buffer, its phase
    RowPoly<METHOD> poly;
    int g = 0;        // steps so far
    float m_prev = 0.f;  // reference of the piece whose O is still to leave
    // this thread's row of a tile: token and head (the box that Q comes in has p.heads heads)
    const int tok = r / p.heads, hh = r - tok * p.heads;
    // heads of a piece's part, its first one
    auto heads_of = [&](const Piece& x, int* g_out, int* head0) -> int {
      const int gk = p.parts == 1 ? x.part : x.part / p.parts, h0 = (x.part - gk * p.parts) * p.heads;
      *g_out = gk;
      *head0 = gk * c.G + h0;
      return min(p.heads, c.G - h0);
    };
    // The results of piece k: O out of its accumulator, normalised or as a partial result.
    auto drain = [&](int k) -> bool {
      const Piece& x = items[k % NSLOT];
      const int xx = k & 1;
      int gk, head0;
      const int heads = heads_of(x, &gk, &head0);
      const bool valid = tok < x.count && hh < heads;
      if (!wait_warp(bar_ofull, k & 1, c.status, &abort_flag)) return false;
      tc_fence_after();
      const uint32_t ob = tmem + lane_off + kOCol + (uint32_t)(OQ * cq);
      uint32_t o[OQ];
#pragma unroll
      for (int h = 0; h < OQ / 16; ++h) tmem_ld16(ob + 16u * h, *reinterpret_cast<uint32_t(*)[16]>(&o[16 * h]));
      tmem_wait_ld();
      settled(o);
      tc_fence_before();
      float zero = 0.f;  // NaN once an output is not finite
#pragma unroll
      for (int e = 0; e < OQ; ++e) zero = fmaf(__uint_as_float(o[e]), 0.f, zero);
      const uint32_t bad_here = __ballot_sync(0xFFFFFFFFu, zero != 0.f);
      // the last of the four warps of these rows knows what all of them saw
      int last = 0;
      if (lane == 0) {
        mbar_arrive(bar_oempty);
        s_bad[xx][cq][quad] = bad_here;
        __threadfence_block();
        last = atomicAdd(&s_drained[xx][quad], 1) == 3;
        if (last) s_drained[xx][quad] = 0;
        __threadfence_block();
      }
      last = __shfl_sync(0xFFFFFFFFu, last, 0);
      __syncwarp();
      if (!wait_warp(bar_sums + 8 * quad, k & 1, c.status, &abort_flag)) return false;
      float l = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) l += sums[(xx * 4 + e) * BM + r];
      const float l_o = l < 0.f ? __bfloat162float(__float2bfloat16_rn(-l)) : l;  // of the rounded P
      l = fabsf(l);
      const bool none = l == 0.f;  // no live slot
      bool bad = false;
      if (last) {
        uint32_t bad_rows = 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) bad_rows |= *const_cast<volatile uint32_t*>(&s_bad[xx][e][quad]);
        bad = !none && (((bad_rows >> lane) & 1u) || !(l >= kLeastSum) || !(l < INFINITY));
      }
      const size_t first = (size_t)(x.row0 + x.i0) * c.Hq + head0;  // row of o of the tile's first
      const size_t row = first + (size_t)tok * c.Hq + hh;
      if (x.whole) {
        const float inv = none ? 0.f : 1.f / l_o;
        // 16-byte chunks of the rows, passed about among four (D = 64: two) lanes so that they
        // write a row's chunks side by side: 32 lanes with a row each met 32 lines a store
        constexpr int CH = OQ / 8;
        uint4 y[CH];
#pragma unroll
        for (int e = 0; e < CH; ++e) {
          uint32_t w[4];
#pragma unroll
          for (int z = 0; z < 4; ++z) {
            const float a = __uint_as_float(o[8 * e + 2 * z]), b = __uint_as_float(o[8 * e + 2 * z + 1]);
            w[z] = none ? 0u : pack_bf16x2(a * inv, b * inv);
          }
          y[e] = make_uint4(w[0], w[1], w[2], w[3]);
        }
#pragma unroll
        for (int d = 1; d < CH; d <<= 1) {
          const bool high = lane & d;
#pragma unroll
          for (int e = 0; e < CH; ++e) {
            if (e & d) continue;
            uint4 give = high ? y[e] : y[e + d];
            give.x = __shfl_xor_sync(0xFFFFFFFFu, give.x, d);
            give.y = __shfl_xor_sync(0xFFFFFFFFu, give.y, d);
            give.z = __shfl_xor_sync(0xFFFFFFFFu, give.z, d);
            give.w = __shfl_xor_sync(0xFFFFFFFFu, give.w, d);
            if (high) y[e] = give; else y[e + d] = give;
          }
        }
        const int where = valid ? tok * c.Hq + hh : -1;
#pragma unroll
        for (int e = 0; e < CH; ++e) {
          const int to = __shfl_sync(0xFFFFFFFFu, where, (lane & ~(CH - 1)) + e);
          if (to >= 0)
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(c.o) + (first + to) * HD + OQ * cq + 8 * (lane & (CH - 1))) = y[e];
        }
        if (valid && last) {
          if (bad) ask_redo(p);
          c.lse[row] = bad ? kNaN32 : none ? -INFINITY : (m_prev + log2f(l)) * kLn2;
        }
        done_with(k);
        return true;
      }
      if (valid) {
        const float scale = l_o == l ? 1.f : l / l_o;
#pragma unroll
        for (int e = 0; e < OQ / 4; ++e)
          reinterpret_cast<float4*>(p.part_o)[part_at<HD, BM>(x.slot, r, cq, e)] =
              make_float4(__uint_as_float(o[4 * e]) * scale, __uint_as_float(o[4 * e + 1]) * scale,
                          __uint_as_float(o[4 * e + 2]) * scale, __uint_as_float(o[4 * e + 3]) * scale);
        if (last) {
          const size_t at = (size_t)x.slot * BM + r;
          p.part_ml[at] = make_float2(m_prev, l);
          p.part_bad[at] = bad ? 1u : 0u;
          if (x.c0 == (int)blockIdx.x) c.lse[row] = 0.f;  // whatever it held asks for nothing
        }
      }
      done_with(k);
      return true;
    };

    // Temperature of this thread's row of piece k (asked for a piece ahead).
    auto temp_of = [&](int k) -> float {
      const Piece& x = items[k % NSLOT];
      return tok < x.count ? __ldg(c.temp + x.row0 + x.i0 + tok) : 1.f;
    };
    float temp = 1.f;
    for (int k = 0;; ++k) {
      const bool more = wait_piece(k);
      // after the last piece only its O is left (and not even that after a wait that gave up)
      if (!more && (k == 0 || !__all_sync(0xFFFFFFFFu, abort_flag == 0))) break;
      const Piece& x = items[k % NSLOT];
      const int n = more ? x.steps : 0, tile0 = x.tile0;
      if (c.temp && k == 0) temp = temp_of(0);
      int gk, head0;
      const int heads = heads_of(x, &gk, &head0);
      const bool valid = more && tok < x.count && hh < heads;
      const float mul = temp * kL2E;
      float m = 0.f;
      RowMask mask = dead_row();
      if (valid) {
        const SeqShape sh = {x.row0, x.n, x.len, x.base};
        mask = row_mask(p, x.b, gk, sh, x.i0 + tok);
      }
      const bool block = __any_sync(0xFFFFFFFFu, valid);  // the warp has rows at all
      poly.set(c.cap, mul);
      if constexpr (!LOOK) m = fminf(fmaxf(0.f, largest_x<METHOD>(c.cap, mul) - 100.f), 40.f);
      float lsum = 0.f;
      bool seen = false;
      // The reference from the live scores of the piece's first step.  The two warps that arrive may
      // do so for piece k + 1 (whose first scores need nothing of piece k's last step) before the
      // other two have looked at piece k; for k + 2 they may not: they have written out piece k by
      // then, which takes the sums of all four, given after that look.  So two barriers in turn, as
      // the maxima have two buffers.
      const uint32_t bar_top = bar_tops + 8 * (2 * quad + (k & 1));
      auto reference = [&]() -> bool {
        const float* t = tops + (k & 1) * 2 * BM;
        if (!wait_warp(bar_top, (k >> 1) & 1, c.status, &abort_flag)) return false;
        const float best = fmaxf(t[r], t[BM + r]);
        m = best == -INFINITY || fabsf(best) <= 40.f ? 0.f : best;
        return true;
      };
      // one step: this half's P over its scores, handed to the issuer
      auto step = [&](int i) -> bool {
        const int c0 = (tile0 + i) * BN + 64 * half;
        if (!wait_warp(bar_sfull + 8 * sb, sp, c.status, &abort_flag)) return false;
        const uint32_t at_s = s_half + 128u * sb;
        if (block) {
          tc_fence_after();
          if (LOOK && i == 0) {
            float best = -INFINITY;
            if constexpr (METHOD == CAPATTN_CAP_NONE) {
#pragma unroll 1
              for (int h = 0; h < 2; ++h) {
                uint32_t v[32];
                tmem_ld32(at_s + 32u * h, v);
                const uint32_t live = valid ? live_slots(p, mask, c0 + 32 * h) : 0u;
                tmem_wait_ld();
                settled(v);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if ((live >> e) & 1u) best = fmaxf(best, __uint_as_float(v[e]) * (c.sm_scale * mul));
              }
            } else {
              uint64_t live = 0;
              if (valid) live = live_slots(p, mask, c0) | (uint64_t)live_slots(p, mask, c0 + 32) << 32;
              __syncwarp();
              // x rises or falls with the score everywhere, so the cap is taken once
              const float way = METHOD == CAPATTN_CAP_ALSC ? c.sm_scale * mul * c.cap.alsc.a : c.sm_scale * mul;
              const float sign = way < 0.f ? -1.f : 1.f, top = live_top(at_s, sign, live);
              if (top > -INFINITY) best = any_cap<METHOD>(sign * top, c.cap) * mul;
            }
            tops[((k & 1) * 2 + half) * BM + r] = best;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_top);
            if (!reference()) return false;
          }
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t v[32], pk[16];
            float top = tmem_ld32_absmax(at_s + 32u * h, v);
            const int at = c0 + 32 * h;
            const bool full = __all_sync(0xFFFFFFFFu, !valid || all_live(mask, at, 32));
            uint32_t live = 0xFFFFFFFFu;
            if (!full) live = live_slots(p, mask, at);
            tmem_wait_ld();
            settled(v);
            asm volatile("" : "+f"(top));
            if (!valid) top = 0.f;
            if (full && is_near<METHOD>(top, c.cap)) {
              F2 acc = f2(0.f, 0.f);
              p_columns<METHOD, kNear, false>(acc, v, pk, poly, mul, -m, live, c.cap);
              lsum += total(acc);
              seen = true;
            } else if (!__any_sync(0xFFFFFFFFu, live != 0u)) {
#pragma unroll
              for (int e = 0; e < 16; ++e) pk[e] = 0u;
            } else {
              if (__builtin_expect(is_near<METHOD>(top, c.cap), 1)) {
                F2 acc = f2(0.f, 0.f);
                p_columns<METHOD, kNear, true>(acc, v, pk, poly, mul, -m, live, c.cap);
                lsum += total(acc);
              } else {
                lsum += p_far<METHOD>(at_s + 32u * h, mul, -m, valid ? live : 0u, c.cap);
                seen = seen || live != 0u;
                continue;
              }
              seen = seen || live != 0u;
            }
            __syncwarp();
            tmem_st16(at_s + 32u * h, pk);
          }
          tmem_wait_st();
          tc_fence_before();
        } else if (LOOK && i == 0) {
          if (lane == 0) mbar_arrive(bar_top);
          if (!reference()) return false;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_pfull + 8 * sb);
        // every other step: two buffers on
        sb += 2;
        if (sb >= NSB) {
          sb -= NSB;
          sp ^= 1u;
        }
        return true;
      };
      // The group of the piece's first step goes on with it, then with the last piece's O (its
      // last P V, of the other group's step, has completed meanwhile); the other group begins
      // with that.
      bool ok = true;
      for (int i = more && (g & 1) == group ? 0 : -1; ok && i < max(n, 1); i += 2) {
        if (i >= 0 && i < n) ok = step(i);
        if (i > 0) continue;
        if (ok && k > 0) ok = drain(k - 1);
        if (!more) break;
        if (c.temp && ok && wait_piece(k + 1)) temp = temp_of(k + 1);
        if (LOOK && i < 0) ok = ok && reference();
      }
      if (!ok || !more) break;
      g += n;
      // l: 0 without a live slot, something positive with one, negative where it is the row's only
      const float l = !seen ? 0.f : lsum == 0.f ? FLT_MIN : lsum;
      sums[((k & 1) * 4 + cq) * BM + r] = valid && only_one(mask) ? -l : l;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_sums + 8 * quad);
      m_prev = m;
    }
  }
  __syncwarp();  // every warp reaches the CTA barrier converged
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    // Every MMA has completed before TMEM is released (bounded non-suspending poll).
    if (lane == 0) mbar_poll(bar_final, 0);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Whether a cap alone, at temperature 1, bounds x by more than 120 (tanh 83): the fixed reference
// then lies far above ordinary scores, or far below the bound.  (Temperatures are in device
// memory: they widen the rows' bounds, not this.)
bool is_wide_cap(const CacheParams& c) {
  if (c.method == CAPATTN_CAP_NONE) return false;
  const float top = c.method == CAPATTN_CAP_ALSC ? c.cap.alsc.out * c.cap.alsc.one_minus_sb : c.cap.cap;
  return !(top * kL2E <= 120.f);
}

template <int METHOD, int HD, bool WIDE>
cudaError_t run_tc(const PagedParams& p, cudaStream_t s) {
  const CacheParams& c = p.c;
  CUtensorMap mq, mk, mv;
  // q: a box is a tile's heads of its tokens; rows past the last token read as zero
  const cuuint64_t qd[3] = {(cuuint64_t)HD, (cuuint64_t)c.Hq, (cuuint64_t)p.n_rows};
  const cuuint64_t qs[2] = {(cuuint64_t)HD * 2, (cuuint64_t)c.q_stride * 2};
  const cuuint32_t qb[3] = {64, (cuuint32_t)p.heads, (cuuint32_t)p.tokens};
  // pages: a box is a page's rows of one head, at most a step's
  const cuuint64_t kd[2] = {(cuuint64_t)HD, (cuuint64_t)c.num_pages * c.Hkv * c.page_size};
  const cuuint64_t ks[1] = {(cuuint64_t)HD * 2};
  const cuuint32_t kb[2] = {64, (cuuint32_t)(c.page_size < BN ? c.page_size : BN)};
  cudaError_t e = encode_bf16_map(&mq, c.q, 3, qd, qs, qb);
  if (e == cudaSuccess) e = encode_bf16_map(&mk, c.k, 2, kd, ks, kb);
  if (e == cudaSuccess) e = encode_bf16_map(&mv, c.v, 2, kd, ks, kb);
  auto* kern = paged_tc_kernel<METHOD, HD, WIDE>;
  static std::atomic<uint64_t> done{0};
  if (e == cudaSuccess) e = allow_smem(reinterpret_cast<const void*>(kern), smem_bytes<HD>(), done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(p.ctas), dim3(NTHREADS), smem_bytes<HD>(), s, mq, mk, mv, p);
}

template <int METHOD>
struct PagedTcLaunch {
  static cudaError_t run(const PagedParams& p, cudaStream_t s) {
    if constexpr (METHOD != CAPATTN_CAP_NONE)
      if (is_wide_cap(p.c)) return p.c.D == 64 ? run_tc<METHOD, 64, true>(p, s) : run_tc<METHOD, 128, true>(p, s);
    return p.c.D == 64 ? run_tc<METHOD, 64, false>(p, s) : run_tc<METHOD, 128, false>(p, s);
  }
};

}  // namespace

cudaError_t launch_paged_attend_tc(const PagedParams& p, cudaStream_t s) {
  return dispatch_cap<PagedTcLaunch>(p.c.method, p, s);
}

}  // namespace capattn
