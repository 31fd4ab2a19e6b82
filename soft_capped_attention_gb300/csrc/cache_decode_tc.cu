// Attention of one new token per sequence over the paged cache, bf16.
//
// What bounds it: every cached key and value is read once, 4 D bytes a token and
// KV head against 4 D G operations, so memory does at any group size G of up to
// 16; the kernel's task is to keep the loads in flight.  Measured: 130,977 keys of 8
// heads (D = 128, 537 MB) in 85 us, 6.3 TB/s, 93 % of the measured copy rate; 32 users
// of 1024 to 3968 keys (82 MB) in 23 us, 3.6 TB/s (16 us when the last call has left
// them in L2); 64 sequences in a window of 1024
// (240 MB) in 45 us, 5.3 TB/s (of a consumer warp's 80,000 cycles 34,000 compute,
// 32,000 wait for memory and 14,000 are the starts, ends and joins of its pieces).  The
// CUDA-core form of the fp32 kernel took 230, 47 (from L2) and 120 us.  A persistent grid, two
// CTAs an SM, takes equal shares of 64-key tiles (cache_sched.cuh).  In each CTA
// one warp fills a ring of shared-memory stages by TMA (a tile's pages are boxes
// of up to a tile's rows x 64 columns in the 128-byte swizzle) and four warps compute,
// every fourth 16 keys of the tile each, with a running (m, l, O) of their own.  At a piece's end
// they leave those in shared memory and go on with the next piece; a sixth warp adds
// them up, writes, counts split pieces in and joins them when it comes last (a
// CTA's last piece they finish themselves: they have nothing else to do).
//
// Per warp and 16 keys, on mma.m16n8k16 (there is one query, so the heads of a
// group are the only other dimension: 8 columns a tile, two tiles for groups of 9
// to 16.  A tcgen05 tile of 128 rows would be 7/8 empty with heads as rows, and
// with keys as rows P would have to go through shared memory; at 24 bytes a clock
// and SM the mma pipe keeps up):
//   S^T = K Q^T  keys are the rows: K by ldmatrix, Q's fragments stay in registers
//   t = temp cap(sm_scale S), P = e^(t - m)
//   O^T += V^T P^T  V by ldmatrix.trans, P^T by transposing its accumulators
//                8 x 8 (movmatrix).  (With the heads as rows, half of them empty for
//                groups of 8, the mma pipe was 79 % busy: 60 us for the windowed
//                batch against 50.)  P goes in as two bf16 halves (P = hi + lo,
//                2^-17 of it lost): rounding P to one bf16 would add half of what
//                rounding o to bf16 does.
// The reference m moves only when the maximum outgrows it by kSlack (P stays
// below e^kSlack), which saves the rescaling of O on nearly every step.
#include <cuda_bf16.h>
#include <limits.h>

#include "cache_internal.h"
#include "cache_math.cuh"
#include "cache_sched.cuh"
#include "tma_maps.h"

namespace capattn {
namespace {

constexpr int kConsumers = 4;          // warps that compute, 16 keys of a tile each
constexpr int kThreads = (kConsumers + 2) * 32;  // and the TMA warp and the writing one
constexpr float kSlack = 8.f;

// Keys of a tile: 32 KB of keys and values, 64 keys (D = 128) or 128.
template <int D>
constexpr int tile_keys() { return 8192 / D; }
template <int D, int NT>
struct Geo {
  static constexpr int TK = tile_keys<D>();
  static constexpr int GROUPS = TK / 64;              // groups of 16 keys of a warp
  static constexpr int SLABS = D / 64;                // 128-byte wide columns of a row
  static constexpr int SLAB = TK * 128;
  static constexpr int HALF = SLABS * SLAB;           // K (or V) of a stage
  static constexpr int STAGE = 2 * HALF;
  static constexpr int STAGES = 3;                    // 96 KB a CTA, two CTAs an SM
  static constexpr int MERGE = 16 * D * 4;            // 4 warps x 4 heads x D floats
  // A group's queries, of as many pieces as there are stages where that fits (with
  // one slot a piece's tiles could not be asked for before the last piece's queries
  // are in registers, which left short sequences waiting for memory)
  static constexpr int Q = 8 * NT * D * 2;
  static constexpr int QSLOTS = D == 128 && NT == 2 ? 1 : 3;
  static constexpr int SMEM = STAGES * STAGE + MERGE + QSLOTS * Q + 1024;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "l"(policy)
      : "memory");
}
// Transposes an 8 x 8 matrix of bf16, a fragment register a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Two floats as bf16 pairs hi + lo.
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(x, y);
  lo = pack_bf16x2(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xFFFF0000u));
}

// NT: tiles of 8 query heads, 1 for groups of at most 8, else 2.
template <int D, int METHOD, int NT>
__global__ void __launch_bounds__(kThreads, 2)
decode_tc_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const CacheParams p) {
  using G = Geo<D, NT>;
  constexpr int TK = G::TK;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * G::STAGES + 2 * G::QSLOTS + 2];
  __shared__ int abort_flag, join_flag;
  __shared__ float s_m[kConsumers * 4], s_l[kConsumers * 4], s_join[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  float* merge = reinterpret_cast<float*>(smem_raw + (base - smem_u32(smem_raw)) + G::STAGES * G::STAGE);
  const uint32_t s_q = base + G::STAGES * G::STAGE + G::MERGE;
  const uint32_t full = smem_u32(&bars[0]), empty = smem_u32(&bars[G::STAGES]);
  const uint32_t q_full = smem_u32(&bars[2 * G::STAGES]), q_empty = q_full + 8 * G::QSLOTS;  // + 8 x: slot x
  const uint32_t m_full = q_empty + 8 * G::QSLOTS, m_empty = m_full + 8;  // the warps' results of four heads
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int s = 0; s < G::STAGES; ++s) {
      mbar_init(full + 8 * s, 1);
      mbar_init(empty + 8 * s, kConsumers);
    }
    for (int x = 0; x < G::QSLOTS; ++x) {
      mbar_init(q_full + 8 * x, 1);
      mbar_init(q_empty + 8 * x, kConsumers);
    }
    mbar_init(m_full, kConsumers);
    mbar_init(m_empty, 1);
    fence_mbar_init();
  }
  pdl_trigger();
  pdl_wait();
  __syncthreads();
  PieceIter<TK> it(p, warp, lane, kThreads / 32, reinterpret_cast<int*>(merge));
  int b, vh, tile;
  SeqSpan sp;
  uint32_t step = 0;   // tiles so far, over the pieces
  uint32_t piece = 0;  // pieces so far

  if (warp == kConsumers) {
    // ------------------------------------------------------------ TMA producer
    const int rows = min(TK, p.page_size);      // rows of a box
    const int pages = TK / rows;                // boxes of a tile, one a lane
    const uint32_t bytes = (uint32_t)rows * D * 2 * 2;
    if (lane == 0) {
      tma_prefetch_desc(&mk);
      tma_prefetch_desc(&mv);
    }
    // With weights, keys and values make room in L2 first, or they push out the scores
    // that the weights pass reads next (16 sequences of up to 8192 keys, 335 MB: 65.5 us
    // without, 60.5 with).
    uint64_t policy;
    if (p.scores)
      asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    else
      asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
    bool ok = true;
    while (ok && it.next(p, &b, &vh, &tile, &sp)) {
      const int g = vh / p.HG;
      // The page of this lane's box of a tile, as read (kNoBox: no live slot in it);
      // looked at a tile later, so that the read is not waited for.
      constexpr int kNoBox = INT_MIN;
      const int32_t* table = p.table + (size_t)b * p.max_pages;
      auto page_at = [&](int t) {
        const int j = t * TK + lane * rows;
        return lane >= pages || j >= sp.len || j + rows <= sp.first ? kNoBox : table[j >> p.page_shift];
      };
      int page = page_at(tile);
      // the group's queries
      const uint32_t qs = piece % G::QSLOTS, q_use = piece / G::QSLOTS;
      if (q_use > 0 && !mbar_wait_warp(q_empty + 8 * qs, (q_use - 1) & 1, p.status, &abort_flag)) break;
      if (lane == 0) {
        const HeadGroup hg = head_group(p, vh);
        const uint32_t q_bytes = (uint32_t)hg.count * D * 2;
        mbar_expect_tx(q_full + 8 * qs, q_bytes);
        bulk_load(s_q + qs * G::Q, static_cast<const __nv_bfloat16*>(p.q) + (size_t)b * p.q_stride + (size_t)hg.h0 * D,
                  q_bytes, q_full + 8 * qs);
      }
      ++piece;
      __syncwarp();
      for (int i = 0; i < it.n; ++i, ++step) {
        const int next = i + 1 < it.n ? page_at(tile + i + 1) : kNoBox;
        const uint32_t s = step % G::STAGES, use = step / G::STAGES;
        if (use > 0 && !mbar_wait_warp(empty + 8 * s, (use - 1) & 1, p.status, &abort_flag)) {
          ok = false;
          break;
        }
        const int boxes = __popc(__ballot_sync(0xFFFFFFFFu, page != kNoBox));
        if (lane == 0) mbar_expect_tx(full + 8 * s, boxes * bytes);
        __syncwarp();
        if (page != kNoBox) {
          if (page < 0 || page >= p.num_pages) {  // flagged, and read as page 0
            atomicOr(p.status, kStatusBadPageBit);
            page = 0;
          }
          const int row = (page * p.Hkv + g) * p.page_size + (((tile + i) * TK + lane * rows) & (p.page_size - 1));
          const uint32_t dst = base + s * G::STAGE + lane * rows * 128;
#pragma unroll
          for (int x = 0; x < G::SLABS; ++x) {
            tma_load_2d(dst + x * G::SLAB, &mk, full + 8 * s, 64 * x, row, policy);
            tma_load_2d(dst + G::HALF + x * G::SLAB, &mv, full + 8 * s, 64 * x, row, policy);
          }
        }
        __syncwarp();
        page = next;
      }
    }
    // normally long complete: the consumers waited for every stage
    for (uint32_t x = piece > G::QSLOTS ? piece - G::QSLOTS : 0; x < piece; ++x)
      drain_wait(q_full + 8 * (x % G::QSLOTS), (x / G::QSLOTS) & 1);
    for (uint32_t x = step > G::STAGES ? step - G::STAGES : 0; x < step; ++x)
      drain_wait(full + 8 * (x % G::STAGES), (x / G::STAGES) & 1);
    return;
  }

  uint32_t round = 0;  // groups of four heads handed over so far
  // Head g0 + e of a piece, from what the four warps left: written, or left as a
  // partial result.
  auto finish_head = [&](const HeadGroup& hg, int g0, int e) {
    constexpr int V = D / 32;
    float y[V], sum, top;
    merge_warps<D>(merge, s_m, s_l, e, lane, y, &sum, &top);
    if (it.whole) {
      const size_t row = (size_t)b * p.Hq + hg.h0 + g0 + e;
      const float inv = sum == 0.f ? 0.f : 1.0f / sum;
#pragma unroll
      for (int x = 0; x < V; x += 2)
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(p.o) + row * D + lane * V + x) =
            pack_bf16x2(y[x] * inv, y[x + 1] * inv);
      if (lane == 0) p.lse[row] = sum == 0.f ? -INFINITY : top + logf(sum);
    } else {
      const size_t at = (size_t)it.slot * kDecodeHeads + g0 + e;
#pragma unroll
      for (int x = 0; x < V; ++x) p.part_o[at * D + lane * V + x] = y[x];
      if (lane == 0) p.part_ml[at] = make_float2(top, sum);
    }
  };
  if (warp == kConsumers + 1) {
    // ------------------------------------------------------------ writing warp
    while (it.next(p, &b, &vh, &tile, &sp)) {
      if (it.u >= it.end) break;  // the last piece is the consumers'
      const HeadGroup hg = head_group(p, vh);
      for (int g0 = 0; g0 < hg.count; g0 += 4, ++round) {
        mbar_wait_warp(m_full, round & 1, p.status, &abort_flag);  // (after a timeout: whatever is there)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (g0 + e < hg.count) finish_head(hg, g0, e);
        __syncwarp();
        if (lane == 0) mbar_arrive(m_empty);
      }
      if (it.whole) continue;
      const Pieces pc(it);
      if (count_piece_warp(p, pc, lane)) join_pieces<__nv_bfloat16, D, 1>(p, pc, b, hg, 0, lane, 0, nullptr, nullptr);
    }
    return;
  }

  // ---------------------------------------------------------------- consumers
  const int gq = lane >> 2, tq = lane & 3;      // fragment row and column group
  const uint32_t sw = lane & 7;
  // this lane's row addresses in a stage's K and V slabs: matrices (keys 0-7, d
  // 0-7), (keys 8-15, d 0-7), (keys 0-7, d 8-15), (keys 8-15, d 8-15) of K, and with
  // the middle two exchanged of V
  const uint32_t k_row = (uint32_t)(16 * warp + (lane & 7) + (((lane >> 3) & 1) << 3)) * 128u, k_add = lane >> 4;
  const uint32_t v_row = (uint32_t)(16 * warp + (lane & 7) + ((lane >> 4) << 3)) * 128u, v_add = (lane >> 3) & 1;
  bool ok = true;
  while (it.next(p, &b, &vh, &tile, &sp)) {
    const HeadGroup hg = head_group(p, vh);
    const float temp = p.temp ? p.temp[b] : 1.f;
    const bool by_pos = p.pos && p.window_len > 0;
    const int32_t* pos = p.pos + ((size_t)b * p.Hkv + hg.g) * p.max_len;
    const int oldest = by_pos ? p.qpos[b] - p.window_len : 0;
    uint32_t q[NT][D / 16][2];
    const uint32_t qs = piece % G::QSLOTS;
    ok = ok && mbar_wait_warp(q_full + 8 * qs, (piece / G::QSLOTS) & 1, p.status, &abort_flag);
    ++piece;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          q[t][ks][e] = 0u;
          if (gq + 8 * t < hg.count)
            asm volatile("ld.shared.b32 %0, [%1];"
                         : "=r"(q[t][ks][e])
                         : "r"(s_q + qs * G::Q + (gq + 8 * t) * D * 2 + 32 * ks + 16 * e + 4 * tq)
                         : "memory");
        }
    __syncwarp();
    if (lane == 0) mbar_arrive(q_empty + 8 * qs);
    // heads of this lane: 8 t + 2 tq + e; keys: 16 warp + gq + 8 k
    float m[NT][2], l[NT][2], o[NT][D / 16][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      m[t][0] = m[t][1] = -INFINITY;
      l[t][0] = l[t][1] = 0.f;
#pragma unroll
      for (int x = 0; x < D / 16; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[t][x][e] = 0.f;
    }

    for (int i = 0; i < it.n; ++i, ++step) {
      const uint32_t s = step % G::STAGES, use = step / G::STAGES;
      // after a timeout the warp still meets the others at every piece's barriers
      ok = ok && mbar_wait_warp(full + 8 * s, use & 1, p.status, &abort_flag);
      if (!ok) break;
#pragma unroll
      for (int group = 0; group < G::GROUPS; ++group) {
        const int j0 = (tile + i) * TK + 64 * group + 16 * warp;
        if (j0 >= sp.len || j0 + 16 <= sp.first) continue;
        const uint32_t kb = base + s * G::STAGE + 64 * 128 * group + k_row;
        const uint32_t vb = base + s * G::STAGE + G::HALF + 64 * 128 * group + v_row;
        float c[NT][4] = {};
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          uint32_t kf[4];
          ldsm4(kb + (ks >> 2) * G::SLAB + (((uint32_t)(2 * (ks & 3)) + k_add) ^ sw) * 16u, kf);
#pragma unroll
          for (int t = 0; t < NT; ++t) mma16816(c[t], kf, q[t][ks][0], q[t][ks][1]);
        }
        // live keys: of the scores this lane's j0 + gq + 8 k, of V's fragments the
        // pairs j0 + 8 k + 2 tq
        const bool all = !by_pos && j0 >= sp.first && j0 + 16 <= sp.len;
        bool live[2] = {true, true};
        uint32_t keep[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};
        if (!all) {
          auto is_live = [&](int j) { return j >= sp.first && j < sp.len && (!by_pos || pos[j] > oldest); };
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            live[k] = is_live(j0 + gq + 8 * k);
            const int j = j0 + 8 * k + 2 * tq;
            keep[k] = (is_live(j) ? 0xFFFFu : 0u) | (is_live(j + 1) ? 0xFFFF0000u : 0u);
          }
        }
        bool grow = false, poly = false;
        if constexpr (has_poly(METHOD)) {
          float am = 0.f;
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) am = fmax3_abs(am, c[t][2 * k], c[t][2 * k + 1]);
          poly = __all_sync(0xFFFFFFFFu, am <= p.cap.xmax && p.cap.xmax > 0.f);
        }
        float mx[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float x[2];
            if (has_poly(METHOD) && poly) {
              f2_split(poly_cap2<METHOD>(f2(c[t][2 * k], c[t][2 * k + 1]), p.cap), x[0], x[1]);
            } else {
              x[0] = any_cap<METHOD>(c[t][2 * k], p.cap);
              x[1] = any_cap<METHOD>(c[t][2 * k + 1], p.cap);
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) c[t][2 * k + e] = live[k] ? x[e] * temp : -INFINITY;
          }
          if (p.scores) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int h = 8 * t + 2 * tq + e;
              float* sc = p.scores + ((size_t)b * p.Hq + hg.h0 + h) * p.max_len + j0 + gq;
#pragma unroll
              for (int k = 0; k < 2; ++k)
                if (h < hg.count && j0 + gq + 8 * k < sp.len) sc[8 * k] = c[t][2 * k + e];
            }
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(c[t][e], c[t][2 + e]);
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, x));
            mx[t][e] = top;
            grow = grow || top > m[t][e] + kSlack;
          }
        }
        if (__any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float top = fmaxf(m[t][e], mx[t][e]);
              const float scale = top == -INFINITY ? 1.f : __expf(m[t][e] - top);
              m[t][e] = top;
              l[t][e] *= scale;
#pragma unroll
              for (int x = 0; x < D / 16; ++x) {
                o[t][x][e] *= scale;
                o[t][x][2 + e] *= scale;
              }
            }
        }
        uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float r0 = m[t][0] == -INFINITY ? 0.f : m[t][0], r1 = m[t][1] == -INFINITY ? 0.f : m[t][1];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float p0 = __expf(c[t][2 * k] - r0), p1 = __expf(c[t][2 * k + 1] - r1);
            l[t][0] += p0;
            l[t][1] += p1;
            split_bf16(p0, p1, hi[t][k], lo[t][k]);
            hi[t][k] = transpose8(hi[t][k]);
            lo[t][k] = transpose8(lo[t][k]);
          }
        }
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          uint32_t vf[4];
          ldsm4_t(vb + (x >> 2) * G::SLAB + (((uint32_t)(2 * (x & 3)) + v_add) ^ sw) * 16u, vf);
          if (!all) {  // whatever a dead slot holds, NaN too, stays out
            vf[0] &= keep[0];
            vf[1] &= keep[0];
            vf[2] &= keep[1];
            vf[3] &= keep[1];
          }
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            mma16816(o[t][x], vf, hi[t][0], hi[t][1]);
            mma16816(o[t][x], vf, lo[t][0], lo[t][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty + 8 * s);
    }
    // ---------------------------------------------------------- end of a piece
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[t][e] += __shfl_xor_sync(0xFFFFFFFFu, l[t][e], x);
    const bool final_piece = it.u >= it.end;
    for (int g0 = 0; g0 < hg.count; g0 += 4) {
      // the buffer is free: the writing warp took the last round of it (in the last
      // piece: all of these warps did, at the barrier below)
      if (round > 0 && (g0 == 0 || !final_piece))
        ok = mbar_wait_warp(m_empty, (round - 1) & 1, p.status, &abort_flag) && ok;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int h = 8 * t + 2 * tq + e - g0;
          if (h >= 0 && h < 4) {
            if (gq == 0) {
              s_m[4 * warp + h] = m[t][e];
              s_l[4 * warp + h] = l[t][e];
            }
#pragma unroll
            for (int x = 0; x < D / 16; ++x) {
              merge[(warp * 4 + h) * D + 16 * x + gq] = o[t][x][e];
              merge[(warp * 4 + h) * D + 16 * x + gq + 8] = o[t][x][2 + e];
            }
          }
        }
      if (!final_piece) {
        __syncwarp();
        if (lane == 0) mbar_arrive(m_full);
        ++round;
      } else {
        named_bar_sync(1, kConsumers * 32);
        if (g0 + warp < hg.count) finish_head(hg, g0, warp);
        named_bar_sync(1, kConsumers * 32);
      }
    }
    if (final_piece && !it.whole) {
      const Pieces pc(it);
      if (threadIdx.x == 0) join_flag = count_piece(p, pc);
      named_bar_sync(1, kConsumers * 32);
      if (join_flag) join_pieces<__nv_bfloat16, D, 4>(p, pc, b, hg, warp, lane, 1, merge, s_join);
    }
  }
}

// 2-D map over the cache's rows [num_pages * Hkv * page_size][D]: boxes of 64
// columns x the rows a tile has of a page, 128-byte swizzle.
cudaError_t make_rows_map(CUtensorMap* map, const void* base, const CacheParams& p, int tile) {
  const cuuint64_t dims[2] = {(cuuint64_t)p.D, (cuuint64_t)p.num_pages * p.Hkv * p.page_size};
  const cuuint64_t strides[1] = {(cuuint64_t)p.D * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)(p.page_size < tile ? p.page_size : tile)};
  return encode_bf16_map(map, base, 2, dims, strides, box);
}

template <int D, int METHOD, int NT>
cudaError_t run_tc(const CacheParams& p, cudaStream_t s) {
  auto* k = decode_tc_kernel<D, METHOD, NT>;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(k), (Geo<D, NT>::SMEM), done);
  CUtensorMap mk, mv;
  if (e == cudaSuccess) e = make_rows_map(&mk, p.k, p, tile_keys<D>());
  if (e == cudaSuccess) e = make_rows_map(&mv, p.v, p, tile_keys<D>());
  if (e != cudaSuccess) return e;
  return launch_pdl(k, dim3(p.ctas), dim3(kThreads), (Geo<D, NT>::SMEM), s, mk, mv, p);
}

template <int D, int METHOD>
cudaError_t run_rows(const CacheParams& p, cudaStream_t s) {
  return p.G <= 8 ? run_tc<D, METHOD, 1>(p, s) : run_tc<D, METHOD, 2>(p, s);
}

template <int D>
cudaError_t run_cap(const CacheParams& p, cudaStream_t s) {
  switch (p.method) {
    case CAPATTN_CAP_TANH: return run_rows<D, CAPATTN_CAP_TANH>(p, s);
    case CAPATTN_CAP_SOFT_SIGN: return run_rows<D, CAPATTN_CAP_SOFT_SIGN>(p, s);
    case CAPATTN_CAP_ALSC: return run_rows<D, CAPATTN_CAP_ALSC>(p, s);
    default: return run_rows<D, CAPATTN_CAP_NONE>(p, s);
  }
}

}  // namespace

cudaError_t launch_decode_tc(const CacheParams& p0, cudaStream_t s) {
  CacheParams p = p0;
  const int tk = 8192 / p.D;
  const int64_t most = (int64_t)p.B * p.VH * ((p.max_len + tk - 1) / tk);
  p.ctas = (int)(most < 152 * 2 ? most : 152 * 2);
  p.min_tiles = 2;
  return p.D == 64 ? run_cap<64>(p, s) : run_cap<128>(p, s);
}

}  // namespace capattn
