// Internal interfaces of the paged cache's calls (capattn_cache.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/capattn_cache.h"
#include "capattn_internal.h"

namespace capattn {

// Status bits of the cache's calls (beside those of status_bits.h).
constexpr uint32_t kStatusBadLensBit = 32u;     // a length outside [0, max_len]
constexpr uint32_t kStatusBadPageBit = 64u;     // a page outside [0, num_pages)
constexpr uint32_t kStatusBadNewRowsBit = 128u; // cu_new decreases or leaves [0, n_rows], or more new rows than lens
constexpr uint32_t kStatusBadRowsBit = 256u;    // rows outside 0 <= lo <= hi <= L

// Constants of a cap in the forms of cache_math.cuh, for raw scores X = <q, k>.
struct AlscCap {
  float a;                   // d = a * s
  float out;                 // cap / denom
  float sb, one_minus_sb;    // sigma(alpha beta) and 1 - sigma
  float eb, emb;             // e^(alpha beta), e^(-alpha beta)
};
// cap tanh(in X) = X (c[0] + z (c[1] + z c[2])), z = X^2, for |X| <= xmax (0: none)
struct NearTanh {
  float c[3];
  float xmax;
};
struct ExactCap {
  float sm_scale;
  float cap, inv_cap;        // tanh, soft_sign
  union {
    AlscCap alsc;
    NearTanh near;
  };
  // cap(sm_scale X) as a polynomial for |X| <= xmax (0: none): tanh
  // X (c0 + z (c1 + z (c2 + z (c3 + z c4)))), z = X^2; alsc X (c0 + X (c1 + .. + X c6))
  float poly[7];
  float xmax;
};

struct CacheParams {
  const void* q;
  int64_t q_stride;          // elements
  const void* k_new;
  const void* v_new;
  int64_t k_new_stride, v_new_stride;
  int32_t n_rows;
  const int32_t* cu_new;
  void* k;                   // pages
  void* v;
  const int32_t* table;
  const int32_t* lens;
  const float* temp;
  int32_t* pos;
  const int32_t* qpos;
  float* weights;
  void* o;
  float* lse;
  // eviction
  int32_t budget, keep_first, keep_last;
  int32_t* lens_out;
  float* weights_out;
  int32_t* pos_out;
  int32_t* src;
  // workspace pieces
  uint32_t* status;
  uint32_t* counters;        // [kDecodeMaxCtas] pieces left so far of the group that starts in a CTA
  float2* part_ml;           // [slots][16] running (max, sum) of a piece's heads
  float* part_o;             // [slots][16][D] unnormalised outputs
  float* scores;             // [B, Hq, max_len] scores of the step (decode with weights)
  int32_t* moves;            // [B, Hkv, max_len] eviction: slots that move, in order
  int32_t* row_src;          // [B, Hkv, budget] eviction: src when the caller wants none
  int2* counts;              // [B, Hkv] eviction: (moves, new length)
  // shapes
  int32_t B, Hq, Hkv, D, G, page_size, page_shift, max_pages, num_pages, max_len;
  int32_t HG, VH;            // groups of at most 16 query heads per KV head; VH = Hkv * HG
  int32_t ctas;              // CTAs of the persistent decode
  int32_t min_tiles;         // least tiles a decode CTA takes
  // method
  float sm_scale;
  int32_t window_len, method;
  ExactCap cap;
};

// Heads a decode CTA handles at once (the columns of two tensor-core tiles).
constexpr int kDecodeHeads = 16;
// Most CTAs of the persistent decode (bounds its partial results).
constexpr int kDecodeMaxCtas = 152 * 4;

// Every cache workspace starts with the status word and the counters, at places
// that no configuration moves.
constexpr size_t kCacheHeaderBytes = 4096;
constexpr size_t kCountersOff = 256;
static_assert(kCountersOff + kDecodeMaxCtas * sizeof(uint32_t) <= kCacheHeaderBytes, "header too small");

struct CacheWorkspace {
  size_t part_ml_off, part_o_off, scores_off, moves_off, row_src_off, counts_off, total;
};

// Rows of capattn_key_weights beyond what Params holds.
struct KeyWeightsParams {
  const int32_t* rows;
  float* w;
  int64_t w_stride;
  ExactCap cap;
  // bf16 (workspace): steps of each (batch, key tile), counters of the split key
  // tiles, partial sums
  int32_t* steps;        // [B, nk]
  uint32_t* counters;    // [kWeightCtas]
  float* partial;        // [2 kWeightCtas][128]
};
constexpr int kWeightCtas = 152;  // CTAs of the persistent bf16 kernel

// Raises a kernel's dynamic shared memory limit, once per device (`done`: a bit a device).
inline cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
  if (bytes <= 48 * 1024) return cudaSuccess;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

cudaError_t launch_cache_append(const CacheParams& p, int dtype, cudaStream_t s);
cudaError_t launch_cache_decode(const CacheParams& p, int dtype, cudaStream_t s);
cudaError_t launch_decode_tc(const CacheParams& p, cudaStream_t s);  // bf16, without the weights pass
cudaError_t launch_cache_evict(const CacheParams& p, int dtype, cudaStream_t s);
cudaError_t launch_key_weights_tc(const Params& p, const KeyWeightsParams& w, cudaStream_t s);  // bf16
cudaError_t launch_key_weights(const Params& p, const KeyWeightsParams& w, int dtype, cudaStream_t s);

}  // namespace capattn
