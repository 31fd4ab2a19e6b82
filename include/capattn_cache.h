/*
 * capattn_cache — serving next to the training attention of capattn.h: a paged
 * key-value cache, attention of one new token per sequence over it with the
 * same caps, the attention weight that each key of a prompt received, and
 * eviction from the cache by accumulated weight.  Same library (libcapattn.so),
 * same status codes, same rules: plain pointers, caller-owned buffers, no device
 * allocation, every call enqueues on `stream` and returns without
 * synchronising, argument errors are found on the host before anything is
 * launched, and errors in device-resident data are recorded in the status word
 * at the start of the workspace (capattn_device_status reads and clears it).
 * Calls take the current device; every pointer belongs to it.
 *
 * The cache
 *   k_cache, v_cache : [num_pages, Hkv, page_size, D]  pages; a head's tokens of
 *                      a page are consecutive rows (one contiguous block)
 *   table            : [B, max_pages] int32, page of slots
 *                      [p * page_size, (p + 1) * page_size) of sequence b.  Only
 *                      the entries of pages that hold slots < lens[b] are read.
 *                      Decoding may read pages that several sequences share
 *                      (a common prefix); a page that append or evict writes
 *                      must belong to one sequence.
 *   lens             : [B] int32, tokens of each sequence, 0 .. max_len,
 *                      max_len = max_pages * page_size
 *   pos   (nullable) : [B, Hkv, max_len] int32, position in the text of the token
 *                      in each slot.  Without it a slot's position is the slot
 *                      itself.  Needed once eviction has moved tokens if a window
 *                      or keep_first / keep_last is used.
 *   qpos             : [B] int32, position of each sequence's newest token;
 *                      required with pos, ignored (lens[b] - 1) without it.
 *   weights (nullable) : [B, Hkv, max_len] float32, attention weight that the
 *                      token in each slot has received so far, summed over the
 *                      query heads of the group.
 * Slots at or behind lens[b] may hold anything (NaN included); they are never
 * used and never written but by append.
 *
 * Lengths: append and decode take lens (and qpos) as they are AFTER the new
 * tokens, so that a decoding step is: lens += 1; append; decode.
 *
 * Every tensor pointer is 16-byte aligned.  D is 64 or 128; page_size a power of
 * two from 8 to 1024 (CAPATTN_ERR_UNSUPPORTED otherwise).
 *
 * Status bits that these calls add (capattn_device_status returns
 * CAPATTN_ERR_DEVICE_DATA): 32 = a length outside [0, max_len]; 64 = a page
 * outside [0, num_pages); 128 = cu_new decreases or leaves [0, n_rows] or a
 * sequence has more new rows than lens[b]; 256 = rows of capattn_key_weights
 * outside 0 <= lo <= hi <= L.  Nothing outside the caller's buffers is read or
 * written then; the results of that sequence (after a bad cu_new: of every sequence
 * that the call gives rows) are unspecified.
 */
#ifndef CAPATTN_CACHE_H_
#define CAPATTN_CACHE_H_

#include "capattn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct capattn_cache_config {
  uint32_t struct_size;        /* sizeof(capattn_cache_config) */
  int32_t cap_method;          /* CAPATTN_CAP_*; cap > 0 activates it, as in capattn_config */
  float cap, alpha, beta;
  float sm_scale;
  int32_t window_len;          /* > 0: a key counts only if its position > qpos - window_len; 0: off */
  int32_t B, Hq, Hkv, D;       /* sequences, heads (Hq a multiple of Hkv), head dim */
  int32_t dtype;               /* CAPATTN_BF16 or CAPATTN_FP32: q, k, v, o and the cache */
  int32_t num_pages, page_size, max_pages;
} capattn_cache_config;

/* Checks a configuration without touching any pointer (same rules as the calls). */
capattn_status capattn_cache_validate_config(const capattn_cache_config* cfg);

#define CAPATTN_CACHE_HEADER_BYTES 4096

/* Calls that a cache workspace serves. */
enum { CAPATTN_CACHE_APPEND = 0, CAPATTN_CACHE_DECODE = 1, CAPATTN_CACHE_DECODE_WEIGHTS = 2,
       CAPATTN_CACHE_EVICT = 3 };

/*
 * Bytes of device workspace of a call (CAPATTN_CACHE_*); 0 if cfg is invalid.
 * 256-byte aligned.  The caller clears its first CAPATTN_CACHE_HEADER_BYTES once,
 * before its first use: they hold the device status (the first word) and counters
 * that every call leaves at zero.  It may serve calls and configurations of any
 * kind, one after another.  A workspace serves one call at a time: calls (or captured graphs) that
 * may overlap on the GPU need one each.  DECODE_WEIGHTS (a decode with weights)
 * also holds the step's scores, 4 bytes per (query head, slot).
 */
size_t capattn_cache_workspace_bytes(const capattn_cache_config* cfg, int call);

/*
 * Appends new keys and values.  k_new, v_new: n_rows rows of [Hkv, D], row r at
 * r * row_stride elements (rows of a fused projection need no copy; the stride
 * is a multiple of 16 bytes and at least Hkv * D).  cu_new [B + 1] int32,
 * nullable: the rows of sequence b are cu_new[b] .. cu_new[b + 1] - 1; NULL: row b
 * is the one new token of sequence b (n_rows == B).  Rows before cu_new[0] and at or
 * behind cu_new[B] are ignored; with n_rows == 0 the call does nothing.  The n new rows of sequence b go to slots lens[b] - n .. lens[b] - 1.
 * With weights, the new slots' weights become 0; with pos, their positions
 * qpos[b] - n + 1 .. qpos[b].
 */
capattn_status capattn_cache_append(const capattn_cache_config* cfg, const void* k_new, const void* v_new,
                                    int64_t k_row_stride, int64_t v_row_stride, int32_t n_rows,
                                    const int32_t* cu_new, void* k_cache, void* v_cache,
                                    const int32_t* table, const int32_t* lens, float* weights,
                                    int32_t* pos, const int32_t* qpos, void* workspace,
                                    size_t workspace_bytes, cudaStream_t stream);

/*
 * Attention of one query token per sequence over its cached tokens:
 *   t_j = temp_b * cap(sm_scale * <q, k_j>) over the live slots j < lens[b] (in
 *   the window: position > qpos - window_len), P = softmax(t), o = sum_j P_j v_j,
 *   lse = log sum_j exp(t_j).
 * The query stands at qpos, behind every cached token, so the causal mask of
 * capattn_fwd adds nothing here.  A sequence without live slots gives o = 0,
 * lse = -inf.  q: B rows of [Hq, D], row b at b * q_row_stride elements; o
 * [B, Hq, D]; lse [B, Hq] float32; temp [B] float32, nullable (1).
 * weights, nullable: weights[b, g, j] += sum of P_j over the query heads of group
 * g, for the live slots.  The result does not depend on scheduling: same inputs,
 * same bits.
 */
capattn_status capattn_cache_decode(const capattn_cache_config* cfg, const void* q, int64_t q_row_stride,
                                    const void* k_cache, const void* v_cache, const int32_t* table,
                                    const int32_t* lens, const float* temp, const int32_t* pos,
                                    const int32_t* qpos, void* o, float* lse, float* weights,
                                    void* workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * Evicts tokens: every (sequence, KV head) with lens[b] > budget keeps `budget`
 * of them, first the protected ones (position < keep_first or position > qpos -
 * keep_last), then those of the largest weight; ties go to the lower slot, a NaN
 * weight goes first.  keep_first + keep_last <= budget, 1 <= budget <= max_len.
 * Kept tokens in slots below the budget stay where they are; the kept ones behind
 * it move, in order, into the slots of evicted ones, in order, so that only rows
 * that have to move are copied.  lens_out [B] = min(lens, budget); weights_out and
 * pos_out (as weights and pos; pos_out only with pos) get the kept tokens' values
 * in slots < lens_out; src [B, Hkv, budget] int32 (nullable) the slot each came
 * from (-1 behind lens_out).  lens_out, weights_out and pos_out may be lens,
 * weights and pos themselves; other overlaps are not allowed.
 */
capattn_status capattn_cache_evict(const capattn_cache_config* cfg, int32_t budget, int32_t keep_first,
                                   int32_t keep_last, void* k_cache, void* v_cache, const int32_t* table,
                                   const int32_t* lens, const float* weights, const int32_t* pos,
                                   const int32_t* qpos, int32_t* lens_out, float* weights_out,
                                   int32_t* pos_out, int32_t* src, void* workspace,
                                   size_t workspace_bytes, cudaStream_t stream);

/*
 * The attention weight that each key of a prompt received, which starts the
 * cache's weights:
 *   w[b, g, j] = sum over query heads h of group g and counted rows i of
 *                P_ij = exp(t_ij - lse[b, h, i])   (0 for masked pairs)
 * with t and every mask as in capattn_fwd (cfg, temp, seg, bounds) and lse as
 * capattn_fwd wrote it for the same inputs.  rows [B, 2] int32 (nullable: all L):
 * the counted query rows rows[b][0] <= i < rows[b][1] (a padded prompt, or an
 * observation window at its end).  w: row (b, g) at (b * Hkv + g) * w_row_stride
 * floats, w_row_stride >= Lk; entries j < Lk are overwritten.  The weights are summed in
 * a fixed order.  workspace: capattn_key_weights_workspace_bytes(cfg) bytes, 256-byte
 * aligned; its first word is the device status.  A capattn_fwd of the same cfg may
 * use it too (it holds what CAPATTN_PASS_FWD asks for).
 */
size_t capattn_key_weights_workspace_bytes(const capattn_config* cfg);
capattn_status capattn_key_weights(const capattn_config* cfg, const void* q, const void* k,
                                   const float* lse, const float* temp, const int32_t* seg,
                                   const int32_t* bounds, const int32_t* rows, float* w,
                                   int64_t w_row_stride, void* workspace, size_t workspace_bytes,
                                   cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CAPATTN_CACHE_H_ */
