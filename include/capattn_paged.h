/*
 * capattn_paged — steps with many new tokens per sequence over the paged cache of
 * capattn_cache.h: the tables and slot maps of a step from request lengths,
 * attention of whole prompts, chunks of prompts or trees of drafted tokens, and the
 * acceptance of a drafted path.  Same library (libcapattn.so), same status codes,
 * same cache and the same rules as capattn_cache.h: plain pointers, caller-owned
 * buffers, no device allocation, every call enqueues on `stream` and returns without
 * synchronising, argument errors are found on the host before anything is launched,
 * errors in device-resident data are recorded in the status word at the start of the
 * workspace (capattn_device_status).  A workspace of capattn_cache.h that is large
 * enough serves these calls too, one call at a time.
 *
 * Packed rows: cu_new [B + 1] int32, non-decreasing; rows cu_new[b] .. cu_new[b + 1] - 1
 * of n_rows are the new tokens of sequence b, in order.  lens (and qpos) count them
 * already: row i of n is slot lens[b] - n + i.  Rows before cu_new[0] and at or behind
 * cu_new[B] belong to nobody: they are not read, and outputs there stay as they were.
 *
 * A step of a program that drafts:
 *   plan (pages and lengths of the new tokens), capattn_cache_append, attend, accept;
 * a later plan gives the pages back that the rejected tokens do not need.
 *
 * Status bits that these calls add: 512 = a parent that is not an earlier row of its
 * sequence (nor -1), or a tree of more than CAPATTN_PAGED_MAX_TREE tokens (its rows stay
 * as they were); 1024 = a plan without the pages or rows that it needs, or with bad lengths,
 * held pages or stack (nothing was changed); 2048 = a path that does not increase within the sequence's
 * rows, or a bad count.  Bits 32, 64 and 128 as in capattn_cache.h.
 */
#ifndef CAPATTN_PAGED_H_
#define CAPATTN_PAGED_H_

#include "capattn_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Most new tokens of a sequence that come as a tree: a row finds its ancestors by walking up
 * from itself, which a chain of all its tokens makes a walk of that many steps per 32 slots.
 */
#define CAPATTN_PAGED_MAX_TREE 8192

enum { CAPATTN_PAGED_ATTEND = 0, CAPATTN_PAGED_PLAN = 1, CAPATTN_PAGED_ACCEPT = 2 };

/*
 * Bytes of device workspace of a call (CAPATTN_PAGED_*); 0 if cfg is invalid.  256-byte
 * aligned, its first CAPATTN_CACHE_HEADER_BYTES cleared once, as a cache workspace's.
 */
size_t capattn_paged_workspace_bytes(const capattn_cache_config* cfg, int call);

/*
 * Attention of the new tokens over their sequence's cached tokens, their own among
 * them (append them first):
 *   t_ij = temp_i * cap(sm_scale * <q_i, k_j>) over the live slots j of row i,
 *   P = softmax(t), o_i = sum_j P_ij v_j, lse_i = log sum_j exp(t_ij).
 * Live slots of row i (slot s_i = lens[b] - n + i):
 *   parents NULL: j <= s_i (a prompt, or a chunk of one, behind what the cache holds);
 *   parents [n_rows] int32: the slots before the new tokens, row i itself and its
 *   ancestors.  parents[r] is the index within the sequence's new tokens of the token
 *   that row r continues, less than its own, or -1: it continues what the cache holds.
 * window_len > 0: and position_j > position_i - window_len.  A slot's position is the
 * slot (or pos[b, g, j]; with pos, row i stands at qpos[b] - n + 1 + i); with parents
 * a new token's position is that of the first new slot plus its depth in the tree.
 * A row without live slots gives o = 0, lse = -inf.
 * q: n_rows rows of [Hq, D], row r at r * q_row_stride elements; o [n_rows, Hq, D];
 * lse [n_rows, Hq] float32; temp [n_rows] float32, nullable (1); o must not overlap q.
 * What a slot holds that is not live for a row (NaN, infinities) does not reach that row.
 * bf16: P enters the product with V as one bf16 (capattn_cache_decode keeps two): o is off by
 * 2.3e-3 of its size, 1.7e-3 of it its own rounding.
 * The result does not depend on scheduling: same inputs, same bits.
 */
capattn_status capattn_paged_attend(const capattn_cache_config* cfg, const void* q, int64_t q_row_stride,
                                    int32_t n_rows, const int32_t* cu_new, const int32_t* parents,
                                    const void* k_cache, const void* v_cache, const int32_t* table,
                                    const int32_t* lens, const float* temp, const int32_t* pos,
                                    const int32_t* qpos, void* o, float* lse, void* workspace,
                                    size_t workspace_bytes, cudaStream_t stream);

/*
 * The tables and slot maps of a step.  n_new [B] int32: tokens that each sequence is
 * about to get; negative: the sequence ends (length 0).  held [B] int32: pages that
 * sequence b owns, table[b][0 .. held[b]), at least those of its lens[b] tokens.  free_pages [num_pages] int32, n_free [1]: a
 * stack of the pages that nobody owns, free_pages[0 .. n_free).
 *   lens_out = lens + n_new (0 for one that ends), qpos_out = qpos + n_new (-1);
 *   held_out = ceil(lens_out / page_size): the pages behind that go on the stack, in the
 *   order of sequences and pages; missing ones come from its top, in the same order;
 *   cu_new [B + 1]: the sums of n_new (0 for one that ends);
 *   slots [n_rows] int64 (nullable): page * page_size + offset of each new token, so that
 *   head g's row of the cache is slots / page_size * Hkv * page_size + g * page_size +
 *   slots % page_size; positions [n_rows] int32 (nullable): its position (the slot, or
 *   with qpos qpos[b] + 1 + i); -1 in both behind the last new token.
 * Either everything is done or, when the stack holds too few pages, a sequence would
 * outgrow max_len, the new tokens do not fit n_rows or held (also one that does not reach
 * lens) or the stack are out of range, nothing: the status word says so, the outputs are what the inputs were, cu_new
 * is 0 and slots and positions are -1.  lens_out, qpos_out, held_out and n_free_out may
 * be lens, qpos, held and n_free; other overlaps are not allowed.  qpos and qpos_out
 * come together or are both NULL.  Table entries behind held_out are left as they were.
 * Sequences that share pages (a common prefix) cannot be planned: counted in held they would
 * be given back while others read them, and held names the front of the table, so they cannot
 * be left out (such a held is refused as above).
 */
capattn_status capattn_paged_plan(const capattn_cache_config* cfg, const int32_t* n_new, int32_t* table,
                                  const int32_t* lens, const int32_t* qpos, const int32_t* held,
                                  int32_t* free_pages, const int32_t* n_free, int32_t* lens_out,
                                  int32_t* qpos_out, int32_t* held_out, int32_t* n_free_out, int32_t n_rows,
                                  int32_t* cu_new, int64_t* slots, int32_t* positions, void* workspace,
                                  size_t workspace_bytes, cudaStream_t stream);

/*
 * Acceptance of a drafted path: of the n new tokens of sequence b those on the path stay,
 * moved to the front of the new slots, the others leave the cache.
 *   path [B, width] int32, strictly increasing indices of new tokens; count [B] int32,
 *   0 <= count <= min(width, n): slot lens[b] - n + path[i] goes to lens[b] - n + i for
 *   i < count (keys, values and, if given, weights), lens_out = lens - n + count; with pos
 *   the kept tokens' positions become qpos[b] - n + 1 + i and qpos_out = qpos - n + count.
 * tokens NULL: path and count are inputs.  With tokens, predicted and parents [n_rows]
 * int32 they are outputs: row 0 is accepted, and from an accepted row i the walk goes on to
 * the first row c with parents[c] == i and tokens[c] == predicted[i], up to `width` tokens;
 * path is -1 behind count, next [B] int32 (nullable) is predicted of the last accepted row
 * (-1, and count 0, for a sequence without new tokens).
 * A sequence with wrong data (lengths, rows, a path, a page that a row would leave or enter)
 * stays as it is: nothing of it moves, lens_out = lens, qpos_out = qpos; with tokens its path is
 * -1, count 0 and next -1.
 * lens_out and qpos_out may be lens and qpos.  The pages of the new tokens belong to one
 * sequence.
 */
capattn_status capattn_paged_accept(const capattn_cache_config* cfg, const int32_t* cu_new, int32_t n_rows,
                                    const int32_t* tokens, const int32_t* predicted, const int32_t* parents,
                                    int32_t width, int32_t* path, int32_t* count, int32_t* next, void* k_cache,
                                    void* v_cache, const int32_t* table, const int32_t* lens, float* weights,
                                    int32_t* pos, const int32_t* qpos, int32_t* lens_out, int32_t* qpos_out,
                                    void* workspace, size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* CAPATTN_PAGED_H_ */
