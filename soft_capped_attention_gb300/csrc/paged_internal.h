// Internal interfaces of the steps with many new tokens (capattn_paged.h).
#pragma once

#include "../../include/capattn_paged.h"
#include "cache_internal.h"

namespace capattn {

// Status bits of these calls (beside those of cache_internal.h).
constexpr uint32_t kStatusBadParentBit = 512u;
constexpr uint32_t kStatusBadPlanBit = 1024u;
constexpr uint32_t kStatusBadPathBit = 2048u;

// Whether rows of attention have to be formed once more, by themselves: a flag and a ticket in
// the workspace's header, behind the counters of capattn_cache.h's calls; both are zero
// between calls.
constexpr size_t kRedoOff = kCacheHeaderBytes - 64;
constexpr size_t kPlanTicketOff = kRedoOff + 32;  // CTAs of a plan that have ended
static_assert(kCountersOff + kDecodeMaxCtas * sizeof(uint32_t) <= kRedoOff, "header too small");

struct Piece;
struct PagedParams {
  CacheParams c;               // shapes, cache, q, temp, o, lse, status, cap
  const int32_t* cu_new;
  int32_t n_rows;
  const int32_t* parents;      // or null: a prompt
  uint32_t* redo;              // flag, ticket
  // query tiles: `tokens` tokens of `heads` query heads of one KV head, parts per KV head
  int32_t tokens, heads, parts;  // parts * heads >= G
  int32_t ctas;                // most CTAs of the persistent grid
  int32_t min_units;           // least units a CTA takes
  // partial results of query tiles that several CTAs share: slot s has rows [s * rows, (s + 1) * rows)
  float* part_o;               // [slots][rows x D] (part_at)
  float2* part_ml;             // [slots][rows]
  uint32_t* part_bad;          // [slots][rows]
  Piece* records;       // [ctas] the shared tile that begins in a CTA
};

// What one CTA does of one query tile.
struct Piece {
  int32_t b, part;         // sequence, part of the heads (KV head * parts + x)
  int32_t row0, n, base, len;
  int32_t i0, count;       // tokens [i0, i0 + count)
  int32_t tile0, steps;    // its steps' first TK slots; steps < 0: there are no more pieces
  int32_t first;           // first slot that the tile needs
  int32_t whole;
  int32_t slot;            // of its partial results
  int32_t c0, c1, late;    // CTAs that share the tile; whether it begins inside c0's range
};

// Slots of partial results: two a CTA.
constexpr int kAttendCtas = 152;       // bf16: one CTA an SM, tiles of 128 rows
constexpr int kAttendRows = 128;
constexpr int kAttendSimtCtas = 304;   // fp32: two an SM at D = 64 (one at D = 128), tiles of 64 rows
constexpr int kAttendSimtRows = 64;
constexpr int kAttendPartRows = 2 * kAttendCtas * kAttendRows;
static_assert(2 * kAttendSimtCtas * kAttendSimtRows <= kAttendPartRows, "partial results");

constexpr int kPlanCopies = 8;  // of the sequences' sums in the workspace, 24 bytes each

struct PlanParams {
  const int32_t* n_new;
  int32_t* table;
  const int32_t *lens, *qpos, *held, *n_free;
  int32_t* free_pages;
  int32_t *lens_out, *qpos_out, *held_out, *n_free_out;
  int32_t n_rows;
  int32_t* cu_new;
  int64_t* slots;
  int32_t* positions;
  int32_t B, page_size, page_shift, max_pages, num_pages, max_len;
  void* seqs;                  // workspace, for more sequences than shared memory holds
  uint32_t* status;
  uint32_t* ticket;            // zero between calls
};

struct AcceptParams {
  CacheParams c;
  const int32_t* cu_new;
  int32_t n_rows;
  const int32_t *tokens, *predicted, *parents;
  int32_t width;
  int32_t *path, *count, *next;
  int32_t *lens_out, *qpos_out;
};

cudaError_t launch_paged_attend_tc(const PagedParams& p, cudaStream_t s);  // bf16
cudaError_t launch_paged_attend_simt(const PagedParams& p, cudaStream_t s);  // fp32
cudaError_t launch_paged_finish(const PagedParams& p, int dtype, cudaStream_t s);  // after either
cudaError_t launch_paged_plan(const PlanParams& p, cudaStream_t s);
cudaError_t launch_paged_accept(const AcceptParams& p, int dtype, cudaStream_t s);

}  // namespace capattn
