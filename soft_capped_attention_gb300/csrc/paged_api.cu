// C-ABI entry points of the steps with many new tokens (capattn_paged.h): argument checks,
// workspace layout and the launches.
#include <string.h>

#include "paged_internal.h"

namespace capattn {
namespace {

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct PagedWorkspace {
  size_t ml_off, bad_off, records_off, o_off, seqs_off, total;
};
PagedWorkspace layout(const capattn_cache_config& c, int call) {
  PagedWorkspace w;
  memset(&w, 0, sizeof(w));
  size_t at = kCacheHeaderBytes;
  if (call == CAPATTN_PAGED_ATTEND) {
    w.ml_off = at;
    at = up256(at + (size_t)kAttendPartRows * sizeof(float2));
    w.bad_off = at;
    at = up256(at + (size_t)kAttendPartRows * sizeof(uint32_t));
    w.records_off = at;
    at = up256(at + (size_t)kAttendSimtCtas * sizeof(Piece));
    w.o_off = at;
    at = up256(at + (size_t)kAttendPartRows * c.D * sizeof(float));
  } else if (call == CAPATTN_PAGED_PLAN) {
    w.seqs_off = at;
    at = up256(at + kPlanCopies * (size_t)c.B * 24);
  }
  w.total = at;
  return w;
}

capattn_status check(const capattn_cache_config* cfg, const void* ws, size_t bytes, int call) {
  const capattn_status st = capattn_cache_validate_config(cfg);
  if (st != CAPATTN_OK) return st;
  if (!ws || !aligned(ws, 256) || bytes < layout(*cfg, call).total) return CAPATTN_ERR_WORKSPACE;
  return CAPATTN_OK;
}

bool all_aligned(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (p && !aligned(p, 16)) return false;
  return true;
}

CacheParams shapes_of(const capattn_cache_config& c, void* ws) {
  CacheParams p;
  memset(&p, 0, sizeof(p));
  p.B = c.B; p.Hq = c.Hq; p.Hkv = c.Hkv; p.D = c.D; p.G = c.Hq / c.Hkv;
  p.page_size = c.page_size;
  while ((1 << p.page_shift) < c.page_size) ++p.page_shift;
  p.max_pages = c.max_pages; p.num_pages = c.num_pages; p.max_len = c.max_pages * c.page_size;
  char* base = static_cast<char*>(ws);
  p.status = reinterpret_cast<uint32_t*>(base);
  return p;
}

capattn_status of(cudaError_t e) { return e == cudaSuccess ? CAPATTN_OK : CAPATTN_ERR_CUDA; }

}  // namespace
}  // namespace capattn

using namespace capattn;

extern "C" {

size_t capattn_paged_workspace_bytes(const capattn_cache_config* cfg, int call) {
  if (capattn_cache_validate_config(cfg) != CAPATTN_OK || call < CAPATTN_PAGED_ATTEND || call > CAPATTN_PAGED_ACCEPT)
    return 0;
  return layout(*cfg, call).total;
}

capattn_status capattn_paged_attend(const capattn_cache_config* cfg, const void* q, int64_t q_row_stride,
                                    int32_t n_rows, const int32_t* cu_new, const int32_t* parents,
                                    const void* k_cache, const void* v_cache, const int32_t* table,
                                    const int32_t* lens, const float* temp, const int32_t* pos,
                                    const int32_t* qpos, void* o, float* lse, void* workspace,
                                    size_t workspace_bytes, cudaStream_t stream) {
  const capattn_status st = check(cfg, workspace, workspace_bytes, CAPATTN_PAGED_ATTEND);
  if (st != CAPATTN_OK) return st;
  if (n_rows < 0 || !cu_new || !k_cache || !v_cache || !table || !lens || (pos && !qpos)) return CAPATTN_ERR_INVALID_ARG;
  if (n_rows > 0 && (!q || !o || !lse)) return CAPATTN_ERR_INVALID_ARG;
  const int elems = cfg->dtype == CAPATTN_BF16 ? 8 : 4;  // of 16 bytes
  if (q_row_stride < (int64_t)cfg->Hq * cfg->D || q_row_stride % elems) return CAPATTN_ERR_INVALID_ARG;
  if (!all_aligned({q, cu_new, parents, k_cache, v_cache, table, lens, temp, pos, qpos, o, lse}))
    return CAPATTN_ERR_INVALID_ARG;
  if (n_rows == 0) return CAPATTN_OK;
  {  // a row may be formed from q once more when o has been written
    const uintptr_t size = cfg->dtype == CAPATTN_BF16 ? 2 : 4, row = (uintptr_t)cfg->Hq * cfg->D * size;
    const uintptr_t q0 = reinterpret_cast<uintptr_t>(q), o0 = reinterpret_cast<uintptr_t>(o);
    const uintptr_t q1 = q0 + (uintptr_t)(n_rows - 1) * (uintptr_t)q_row_stride * size + row;
    if (o0 < q1 && q0 < o0 + (uintptr_t)n_rows * row) return CAPATTN_ERR_INVALID_ARG;
  }
  PagedParams p;
  memset(&p, 0, sizeof(p));
  p.c = shapes_of(*cfg, workspace);
  CacheParams& c = p.c;
  c.sm_scale = cfg->sm_scale;
  c.window_len = cfg->window_len;
  c.cap = exact_cap_of(cfg->cap_method, cfg->cap, cfg->alpha, cfg->beta, cfg->sm_scale, &c.method);
  c.q = q; c.q_stride = q_row_stride; c.k = const_cast<void*>(k_cache); c.v = const_cast<void*>(v_cache);
  c.table = table; c.lens = lens; c.temp = temp; c.o = o; c.lse = lse;
  // positions matter to a window only, and without them one that every sequence fits into is none
  c.pos = cfg->window_len > 0 ? const_cast<int32_t*>(pos) : nullptr;
  if (!pos && c.window_len > c.max_len) c.window_len = 0;
  c.qpos = qpos;
  p.cu_new = cu_new; p.n_rows = n_rows; p.parents = parents;
  const PagedWorkspace w = layout(*cfg, CAPATTN_PAGED_ATTEND);
  char* base = static_cast<char*>(workspace);
  p.redo = reinterpret_cast<uint32_t*>(base + kRedoOff);
  p.part_ml = reinterpret_cast<float2*>(base + w.ml_off);
  p.part_bad = reinterpret_cast<uint32_t*>(base + w.bad_off);
  p.records = reinterpret_cast<Piece*>(base + w.records_off);
  p.part_o = reinterpret_cast<float*>(base + w.o_off);
  // query tiles, as both kernels of the call see them
  const int rows = cfg->dtype == CAPATTN_BF16 ? kAttendRows : kAttendSimtRows;
  p.parts = (c.G + rows - 1) / rows;
  p.heads = (c.G + p.parts - 1) / p.parts;
  p.tokens = rows / p.heads;
  p.ctas = cfg->dtype == CAPATTN_FP32 && c.D == 64 ? kAttendSimtCtas : kAttendCtas;
  p.min_units = 2;
  cudaError_t e = cfg->dtype == CAPATTN_BF16 ? launch_paged_attend_tc(p, stream) : launch_paged_attend_simt(p, stream);
  if (e == cudaSuccess) e = launch_paged_finish(p, cfg->dtype, stream);
  return of(e);
}

capattn_status capattn_paged_plan(const capattn_cache_config* cfg, const int32_t* n_new, int32_t* table,
                                  const int32_t* lens, const int32_t* qpos, const int32_t* held,
                                  int32_t* free_pages, const int32_t* n_free, int32_t* lens_out,
                                  int32_t* qpos_out, int32_t* held_out, int32_t* n_free_out, int32_t n_rows,
                                  int32_t* cu_new, int64_t* slots, int32_t* positions, void* workspace,
                                  size_t workspace_bytes, cudaStream_t stream) {
  const capattn_status st = check(cfg, workspace, workspace_bytes, CAPATTN_PAGED_PLAN);
  if (st != CAPATTN_OK) return st;
  if (!n_new || !table || !lens || !held || !free_pages || !n_free || !lens_out || !held_out || !n_free_out || !cu_new)
    return CAPATTN_ERR_INVALID_ARG;
  if (n_rows < 0 || (qpos == nullptr) != (qpos_out == nullptr)) return CAPATTN_ERR_INVALID_ARG;
  if (!all_aligned({n_new, table, lens, qpos, held, free_pages, n_free, lens_out, qpos_out, held_out, n_free_out, cu_new,
                    slots, positions}))
    return CAPATTN_ERR_INVALID_ARG;
  const CacheParams c = shapes_of(*cfg, workspace);
  PlanParams p;
  memset(&p, 0, sizeof(p));
  p.n_new = n_new; p.table = table; p.lens = lens; p.qpos = qpos; p.held = held; p.n_free = n_free;
  p.free_pages = free_pages; p.lens_out = lens_out; p.qpos_out = qpos_out; p.held_out = held_out;
  p.n_free_out = n_free_out; p.n_rows = n_rows; p.cu_new = cu_new; p.slots = slots; p.positions = positions;
  p.B = c.B; p.page_size = c.page_size; p.page_shift = c.page_shift; p.max_pages = c.max_pages;
  p.num_pages = c.num_pages; p.max_len = c.max_len;
  p.seqs = static_cast<char*>(workspace) + layout(*cfg, CAPATTN_PAGED_PLAN).seqs_off;
  p.ticket = reinterpret_cast<uint32_t*>(static_cast<char*>(workspace) + kPlanTicketOff);
  p.status = c.status;
  return of(launch_paged_plan(p, stream));
}

capattn_status capattn_paged_accept(const capattn_cache_config* cfg, const int32_t* cu_new, int32_t n_rows,
                                    const int32_t* tokens, const int32_t* predicted, const int32_t* parents,
                                    int32_t width, int32_t* path, int32_t* count, int32_t* next, void* k_cache,
                                    void* v_cache, const int32_t* table, const int32_t* lens, float* weights,
                                    int32_t* pos, const int32_t* qpos, int32_t* lens_out, int32_t* qpos_out,
                                    void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  const capattn_status st = check(cfg, workspace, workspace_bytes, CAPATTN_PAGED_ACCEPT);
  if (st != CAPATTN_OK) return st;
  if (!cu_new || n_rows < 0 || width < 1 || !path || !count || !k_cache || !v_cache || !table || !lens || !lens_out)
    return CAPATTN_ERR_INVALID_ARG;
  if ((tokens == nullptr) != (predicted == nullptr) || (tokens == nullptr) != (parents == nullptr) || (!tokens && next))
    return CAPATTN_ERR_INVALID_ARG;
  if ((pos && !qpos) || (qpos == nullptr) != (qpos_out == nullptr)) return CAPATTN_ERR_INVALID_ARG;
  if (!all_aligned({cu_new, tokens, predicted, parents, path, count, next, k_cache, v_cache, table, lens, weights, pos,
                    qpos, lens_out, qpos_out}))
    return CAPATTN_ERR_INVALID_ARG;
  AcceptParams p;
  memset(&p, 0, sizeof(p));
  p.c = shapes_of(*cfg, workspace);
  p.c.k = k_cache; p.c.v = v_cache; p.c.table = table; p.c.lens = lens; p.c.weights = weights; p.c.pos = pos;
  p.c.qpos = qpos;
  p.cu_new = cu_new; p.n_rows = n_rows; p.tokens = tokens; p.predicted = predicted; p.parents = parents;
  p.width = width; p.path = path; p.count = count; p.next = next; p.lens_out = lens_out; p.qpos_out = qpos_out;
  return of(launch_paged_accept(p, cfg->dtype, stream));
}

}  // extern "C"
