// C-ABI entry points of the paged cache (capattn_cache.h): argument checks,
// workspace layout and the launches.
#include <float.h>
#include <math.h>
#include <string.h>

#include "cache_internal.h"
#include "near_soft_sign.h"
#include "near_tanh.h"
#include "softmax_elem.cuh"

namespace capattn {
namespace {

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
int heads_of(const capattn_cache_config& c) { return c.Hq / c.Hkv; }
int max_len_of(const capattn_cache_config& c) { return c.max_pages * c.page_size; }
int elem(int dtype) { return dtype == CAPATTN_BF16 ? 2 : 4; }

capattn_status check_config(const capattn_cache_config* c) {
  if (!c || c->struct_size != sizeof(capattn_cache_config)) return CAPATTN_ERR_INVALID_ARG;
  if (c->B < 1 || c->Hq < 1 || c->Hkv < 1 || c->D < 1 || c->Hq % c->Hkv) return CAPATTN_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->page_size < 1 || c->max_pages < 1) return CAPATTN_ERR_INVALID_ARG;
  if (c->dtype != CAPATTN_BF16 && c->dtype != CAPATTN_FP32) return CAPATTN_ERR_INVALID_ARG;
  if (c->cap_method < CAPATTN_CAP_NONE || c->cap_method > CAPATTN_CAP_ALSC) return CAPATTN_ERR_INVALID_ARG;
  if (!isfinite(c->sm_scale) || !isfinite(c->cap) || !isfinite(c->alpha) || !isfinite(c->beta))
    return CAPATTN_ERR_INVALID_ARG;
  if (c->window_len < 0) return CAPATTN_ERR_INVALID_ARG;
  if (c->D != 64 && c->D != 128) return CAPATTN_ERR_UNSUPPORTED;
  if (c->page_size < 8 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)))
    return CAPATTN_ERR_UNSUPPORTED;
  // slots and cache rows are 32-bit indices (offsets in bytes are 64-bit)
  if ((int64_t)c->max_pages * c->page_size > (1ll << 30)) return CAPATTN_ERR_UNSUPPORTED;
  if ((int64_t)c->num_pages * c->Hkv * c->page_size > (1ll << 31) - 1) return CAPATTN_ERR_UNSUPPORTED;
  // units of work of a decode (64-key tiles) and (sequence, head) rows are 32-bit too
  if ((int64_t)c->B * c->Hq * (max_len_of(*c) / 32 + 4) > (1ll << 31) - 1) return CAPATTN_ERR_UNSUPPORTED;
  return CAPATTN_OK;
}

}  // namespace

ExactCap exact_cap_of(int method, float cap_in, float alpha, float beta, float sm_scale, int* active) {
  ExactCap k;
  memset(&k, 0, sizeof(k));
  *active = cap_in > 0.f ? method : CAPATTN_CAP_NONE;
  const double cap = cap_in > 0.f ? (double)cap_in : 1.0;
  k.sm_scale = sm_scale;
  k.cap = (float)cap;
  k.inv_cap = (float)(1.0 / cap);
  if (*active == CAPATTN_CAP_TANH) {
    // cap tanh(in X): the odd polynomial of softmax_elem.cuh with both scales folded in
    const double in = (double)sm_scale / cap, w = in * in;
    const double c[5] = {1.0, kTanhC0, kTanhC1, kTanhC2, kTanhC3};
    double f = cap * in;
    for (int i = 0; i < 5; ++i, f *= w) k.poly[i] = (float)(c[i] * f);
    near_tanh_fit(cap, in, k.near.c);
    // usable while the last coefficient is a normal number
    k.near.xmax = fabsf(k.near.c[2]) >= 1e-30f && isfinite(k.near.c[2]) ? (float)(kNearTanh / fabs(in)) : 0.f;
    k.xmax = fabsf(k.poly[4]) >= 1e-30f && isfinite(k.poly[4]) ? (float)(kTanhPolyMaxU / fabs(in)) : 0.f;
  } else if (*active == CAPATTN_CAP_SOFT_SIGN) {
    near_soft_sign_fit(cap, sm_scale, k.poly);
    k.xmax = fabsf(k.poly[6]) >= 1e-30f && isfinite(k.poly[6]) ? (float)(kNearSoftSign * cap / fabs((double)sm_scale)) : 0.f;
  } else if (*active == CAPATTN_CAP_ALSC) {
    const double ab = (double)alpha * (double)beta;
    const double sb = 1.0 / (1.0 + exp(-ab));
    k.alsc.a = (float)((double)alpha / cap);
    k.alsc.out = (float)(cap / (sb * (1.0 - sb) + 1e-12));
    k.alsc.sb = (float)sb;
    k.alsc.one_minus_sb = (float)(1.0 / (1.0 + exp(ab)));
    k.alsc.eb = (float)fmin(exp(ab), (double)FLT_MAX);
    k.alsc.emb = (float)fmin(exp(-ab), (double)FLT_MAX);
    capattn_config c;  // the fit asks for a whole configuration; the shape plays no part
    memset(&c, 0, sizeof(c));
    c.struct_size = sizeof(c);
    c.cap_method = method;
    c.cap = cap_in; c.alpha = alpha; c.beta = beta; c.sm_scale = sm_scale;
    c.q_heads_per_kv_head = c.B = c.L = c.Hq = c.Hkv = 1;
    c.D = 64;
    bool fine = capattn_debug_alsc_poly(&c, k.poly, &k.xmax) == CAPATTN_OK && isfinite(k.xmax);
    for (int i = 0; i < 7; ++i) {
      k.poly[i] *= k.alsc.out;
      fine = fine && isfinite(k.poly[i]) && (fabsf(k.poly[i]) >= 1e-30f || k.poly[i] == 0.f);
    }
    if (!fine) k.xmax = 0.f;
  }
  return k;
}

namespace {

CacheWorkspace layout(const capattn_cache_config& c, int call) {
  CacheWorkspace w;
  memset(&w, 0, sizeof(w));
  size_t at = kCacheHeaderBytes;
  const size_t rows = (size_t)c.B * c.Hkv, max_len = max_len_of(c);
  if (call == CAPATTN_CACHE_DECODE || call == CAPATTN_CACHE_DECODE_WEIGHTS) {
    const size_t slots = 2 * (size_t)kDecodeMaxCtas;
    w.part_ml_off = at;
    at = up256(at + slots * kDecodeHeads * sizeof(float2));
    w.part_o_off = at;
    at = up256(at + slots * kDecodeHeads * c.D * sizeof(float));
    if (call == CAPATTN_CACHE_DECODE_WEIGHTS) {
      w.scores_off = at;
      at = up256(at + (size_t)c.B * c.Hq * max_len * sizeof(float));
    }
  } else if (call == CAPATTN_CACHE_EVICT) {
    w.counts_off = at;
    at = up256(at + rows * sizeof(int2));
    w.moves_off = at;
    at = up256(at + rows * max_len * sizeof(int32_t));
    w.row_src_off = at;
    at = up256(at + rows * max_len * sizeof(int32_t));
  }
  w.total = at;
  return w;
}

capattn_status check_workspace(const capattn_cache_config& c, const void* ws, size_t bytes, int call) {
  if (!ws || !aligned(ws, 256) || bytes < layout(c, call).total) return CAPATTN_ERR_WORKSPACE;
  return CAPATTN_OK;
}

CacheParams params_of(const capattn_cache_config& c, void* ws, int call) {
  CacheParams p;
  memset(&p, 0, sizeof(p));
  p.B = c.B; p.Hq = c.Hq; p.Hkv = c.Hkv; p.D = c.D; p.G = heads_of(c);
  p.page_size = c.page_size;
  while ((1 << p.page_shift) < c.page_size) ++p.page_shift;
  p.max_pages = c.max_pages; p.num_pages = c.num_pages; p.max_len = max_len_of(c);
  p.HG = (p.G + kDecodeHeads - 1) / kDecodeHeads;
  p.VH = p.Hkv * p.HG;
  p.sm_scale = c.sm_scale;
  p.window_len = c.window_len;
  p.cap = exact_cap_of(c.cap_method, c.cap, c.alpha, c.beta, c.sm_scale, &p.method);
  const CacheWorkspace w = layout(c, call);
  char* base = static_cast<char*>(ws);
  p.status = reinterpret_cast<uint32_t*>(base);
  p.counters = reinterpret_cast<uint32_t*>(base + kCountersOff);
  p.part_ml = reinterpret_cast<float2*>(base + w.part_ml_off);
  p.part_o = reinterpret_cast<float*>(base + w.part_o_off);
  p.scores = w.scores_off ? reinterpret_cast<float*>(base + w.scores_off) : nullptr;
  p.moves = reinterpret_cast<int32_t*>(base + w.moves_off);
  p.row_src = reinterpret_cast<int32_t*>(base + w.row_src_off);
  p.counts = reinterpret_cast<int2*>(base + w.counts_off);
  return p;
}

// Workspace of capattn_key_weights: the forward's (spans and visit maps), then
// what the bf16 kernel adds.
struct KeyWeightsWorkspace {
  size_t fwd, steps_off, counters_off, partial_off, total;
};
KeyWeightsWorkspace key_weights_layout(const capattn_config& c) {
  KeyWeightsWorkspace w;
  w.fwd = capattn_workspace_bytes(&c, CAPATTN_PASS_FWD);
  int32_t bq = 0, bk = 0;
  capattn_tile_sizes(&c, &bq, &bk);
  const size_t nk = ((c.Lk > 0 ? c.Lk : c.L) + bk - 1) / bk;
  w.steps_off = w.fwd;
  w.counters_off = up256(w.steps_off + sizeof(int32_t) * c.B * nk);
  w.partial_off = up256(w.counters_off + sizeof(uint32_t) * kWeightCtas);
  w.total = up256(w.partial_off + sizeof(float) * 2 * kWeightCtas * 128);
  return w;
}

capattn_status of(cudaError_t e) { return e == cudaSuccess ? CAPATTN_OK : CAPATTN_ERR_CUDA; }

// A row stride of [heads, D] rows: whole 16-byte units, no overlap.
bool good_stride(int64_t stride, int heads, int D, int dtype) {
  return stride >= (int64_t)heads * D && stride % (16 / elem(dtype)) == 0;
}

}  // namespace
}  // namespace capattn

using namespace capattn;

extern "C" {

capattn_status capattn_cache_validate_config(const capattn_cache_config* cfg) { return check_config(cfg); }

size_t capattn_cache_workspace_bytes(const capattn_cache_config* cfg, int call) {
  if (check_config(cfg) != CAPATTN_OK || call < CAPATTN_CACHE_APPEND || call > CAPATTN_CACHE_EVICT) return 0;
  return layout(*cfg, call).total;
}

capattn_status capattn_cache_append(const capattn_cache_config* cfg, const void* k_new, const void* v_new,
                                    int64_t k_row_stride, int64_t v_row_stride, int32_t n_rows,
                                    const int32_t* cu_new, void* k_cache, void* v_cache,
                                    const int32_t* table, const int32_t* lens, float* weights,
                                    int32_t* pos, const int32_t* qpos, void* workspace,
                                    size_t workspace_bytes, cudaStream_t stream) {
  capattn_status st = check_config(cfg);
  if (st != CAPATTN_OK) return st;
  if (n_rows < 0 || (!cu_new && n_rows != cfg->B)) return CAPATTN_ERR_INVALID_ARG;
  if (n_rows > 0 && (!k_new || !v_new)) return CAPATTN_ERR_INVALID_ARG;
  if (!k_cache || !v_cache || !table || !lens || (pos && !qpos)) return CAPATTN_ERR_INVALID_ARG;
  if (!good_stride(k_row_stride, cfg->Hkv, cfg->D, cfg->dtype) ||
      !good_stride(v_row_stride, cfg->Hkv, cfg->D, cfg->dtype))
    return CAPATTN_ERR_INVALID_ARG;
  const void* ptrs[] = {k_new, v_new, cu_new, k_cache, v_cache, table, lens, weights, pos, qpos};
  for (const void* ptr : ptrs)
    if (ptr && !aligned(ptr, 16)) return CAPATTN_ERR_INVALID_ARG;
  st = check_workspace(*cfg, workspace, workspace_bytes, CAPATTN_CACHE_APPEND);
  if (st != CAPATTN_OK) return st;
  if (n_rows == 0) return CAPATTN_OK;
  CacheParams p = params_of(*cfg, workspace, CAPATTN_CACHE_APPEND);
  p.k_new = k_new; p.v_new = v_new; p.k_new_stride = k_row_stride; p.v_new_stride = v_row_stride;
  p.n_rows = n_rows; p.cu_new = cu_new; p.k = k_cache; p.v = v_cache; p.table = table; p.lens = lens;
  p.weights = weights; p.pos = pos; p.qpos = qpos;
  return of(launch_cache_append(p, cfg->dtype, stream));
}

capattn_status capattn_cache_decode(const capattn_cache_config* cfg, const void* q, int64_t q_row_stride,
                                    const void* k_cache, const void* v_cache, const int32_t* table,
                                    const int32_t* lens, const float* temp, const int32_t* pos,
                                    const int32_t* qpos, void* o, float* lse, float* weights,
                                    void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  capattn_status st = check_config(cfg);
  if (st != CAPATTN_OK) return st;
  if (!q || !k_cache || !v_cache || !table || !lens || !o || !lse || (pos && !qpos))
    return CAPATTN_ERR_INVALID_ARG;
  if (!good_stride(q_row_stride, cfg->Hq, cfg->D, cfg->dtype)) return CAPATTN_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k_cache, v_cache, table, lens, temp, pos, qpos, o, lse, weights};
  for (const void* ptr : ptrs)
    if (ptr && !aligned(ptr, 16)) return CAPATTN_ERR_INVALID_ARG;
  const int call = weights ? CAPATTN_CACHE_DECODE_WEIGHTS : CAPATTN_CACHE_DECODE;
  st = check_workspace(*cfg, workspace, workspace_bytes, call);
  if (st != CAPATTN_OK) return st;
  CacheParams p = params_of(*cfg, workspace, call);
  p.q = q; p.q_stride = q_row_stride; p.k = const_cast<void*>(k_cache); p.v = const_cast<void*>(v_cache);
  p.table = table; p.lens = lens; p.temp = temp; p.pos = const_cast<int32_t*>(pos); p.qpos = qpos;
  p.o = o; p.lse = lse; p.weights = weights;
  return of(launch_cache_decode(p, cfg->dtype, stream));
}

capattn_status capattn_cache_evict(const capattn_cache_config* cfg, int32_t budget, int32_t keep_first,
                                   int32_t keep_last, void* k_cache, void* v_cache, const int32_t* table,
                                   const int32_t* lens, const float* weights, const int32_t* pos,
                                   const int32_t* qpos, int32_t* lens_out, float* weights_out,
                                   int32_t* pos_out, int32_t* src, void* workspace,
                                   size_t workspace_bytes, cudaStream_t stream) {
  capattn_status st = check_config(cfg);
  if (st != CAPATTN_OK) return st;
  if (budget < 1 || budget > max_len_of(*cfg) || keep_first < 0 || keep_last < 0 ||
      keep_first > budget - keep_last)
    return CAPATTN_ERR_INVALID_ARG;
  if (!k_cache || !v_cache || !table || !lens || !weights || !lens_out || !weights_out)
    return CAPATTN_ERR_INVALID_ARG;
  if ((pos && (!qpos || !pos_out)) || (!pos && pos_out)) return CAPATTN_ERR_INVALID_ARG;
  const void* ptrs[] = {k_cache, v_cache, table, lens, weights, pos, qpos, lens_out, weights_out, pos_out, src};
  for (const void* ptr : ptrs)
    if (ptr && !aligned(ptr, 16)) return CAPATTN_ERR_INVALID_ARG;
  st = check_workspace(*cfg, workspace, workspace_bytes, CAPATTN_CACHE_EVICT);
  if (st != CAPATTN_OK) return st;
  CacheParams p = params_of(*cfg, workspace, CAPATTN_CACHE_EVICT);
  p.budget = budget; p.keep_first = keep_first; p.keep_last = keep_last;
  p.k = k_cache; p.v = v_cache; p.table = table; p.lens = lens; p.weights = const_cast<float*>(weights);
  p.pos = const_cast<int32_t*>(pos); p.qpos = qpos; p.lens_out = lens_out; p.weights_out = weights_out;
  p.pos_out = pos_out;
  p.src = src ? src : p.row_src;
  return of(launch_cache_evict(p, cfg->dtype, stream));
}

size_t capattn_key_weights_workspace_bytes(const capattn_config* cfg) {
  return capattn_validate_config(cfg) == CAPATTN_OK ? key_weights_layout(*cfg).total : 0;
}

capattn_status capattn_key_weights(const capattn_config* cfg, const void* q, const void* k,
                                   const float* lse, const float* temp, const int32_t* seg,
                                   const int32_t* bounds, const int32_t* rows, float* w,
                                   int64_t w_row_stride, void* workspace, size_t workspace_bytes,
                                   cudaStream_t stream) {
  capattn_status st = capattn_validate_config(cfg);
  if (st != CAPATTN_OK) return st;
  if (!q || !k || !lse || !w) return CAPATTN_ERR_INVALID_ARG;
  const int32_t Lk = cfg->Lk > 0 ? cfg->Lk : cfg->L;
  if (Lk != cfg->L && (seg || bounds)) return CAPATTN_ERR_INVALID_ARG;
  if (w_row_stride < Lk) return CAPATTN_ERR_INVALID_ARG;
  const void* ptrs[] = {q, k, lse, temp, seg, bounds, rows, w};
  for (const void* ptr : ptrs)
    if (ptr && !aligned(ptr, 16)) return CAPATTN_ERR_INVALID_ARG;
  const KeyWeightsWorkspace kl = key_weights_layout(*cfg);
  if (!workspace || !aligned(workspace, 256) || workspace_bytes < kl.total) return CAPATTN_ERR_WORKSPACE;
  Params p;
  memset(&p, 0, sizeof(p));
  p.B = cfg->B; p.L = cfg->L; p.Lk = Lk; p.Hq = cfg->Hq; p.Hkv = cfg->Hkv; p.D = cfg->D;
  p.G = cfg->q_heads_per_kv_head;
  capattn_tile_sizes(cfg, &p.block_q, &p.block_kv);
  p.nq = (p.L + p.block_q - 1) / p.block_q;
  p.nk = (p.Lk + p.block_kv - 1) / p.block_kv;
  p.wq = (p.nq + 31) / 32;
  p.wk = (p.nk + 31) / 32;
  p.sm_scale = cfg->sm_scale;
  p.causal = cfg->causal ? 1 : 0;
  p.window_len = cfg->window_len;
  KeyWeightsParams kw;
  kw.cap = exact_cap_of(cfg->cap_method, cfg->cap, cfg->alpha, cfg->beta, cfg->sm_scale, &p.cap.method);
  kw.rows = rows; kw.w = w; kw.w_stride = w_row_stride;
  const WorkspaceLayout l = workspace_layout(*cfg, p.block_q, p.block_kv);
  char* base = static_cast<char*>(workspace);
  p.status = reinterpret_cast<uint32_t*>(base + l.status_off);
  p.fwd_work = reinterpret_cast<uint32_t*>(base + l.status_off + 192);
  p.rowinfo = reinterpret_cast<int4*>(base + l.rowinfo_off);
  p.qmap = reinterpret_cast<uint32_t*>(base + l.qmap_off);
  p.kmap = reinterpret_cast<uint32_t*>(base + l.kmap_off);
  p.qfull = reinterpret_cast<int2*>(base + l.qfull_off);
  p.q = q; p.k = k; p.lse = const_cast<float*>(lse); p.temp = temp; p.seg = seg; p.bounds = bounds;
  kw.steps = reinterpret_cast<int32_t*>(base + kl.steps_off);
  kw.counters = reinterpret_cast<uint32_t*>(base + kl.counters_off);
  kw.partial = reinterpret_cast<float*>(base + kl.partial_off);
  // bf16 builds its own key-tile map, with the steps it splits
  cudaError_t e = launch_prepass(p, true, cfg->dtype != CAPATTN_BF16, stream);
  if (e != cudaSuccess) return of(e);
  return of(launch_key_weights(p, kw, cfg->dtype, stream));
}

}  // extern "C"
