// sa_kv8_api.cu -- the extern "C" entry points of serving over a paged KV cache
// held in 8 bits (sa_page_plan, sa_kv8_write, sa_kv8_fwd): host-side argument
// validation and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "../../include/sparse_attn.h"
#include "sa_kv8.h"

namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
sa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? SA_OK : SA_ERR_CUDA; }

long long tokens_of(const sa_kv8_cache* c) {
  return c->layout == SA_LAYOUT_BSND ? (long long)c->batch * c->s_q : c->t_q;
}

sa_status validate_cache(const sa_kv8_cache* c) {
  if (!c) return SA_ERR_NULLPTR;
  if (c->format != SA_KV8_E4M3 && c->format != SA_KV8_INT8) return SA_ERR_PARAM;
  if (c->layout != SA_LAYOUT_BSND && c->layout != SA_LAYOUT_TND) return SA_ERR_PARAM;
  if (c->n_heads_kv < 1 || c->n_heads_kv > 65535) return SA_ERR_PARAM;
  if (c->d_qk < 16 || c->d_v < 16 || c->d_qk % 16 || c->d_v % 16 || c->d_qk > 576 || c->d_v > 512) return SA_ERR_PARAM;
  if (c->kv_shared && c->d_v > c->d_qk) return SA_ERR_PARAM;
  if (c->page_size < 1 || c->n_pages < 1 || c->max_pages < 1 || c->batch < 0) return SA_ERR_PARAM;
  // rows are numbered in 32 bits: inside the cache, and with room to spare inside a sequence
  if ((long long)c->page_size * c->n_pages >= (1ll << 31)) return SA_ERR_PARAM;
  if ((long long)c->page_size * c->max_pages > (1ll << 30)) return SA_ERR_PARAM;
  if (c->table_stride < c->max_pages) return SA_ERR_PARAM;
  if (c->layout == SA_LAYOUT_BSND ? c->s_q < 0 : c->t_q < 0) return SA_ERR_PARAM;
  const long long T = tokens_of(c);
  if (T >= (1ll << 30)) return SA_ERR_PARAM;
  if (T > 0 && c->batch > 0) {
    if (!c->k || !c->k_scale || !c->block_table || !c->seq_lens) return SA_ERR_NULLPTR;
    if (!c->kv_shared && (!c->v || !c->v_scale)) return SA_ERR_NULLPTR;
    if (c->layout == SA_LAYOUT_TND && !c->cu_seqlens_q) return SA_ERR_NULLPTR;
    if (!aligned16(c->k) || (!c->kv_shared && !aligned16(c->v))) return SA_ERR_PARAM;
  }
  if (!sa::k8_built(c->d_qk, c->d_v, c->kv_shared != 0)) return SA_ERR_UNSUPPORTED;
  return SA_OK;
}

sa::K8Cache make_cache(const sa_kv8_cache* c) {
  sa::K8Cache r;
  memset(&r, 0, sizeof(r));
  r.fmt = c->format;
  r.Hkv = c->n_heads_kv;
  r.dqk = c->d_qk;
  r.dv = c->d_v;
  r.shared = c->kv_shared ? 1 : 0;
  r.ps = c->page_size;
  r.by_ps = sa::k8_div_of(c->page_size);
  r.n_pages = c->n_pages;
  r.B = c->batch;
  r.max_pages = c->max_pages;
  r.s_q = c->s_q;
  r.T = (int)tokens_of(c);
  r.tstride = c->table_stride;
  r.k = static_cast<uint8_t*>(c->k);
  r.v = static_cast<uint8_t*>(c->kv_shared ? c->k : c->v);
  r.ks = c->k_scale;
  r.vs = c->kv_shared ? c->k_scale : c->v_scale;
  r.table = c->block_table;
  r.lens = c->seq_lens;
  r.cu = c->layout == SA_LAYOUT_TND ? c->cu_seqlens_q : nullptr;
  r.status = c->status;
  return r;
}

sa_status validate_query(const sa_kv8_cache* c, const sa_kv8_query* q) {
  sa_status st = validate_cache(c);
  if (st != SA_OK) return st;
  if (!q) return SA_ERR_NULLPTR;
  if (q->dtype != SA_DTYPE_BF16 && q->dtype != SA_DTYPE_FP16) return SA_ERR_PARAM;
  if (q->n_heads_q < 1 || q->n_heads_q % c->n_heads_kv || q->n_heads_q > 65535) return SA_ERR_PARAM;
  if (q->block_size < 1 || q->topk < 0 || q->win_left < -1 || q->flags != 0 || !isfinite(q->scale)) return SA_ERR_PARAM;
  if ((long long)q->topk * q->block_size >= (1ll << 30)) return SA_ERR_PARAM;
  if (q->q_stride < (long long)q->n_heads_q * c->d_qk || q->q_stride % 8) return SA_ERR_PARAM;
  const long long T = tokens_of(c);
  if (T * q->n_heads_q >= (1ll << 31)) return SA_ERR_PARAM;
  if (T > 0 && c->batch > 0) {
    if (!q->q || !q->o || !q->lse || (q->topk > 0 && !q->idx)) return SA_ERR_NULLPTR;
    if (!aligned16(q->q) || !aligned16(q->o)) return SA_ERR_PARAM;
  }
  return SA_OK;
}

sa::K8Fwd make_fwd(const sa_kv8_cache* c, const sa_kv8_query* q) {
  sa::K8Fwd r;
  memset(&r, 0, sizeof(r));
  r.c = make_cache(c);
  r.f16 = q->dtype == SA_DTYPE_FP16 ? 1 : 0;
  r.Hq = q->n_heads_q;
  r.G = q->n_heads_q / c->n_heads_kv;
  r.bs = q->block_size;
  r.by_bs = sa::k8_div_of(q->block_size);
  r.topk = q->topk;
  r.win = q->win_left < 0 || q->win_left > (1 << 30) ? 1 << 30 : (int)q->win_left;  // no sequence is longer
  r.scale_log2 = q->scale * 1.4426950408889634f;
  r.q = q->q;
  r.qstride = q->q_stride;
  r.idx = q->topk > 0 ? q->idx : nullptr;
  r.topk_len = q->topk > 0 ? q->topk_len : nullptr;
  r.sinks = q->sinks;
  r.o = q->o;
  r.lse = q->lse;
  return r;
}

}  // namespace

extern "C" {

sa_status sa_page_plan(const sa_page_plan_args* a, void* stream) {
  if (!a) return SA_ERR_NULLPTR;
  if (a->batch < 0 || a->batch > sa::kPlanMaxBatch || a->max_pages < 1 || a->page_size < 1 || a->n_tokens < 0 ||
      a->free_capacity < 0 || a->table_stride < a->max_pages)
    return SA_ERR_PARAM;
  if ((long long)a->max_pages * a->page_size > (1ll << 30)) return SA_ERR_PARAM;
  if (a->batch > 0 && (!a->old_lens || !a->new_lens || !a->block_table || !a->seq_lens)) return SA_ERR_NULLPTR;
  if (!a->n_free || !a->cu_seqlens_q || !a->n_free_out || !a->n_served) return SA_ERR_NULLPTR;
  if ((a->n_tokens > 0 && !a->slots) || (a->free_capacity > 0 && !a->free_pages)) return SA_ERR_NULLPTR;
  // every block reads the inputs while block 0 writes these
  if (a->n_free_out == a->n_free || a->n_served == a->n_free) return SA_ERR_PARAM;
  if (a->batch > 0 && (a->seq_lens == a->old_lens || a->seq_lens == a->new_lens || a->cu_seqlens_q == a->old_lens ||
                       a->cu_seqlens_q == a->new_lens))
    return SA_ERR_PARAM;
  sa::PagePlan p;
  memset(&p, 0, sizeof(p));
  p.B = a->batch;
  p.max_pages = a->max_pages;
  p.ps = a->page_size;
  p.T = a->n_tokens;
  p.free_cap = a->free_capacity;
  p.tstride = a->table_stride;
  p.old_lens = a->old_lens;
  p.new_lens = a->new_lens;
  p.free_pages = a->free_pages;
  p.n_free = a->n_free;
  p.table = a->block_table;
  p.seq_lens = a->seq_lens;
  p.cu = a->cu_seqlens_q;
  p.slots = reinterpret_cast<long long*>(a->slots);
  p.n_free_out = a->n_free_out;
  p.n_served = a->n_served;
  return cuda_status(sa::launch_page_plan(p, static_cast<cudaStream_t>(stream)));
}

sa_status sa_kv8_write(const sa_kv8_cache* cache, const sa_kv8_rows* rows, void* stream) {
  sa_status st = validate_cache(cache);
  if (st != SA_OK) return st;
  if (!rows) return SA_ERR_NULLPTR;
  if (rows->dtype != SA_DTYPE_BF16 && rows->dtype != SA_DTYPE_FP16) return SA_ERR_PARAM;
  const bool sep = !cache->kv_shared;
  // a page's rows of a head are counted in 32 bits, by pieces of 8 elements (d_v is at most d_qk in every built pair)
  if ((long long)cache->page_size * (cache->d_qk / 8) > (1ll << 30)) return SA_ERR_PARAM;
  if (rows->k_stride < (long long)cache->n_heads_kv * cache->d_qk || rows->k_stride % 8) return SA_ERR_PARAM;
  if (sep && (rows->v_stride < (long long)cache->n_heads_kv * cache->d_v || rows->v_stride % 8)) return SA_ERR_PARAM;
  if (tokens_of(cache) == 0 || cache->batch == 0) return SA_OK;
  if (!rows->k || (sep && !rows->v)) return SA_ERR_NULLPTR;
  if (!aligned16(rows->k) || (sep && !aligned16(rows->v))) return SA_ERR_PARAM;
  sa::K8Write w;
  memset(&w, 0, sizeof(w));
  w.c = make_cache(cache);
  w.f16 = rows->dtype == SA_DTYPE_FP16 ? 1 : 0;
  w.k = rows->k;
  w.v = rows->v;
  w.kstride = rows->k_stride;
  w.vstride = rows->v_stride;
  return cuda_status(sa::launch_kv8_write(w, static_cast<cudaStream_t>(stream)));
}

sa_status sa_kv8_fwd_get_workspace_size(const sa_kv8_cache* cache, const sa_kv8_query* query, size_t* ws_bytes) {
  if (!ws_bytes) return SA_ERR_NULLPTR;
  sa_status st = validate_query(cache, query);
  if (st != SA_OK) return st;
  *ws_bytes = sa::k8_fwd_workspace(make_fwd(cache, query));
  return SA_OK;
}

sa_status sa_kv8_fwd(const sa_kv8_cache* cache, const sa_kv8_query* query, void* ws, size_t ws_bytes, void* stream) {
  sa_status st = validate_query(cache, query);
  if (st != SA_OK) return st;
  if (tokens_of(cache) == 0 || cache->batch == 0) return SA_OK;
  sa::K8Fwd a = make_fwd(cache, query);
  const size_t need = sa::k8_fwd_workspace(a);
  if (need && (!ws || ws_bytes < need)) return SA_ERR_WORKSPACE;
  if (need && !aligned16(ws)) return SA_ERR_PARAM;
  return cuda_status(sa::launch_kv8_fwd(a, ws, static_cast<cudaStream_t>(stream)));
}

sa_status sa_selftest_kv8_give_up(const sa_kv8_cache* cache, const sa_kv8_query* query, int32_t warp, int32_t wait,
                                  int32_t chunk, void* ws, size_t ws_bytes, void* stream) {
  sa_status st = validate_query(cache, query);
  if (st != SA_OK) return st;
  if (warp < 0 || warp > 8 || wait < 0 || wait > 8 || (warp == 8) != (wait < 3) || chunk < 0) return SA_ERR_PARAM;
  sa::K8Fwd a = make_fwd(cache, query);
  const size_t need = sa::k8_fwd_workspace(a);
  if (need && (!ws || ws_bytes < need)) return SA_ERR_WORKSPACE;
  if (need && !aligned16(ws)) return SA_ERR_PARAM;
  a.give_up_warp = warp;
  a.give_up_wait = wait;
  a.give_up_chunk = chunk;
  const cudaError_t e = sa::launch_kv8_give_up(a, ws, static_cast<cudaStream_t>(stream));
  return e == cudaErrorNotSupported ? SA_ERR_UNSUPPORTED : cuda_status(e);
}

}  // extern "C"
