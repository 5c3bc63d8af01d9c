// C ABI of the paged cache: argument checks and launches.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include "dflash.h"
#include "kernels.h"

namespace dfl {
void set_global_error(const char* msg);
}

using namespace dfl;

namespace {

int refuse(int code, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  try {
    set_global_error(buf);
  } catch (...) {
  }
  return code;
}

int launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return DFLASH_OK;
  return refuse(DFLASH_ECUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

bool misaligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

// A device array that a call needs: not NULL and 16-byte aligned.
int need(const void* p, const char* name) {
  if (!p) return refuse(DFLASH_EINVAL, "paged: %s is NULL", name);
  if (misaligned(p)) return refuse(DFLASH_EINVAL, "paged: %s is not 16-byte aligned", name);
  return DFLASH_OK;
}
int may(const void* p, const char* name) { return p ? need(p, name) : DFLASH_OK; }
// An array that is read or written an element of four bytes at a time: a slice
// of a larger one may start anywhere.
int need4(const void* p, const char* name) {
  if (!p) return refuse(DFLASH_EINVAL, "paged: %s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) & 3u) return refuse(DFLASH_EINVAL, "paged: %s is not 4-byte aligned", name);
  return DFLASH_OK;
}
int may4(const void* p, const char* name) { return p ? need4(p, name) : DFLASH_OK; }

#define PG(call)          \
  do {                    \
    int rc_ = (call);     \
    if (rc_) return rc_;  \
  } while (0)

int check_cache(const dflash_paged_cache* c, PagedView* v) {
  if (!c) return refuse(DFLASH_EINVAL, "paged: cache is NULL");
  if (c->dtype != DFLASH_F32 && c->dtype != DFLASH_BF16)
    return refuse(DFLASH_EINVAL, "paged: dtype must be DFLASH_F32 or DFLASH_BF16");
  if (c->n_pages < 1 || c->kv_heads < 1 || c->kv_heads > 1024 || c->max_pages < 1)
    return refuse(DFLASH_EINVAL, "paged: n_pages, max_pages and kv_heads (at most 1024) must be positive");
  if (c->n_seq < 1 || c->n_seq > 65535) return refuse(DFLASH_EINVAL, "paged: n_seq outside [1, 65535]");
  if (c->head_dim < 8 || c->head_dim > 256 || c->head_dim % 8)
    return refuse(DFLASH_EINVAL, "paged: head_dim must be a multiple of 8 in [8, 256]");
  if (c->page_rows < 8 || c->page_rows > 4096 || (c->page_rows & (c->page_rows - 1)))
    return refuse(DFLASH_EINVAL, "paged: page_rows must be a power of two in [8, 4096]");
  if ((int64_t)c->n_pages * c->kv_heads * c->page_rows >= (1ll << 31))
    return refuse(DFLASH_ERANGE, "paged: n_pages * kv_heads * page_rows reaches 2^31");
  if ((int64_t)c->max_pages * c->page_rows > (1 << 20))
    return refuse(DFLASH_ERANGE, "paged: a table of more than 2^20 rows a sequence");
  PG(need(c->k, "cache.k"));
  PG(need(c->v, "cache.v"));
  PG(need(c->pos, "cache.pos"));
  PG(need4(c->table, "cache.table"));
  PG(need4(c->length, "cache.length"));
  PG(may4(c->status, "cache.status"));
  v->k = c->k; v->v = c->v; v->pos = c->pos; v->table = c->table; v->length = c->length; v->status = c->status;
  v->n_pages = c->n_pages;
  v->lg_rows = 0;
  while ((1 << v->lg_rows) < c->page_rows) ++v->lg_rows;
  v->nkv = c->kv_heads; v->hd = c->head_dim; v->n_seq = c->n_seq; v->max_pages = c->max_pages;
  return DFLASH_OK;
}

int check_heads(const dflash_paged_cache* c, int rows, int nq) {
  if (rows < 0) return refuse(DFLASH_EINVAL, "paged: rows is negative");
  if (nq < 1 || nq % c->kv_heads || nq / c->kv_heads > 128)
    return refuse(DFLASH_EINVAL, "paged: n_q_heads must be a multiple of kv_heads, at most 128 to each");
  if ((int64_t)rows * nq >= (1ll << 31)) return refuse(DFLASH_ERANGE, "paged: rows * n_q_heads reaches 2^31");
  return DFLASH_OK;
}

int check_stride(int64_t stride, int64_t least, const char* name) {
  if (stride < least || stride % 8 || stride >= (1ll << 36))
    return refuse(DFLASH_EINVAL, "paged: %s must be a multiple of 8 of at least the row's %lld elements", name, (long long)least);
  return DFLASH_OK;
}

int check_attention(const dflash_paged_cache* c, const dflash_paged_attention_args* a, bool weights, PagedAttnArgs* x) {
  PG(check_cache(c, &x->c));
  if (!a) return refuse(DFLASH_EINVAL, "paged attention: args is NULL");
  PG(check_heads(c, a->rows, a->n_q_heads));
  if (a->rows > 0) {
    PG(check_stride(a->q_stride, (int64_t)a->n_q_heads * c->head_dim, "q_stride"));
    PG(need(a->q, "q"));
    PG(need4(a->q_pos, "q_pos"));
    if (!weights) PG(need(a->out, "out"));
    if (weights) PG(need4(a->lse, "lse"));
  }
  PG(need4(a->start, "start"));
  PG(may4(a->slopes, "slopes"));
  PG(may4(a->prefix, "prefix"));
  PG(may4(a->lse, "lse"));
  // (within these no product or quotient of the two leaves fp32)
  if (!(a->scale > 0.f && a->scale <= 1e18f)) return refuse(DFLASH_EINVAL, "paged attention: scale must be positive and at most 1e18");
  if (a->softcap != 0.f && !(a->softcap >= 1e-18f && a->softcap <= 1e18f))
    return refuse(DFLASH_EINVAL, "paged attention: softcap must be 0 or in [1e-18, 1e18]");
  if (a->max_len < 0) return refuse(DFLASH_EINVAL, "paged attention: max_len is negative");
  x->q = a->q; x->q_pos = a->q_pos; x->start = a->start; x->slopes = a->slopes; x->prefix = a->prefix;
  x->out = a->out; x->lse = a->lse;
  x->part_o = nullptr; x->part_ml = nullptr;
  x->q_stride = a->q_stride; x->rows = a->rows; x->nq = a->n_q_heads; x->G = a->n_q_heads / c->kv_heads;
  x->causal = a->causal != 0; x->window = a->window; x->splits = 1; x->cluster = 0; x->max_len = a->max_len;
  x->scale = a->scale; x->softcap = a->softcap;
  x->weight_in = nullptr; x->weight_out = nullptr; x->decay = 0.f;
  return DFLASH_OK;
}

// Rows of holes and late rows an eviction can have per (sequence, kv head).
int evict_moves(const dflash_paged_cache* c, int budget) {
  const int cap = c->max_pages * c->page_rows;
  const int over = cap > budget ? cap - budget : 0;
  return budget < over ? budget : over;
}
int64_t evict_bytes(const dflash_paged_cache* c, int budget) {
  return (int64_t)c->n_seq * c->kv_heads * (1 + 2 * (int64_t)evict_moves(c, budget)) * 4;
}

int check_evict(const dflash_paged_cache* c, const dflash_paged_evict_args* a, PagedEvictArgs* x) {
  PG(check_cache(c, &x->c));
  if (!a) return refuse(DFLASH_EINVAL, "paged evict: args is NULL");
  if (a->budget < 1) return refuse(DFLASH_EINVAL, "paged evict: budget must be at least 1");
  if (a->recent < 0) return refuse(DFLASH_EINVAL, "paged evict: recent is negative");
  return DFLASH_OK;
}

}  // namespace

extern "C" {

int dflash_paged_append(const dflash_paged_cache* cache, const dflash_paged_append_args* a, void* stream) {
  PagedAppendArgs x;
  PG(check_cache(cache, &x.c));
  if (!a) return refuse(DFLASH_EINVAL, "paged append: args is NULL");
  PG(check_heads(cache, a->rows, a->n_q_heads));
  const int hd = cache->head_dim;
  if (a->n_axes < 1 || a->n_axes > 4) return refuse(DFLASH_EINVAL, "paged append: n_axes outside [1, 4]");
  if (a->rot_pairs < 0 || a->rot_pairs > hd / 2) return refuse(DFLASH_EINVAL, "paged append: rot_pairs outside [0, head_dim / 2]");
  if (!(a->rope_theta >= 1.f) || isinf(a->rope_theta)) return refuse(DFLASH_EINVAL, "paged append: rope_theta must be finite and at least 1");
  if (!(a->rms_eps > 0.f) || isinf(a->rms_eps)) return refuse(DFLASH_EINVAL, "paged append: rms_eps must be positive and finite");
  if (a->rot_pairs > 0 && !a->pair_axis_host) return refuse(DFLASH_EINVAL, "paged append: pair_axis_host is NULL");
  for (int i = 0; i < a->rot_pairs; ++i)
    if (a->pair_axis_host[i] >= a->n_axes)
      return refuse(DFLASH_ERANGE, "paged append: pair_axis_host[%d] is not below n_axes", i);
  PG(need4(a->start, "start"));
  PG(may(a->weight, "weight"));
  PG(may(a->q_norm, "q_norm"));
  PG(may(a->k_norm, "k_norm"));
  if (a->rows == 0) return DFLASH_OK;
  PG(check_stride(a->q_stride, (int64_t)a->n_q_heads * hd, "q_stride"));
  PG(check_stride(a->k_stride, (int64_t)cache->kv_heads * hd, "k_stride"));
  PG(check_stride(a->v_stride, (int64_t)cache->kv_heads * hd, "v_stride"));
  PG(need(a->q, "q"));
  PG(need(a->k, "k"));
  PG(need(a->v, "v"));
  PG(need4(a->row_pos, "row_pos"));
  if (a->rot_pairs > 0) PG(need4(a->rope_pos, "rope_pos"));
  PG(need(a->q_out, "q_out"));
  if (a->q_out == a->q && a->q_stride != (int64_t)a->n_q_heads * hd)
    return refuse(DFLASH_EINVAL, "paged append: q_out may be q only when q is dense");
  x.q = a->q; x.k = a->k; x.v = a->v; x.row_pos = a->row_pos; x.start = a->start; x.rope_pos = a->rope_pos;
  x.q_norm = a->q_norm; x.k_norm = a->k_norm; x.q_out = a->q_out; x.weight = a->weight;
  x.q_stride = a->q_stride; x.k_stride = a->k_stride; x.v_stride = a->v_stride;
  x.rows = a->rows; x.nq = a->n_q_heads; x.pairs = a->rot_pairs; x.neox = a->rope_neox != 0; x.eps = a->rms_eps;
  // theta^(-i / pairs) in turns: the first eight by pow, the others eighth by
  // eighth (at most 15 roundings of 2^-53, and a third of the call's host time less)
  double turns[kPagedMaxPairs];
  const double eighth = a->rot_pairs > 8 ? pow((double)a->rope_theta, -8.0 / a->rot_pairs) : 1.0;
  for (int i = 0; i < a->rot_pairs; ++i) {
    turns[i] = i < 8 ? pow((double)a->rope_theta, -(double)i / a->rot_pairs) * 0.15915494309189533577   // 1 / (2 pi)
                     : turns[i - 8] * eighth;
    x.freq[i] = (unsigned long long)(turns[i] * 18446744073709551616.0);
    x.axis[i] = a->pair_axis_host[i];
  }
  return launched(launch_paged_append(cache->dtype, x, static_cast<cudaStream_t>(stream)), "paged append");
}

int dflash_paged_attention_workspace(const dflash_paged_cache* cache, const dflash_paged_attention_args* a, int64_t* bytes_host) {
  PagedAttnArgs x;
  if (!bytes_host) return refuse(DFLASH_EINVAL, "paged attention: bytes_host is NULL");
  *bytes_host = 0;
  PG(check_attention(cache, a, false, &x));
  if (a->rows > 0) *bytes_host = paged_attn_plan(cache->dtype, x).bytes;
  return DFLASH_OK;
}

int dflash_paged_attention(const dflash_paged_cache* cache, const dflash_paged_attention_args* a, void* stream) {
  PagedAttnArgs x;
  PG(check_attention(cache, a, false, &x));
  if (a->rows == 0) return DFLASH_OK;
  const PagedPlan p = paged_attn_plan(cache->dtype, x);
  if (p.bytes > 0) {
    PG(need(a->workspace, "workspace"));
    if (a->workspace_bytes < p.bytes)
      return refuse(DFLASH_EINVAL, "paged attention: workspace of %lld bytes, %lld needed", (long long)a->workspace_bytes, (long long)p.bytes);
    x.part_o = static_cast<float*>(a->workspace);
    x.part_ml = reinterpret_cast<float2*>(x.part_o + (int64_t)p.splits * a->rows * a->n_q_heads * cache->head_dim);
  }
  x.splits = p.splits;
  x.cluster = p.cluster;
  return launched(launch_paged_attention(cache->dtype, x, p, static_cast<cudaStream_t>(stream)), "paged attention");
}

int dflash_paged_key_weight(const dflash_paged_cache* cache, const dflash_paged_attention_args* a, const float* weight_in,
                            float decay, float* weight_out, void* stream) {
  PagedAttnArgs x;
  PG(check_attention(cache, a, true, &x));
  PG(may(weight_in, "weight_in"));
  PG(need(weight_out, "weight_out"));
  if (!isfinite(decay)) return refuse(DFLASH_EINVAL, "paged key weight: decay must be finite");
  x.weight_in = weight_in; x.weight_out = weight_out; x.decay = decay;
  return launched(launch_paged_key_weight(cache->dtype, x, static_cast<cudaStream_t>(stream)), "paged key weight");
}

int dflash_paged_evict_workspace(const dflash_paged_cache* cache, const dflash_paged_evict_args* a, int64_t* bytes_host) {
  PagedEvictArgs x;
  if (!bytes_host) return refuse(DFLASH_EINVAL, "paged evict: bytes_host is NULL");
  *bytes_host = 0;
  PG(check_evict(cache, a, &x));
  *bytes_host = evict_bytes(cache, a->budget);
  return DFLASH_OK;
}

int dflash_paged_evict(const dflash_paged_cache* cache, const dflash_paged_evict_args* a, void* stream) {
  PagedEvictArgs x;
  PG(check_evict(cache, a, &x));
  PG(need(a->weight, "weight"));
  PG(need4(a->next_pos, "next_pos"));
  PG(need(a->weight_out, "weight_out"));
  PG(need(a->pos_out, "pos_out"));
  PG(need4(a->length_out, "length_out"));
  PG(need(a->workspace, "workspace"));
  const int64_t bytes = evict_bytes(cache, a->budget);
  if (a->workspace_bytes < bytes)
    return refuse(DFLASH_EINVAL, "paged evict: workspace of %lld bytes, %lld needed", (long long)a->workspace_bytes, (long long)bytes);
  x.weight = a->weight; x.next_pos = a->next_pos; x.weight_out = a->weight_out; x.pos_out = a->pos_out;
  x.length_out = a->length_out; x.moves = static_cast<int*>(a->workspace);
  x.budget = a->budget; x.recent = a->recent; x.max_moves = evict_moves(cache, a->budget);
  return launched(launch_paged_evict(cache->dtype, x, static_cast<cudaStream_t>(stream)), "paged evict");
}

}  // extern "C"
