// C ABI of sampling and of the walk through trees of drafted tokens: argument checks
// and launches.
#include "refuse.h"

using namespace dfl;

extern "C" {

int dflash_sample(const dflash_sample_args* a, void* stream) {
  auto need = [](const void* p, const char* name, unsigned bytes) { return need_aligned("sample", p, name, bytes); };
  if (!a) return refuse(DFLASH_EINVAL, "sample: args is NULL");
  if (a->dtype != DFLASH_F32 && a->dtype != DFLASH_BF16) return refuse(DFLASH_EINVAL, "sample: dtype must be DFLASH_F32 or DFLASH_BF16");
  if (a->rows < 0 || a->rows > (1 << 27)) return refuse(DFLASH_EINVAL, "sample: rows outside [0, 2^27]");
  if (a->vocab < 1 || a->vocab > (1 << 20)) return refuse(DFLASH_ERANGE, "sample: vocab outside [1, 2^20]");
  if (a->rows == 0) return DFLASH_OK;
  if (a->logit_stride < a->vocab || a->logit_stride >= (1ll << 36)) return refuse(DFLASH_EINVAL, "sample: logit_stride is below vocab (or 2^36 and more)");
  PG(need(a->logits, "logits", a->dtype == DFLASH_BF16 ? 2 : 4));
  PG(need(a->uniform, "uniform", 4));
  if (a->temperature) PG(need(a->temperature, "temperature", 4));
  if (a->top_k) PG(need(a->top_k, "top_k", 4));
  if (a->top_p) PG(need(a->top_p, "top_p", 4));
  if (a->min_p) PG(need(a->min_p, "min_p", 4));
  PG(need(a->token, "token", 4));
  if (a->prob) PG(need(a->prob, "prob", 4));
  const SampleArgs x{a->logits, a->uniform, a->temperature, a->top_k, a->top_p, a->min_p, a->token, a->prob, a->logit_stride, a->rows, a->vocab};
  return launched(launch_sample(a->dtype, x, static_cast<cudaStream_t>(stream)), "sample");
}

int dflash_tree_accept(const dflash_tree_accept_args* a, void* stream) {
  auto need = [](const void* p, const char* name) { return need_aligned("tree accept", p, name, 4); };
  if (!a) return refuse(DFLASH_EINVAL, "tree accept: args is NULL");
  if (a->rows < 0) return refuse(DFLASH_EINVAL, "tree accept: rows is negative");
  if (a->n_seq < 1 || a->n_seq > 65535) return refuse(DFLASH_EINVAL, "tree accept: n_seq outside [1, 65535]");
  if (a->width < 1 || a->width > (1 << 20)) return refuse(DFLASH_EINVAL, "tree accept: width outside [1, 2^20]");
  if ((int64_t)a->n_seq * a->width >= (1ll << 31)) return refuse(DFLASH_ERANGE, "tree accept: n_seq * width reaches 2^31");
  PG(need(a->start, "start"));
  if (a->rows > 0) {
    PG(need(a->tree_end, "tree_end"));
    PG(need(a->draft, "draft"));
    PG(need(a->sampled, "sampled"));
  }
  PG(need(a->tokens, "tokens"));
  PG(need(a->path, "path"));
  PG(need(a->count, "count"));
  if (!a->length != !a->length_out) return refuse(DFLASH_EINVAL, "tree accept: length and length_out come together");
  if (a->length) {
    PG(need(a->length, "length"));
    PG(need(a->length_out, "length_out"));
  }
  const TreeAcceptArgs x{a->tree_end, a->start, a->draft, a->sampled, a->tokens, a->path, a->count, a->length, a->length_out, a->rows, a->n_seq, a->width};
  return launched(launch_tree_accept(x, static_cast<cudaStream_t>(stream)), "tree accept");
}

}  // extern "C"
