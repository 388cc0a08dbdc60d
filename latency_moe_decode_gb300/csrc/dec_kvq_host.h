// What the entry points of the paged 4-bit cache share: their checks of arguments, and the arguments as
// the kernels take them.
#pragma once
#include <climits>
#include <cstdio>

#include "dec_kvq.cuh"
#include "dec_ops.h"

namespace dec {
namespace kvq {

inline dec_status check_cache(const dec_kvq_cache* c) {
  if (!c || !c->pages) return op_fail(DEC_ERR_ARG, "cache: NULL");
  if (c->head_dim < 1 || c->n_kv_heads < 1 || c->page_tokens < 1 || c->n_pages < 1)
    return op_fail(DEC_ERR_ARG, "cache: sizes must be positive");
  if (c->head_dim != 64 && c->head_dim != 128) return op_fail(DEC_ERR_UNSUPPORTED, "cache: head_dim must be 64 or 128");
  if (c->n_kv_heads > 1024) return op_fail(DEC_ERR_UNSUPPORTED, "cache: more than 1024 KV heads");
  if (dec_kvq_page_bytes(c->page_tokens, c->n_kv_heads, c->head_dim) == 0)
    return op_fail(DEC_ERR_UNSUPPORTED, "cache: page_tokens must be 16, 32, 64, 128 or 256");
  if (!op_aligned(c->pages)) return op_fail(DEC_ERR_ARG, "cache: pages must be 16-byte aligned");
  return DEC_OK;
}

inline dec_status check_seqs(const dec_kvq_seqs* s, const dec_kvq_cache* c) {
  if (!s) return op_fail(DEC_ERR_ARG, "sequences: NULL");
  if (s->batch < 0 || s->n_tokens < 0 || s->max_pages < 0) return op_fail(DEC_ERR_ARG, "sequences: negative size");
  if (!s->cu_tokens && s->n_tokens != s->batch)
    return op_fail(DEC_ERR_ARG, "sequences: without cu_tokens every sequence has one row (n_tokens == batch)");
  if (s->batch == 0 || s->n_tokens == 0) return DEC_OK;
  if (!s->lengths || !s->table || s->max_pages == 0) return op_fail(DEC_ERR_ARG, "sequences: lengths and table are needed");
  // (sequences are counted in 32 bits, up to a launch's share past the last)
  if (s->batch > INT_MAX - 4 * kMaxSeqs) return op_fail(DEC_ERR_UNSUPPORTED, "sequences: a batch of 2^31");
  if (s->table_stride < 0) return op_fail(DEC_ERR_ARG, "sequences: negative table_stride");
  if ((long long)s->max_pages * c->page_tokens > INT_MAX - 65536)
    return op_fail(DEC_ERR_UNSUPPORTED, "sequences: a page table of 2^31 positions or more");
  return DEC_OK;
}

inline dec_status check_rows(const dec_rows* r, dec_dtype t, const char* name) {
  char buf[120];
  const int per = t == DEC_F32 ? 4 : 8;
  if (!r || !r->p) {
    snprintf(buf, sizeof buf, "%s: NULL", name);
    return op_fail(DEC_ERR_ARG, buf);
  }
  if (!op_aligned(r->p) || r->token_stride % per || r->head_stride % per) {
    snprintf(buf, sizeof buf, "%s: rows and strides must be multiples of 16 bytes", name);
    return op_fail(DEC_ERR_ARG, buf);
  }
  return DEC_OK;
}

inline Cache cache_of(const dec_kvq_cache* c) {
  Cache k;
  k.pages = static_cast<uint8_t*>(c->pages);
  k.n_pages = c->n_pages;
  k.page_shift = 0;
  while ((1 << k.page_shift) < c->page_tokens) ++k.page_shift;
  k.hkv = c->n_kv_heads;
  k.status = c->status;
  return k;
}
inline Seqs seqs_of(const dec_kvq_seqs* s) {
  Seqs k;
  k.batch = s->batch;
  k.n_tokens = s->n_tokens;
  k.max_pages = s->max_pages;
  k.cu = s->cu_tokens;
  k.lengths = s->lengths;
  k.table = s->table;
  k.table_stride = s->table_stride;
  return k;
}
inline Rows rows_of(const dec_rows& r) { return Rows{r.p, r.token_stride, r.head_stride}; }

inline dec_status launched(const char* what) {
  const cudaError_t ce = cudaGetLastError();
  return ce == cudaSuccess ? DEC_OK : op_cuda(ce, what);
}

}  // namespace kvq
}  // namespace dec
