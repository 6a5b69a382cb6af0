// What the serving operators (paging.cu, attention*.cu, verify.cu) share:
// argument checks, and the ragged rows of a request.
#pragma once
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "errors.h"

namespace dsm {

inline int check_attn_shape(const ds_moe_attn_shape *s, char *err, size_t errlen) {
  if (!s) return fail(err, errlen, DS_ERR_INVALID_ARG, "shape is NULL");
  if (s->n_head_kv < 1 || s->n_head < 1 || s->n_head > 1024 || s->n_head % s->n_head_kv)
    return fail(err, errlen, DS_ERR_INVALID_ARG, "n_head=%d, n_head_kv=%d: need 1..1024, a multiple", s->n_head, s->n_head_kv);
  if (s->head_dim < 1 || s->head_dim > 128)
    return fail(err, errlen, DS_ERR_UNSUPPORTED, "head_dim=%d: need 1..128", s->head_dim);
  if (s->page_size < 1 || s->page_size > 65536)
    return fail(err, errlen, DS_ERR_INVALID_ARG, "page_size=%d: need 1..65536", s->page_size);
  if (s->dtype != DS_BF16 && s->dtype != DS_F16)
    return fail(err, errlen, DS_ERR_INVALID_ARG, "dtype must be DS_BF16 or DS_F16");
  if (!isfinite(s->scale) || s->scale < 0.f) return fail(err, errlen, DS_ERR_INVALID_ARG, "scale must be finite and >= 0");
  if (s->window < 0) return fail(err, errlen, DS_ERR_INVALID_ARG, "window must be >= 0");
  return DS_OK;
}

inline int check_kv_cache(const ds_moe_attn_shape *s, const ds_moe_kv_cache *c, char *err, size_t errlen) {
  if (!c) return fail(err, errlen, DS_ERR_INVALID_ARG, "cache is NULL");
  if (c->n_pages < 0 || c->n_pages > INT32_MAX) return fail(err, errlen, DS_ERR_INVALID_ARG, "n_pages out of range");
  if (c->n_pages && (!c->k || !c->v)) return fail(err, errlen, DS_ERR_INVALID_ARG, "cache k and v are required");
  if (!aligned(c->k, 2) || !aligned(c->v, 2))
    return fail(err, errlen, DS_ERR_INVALID_ARG, "cache k and v must be aligned to their elements");
  if (c->page_stride < 0 || c->row_stride < 0 || c->head_stride < 0)
    return fail(err, errlen, DS_ERR_INVALID_ARG, "negative cache stride");
  // rows that overlap would make an append's result depend on its order
  if ((s->page_size > 1 && c->row_stride < s->head_dim) || (s->n_head_kv > 1 && c->head_stride < s->head_dim) ||
      (c->n_pages > 1 && c->page_stride < s->head_dim))
    return fail(err, errlen, DS_ERR_INVALID_ARG, "cache strides are smaller than head_dim");
  return DS_OK;
}

// Rows of one request: its tokens t0 .. t0 + n - 1, whose first is at
// position pos0 of a sequence of seq keys.
struct Span {
  int t0, n, pos0, seq;
};
// What it is made of, as it is in memory.
struct RawSpan {
  int c0, c1, seq;
};

__device__ __forceinline__ RawSpan request_raw(const int32_t *__restrict__ cu, const int32_t *__restrict__ seq_lens, int r) {
  return RawSpan{cu[r], cu[r + 1], seq_lens[r]};
}

__device__ __forceinline__ Span request_span(const RawSpan &w, int T, int max_new, int64_t max_seq, bool &bad) {
  Span s;
  s.t0 = min(max(w.c0, 0), T);
  const int end = min(max(w.c1, s.t0), T), n = end - s.t0;
  s.seq = (int)min((int64_t)max(w.seq, 0), max_seq);
  s.pos0 = s.seq - n;
  s.n = min(n, max_new);
  bad = bad || w.c0 != s.t0 || w.c1 != end || w.seq != s.seq || n != s.n;
  return s;
}

__device__ __forceinline__ Span request_span(const int32_t *__restrict__ cu, const int32_t *__restrict__ seq_lens, int r,
                                             int T, int max_new, int64_t max_seq, bool &bad) {
  return request_span(request_raw(cu, seq_lens, r), T, max_new, max_seq, bad);
}

}  // namespace dsm
