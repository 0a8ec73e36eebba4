// Argument checks that the host sources of the paged-cache operators share: pages, a layer's
// cache, rows of activations.
#pragma once

#include <hip/hip_runtime_api.h>

#include <algorithm>
#include <cmath>

#include "host_util.h"
#include "kv.h"

namespace rax {

inline bool page_size_ok(int p) { return p >= 16 && p <= 1024 && (p & (p - 1)) == 0; }
inline int log2_of(int p) {
  int s = 0;
  while ((1 << s) < p) ++s;
  return s;
}

inline lora_status check_pages(int page_size, int num_pages) {
  if (!page_size_ok(page_size)) return fail(LORA_ERR_SHAPE, "page_size %d is not a power of two in [16, 1024]", page_size);
  if (num_pages < 1 || (long long)num_pages * page_size > 0x7fffffffLL)
    return fail(LORA_ERR_SHAPE, "num_pages %d outside [1, (2^31 - 1) / page_size]", num_pages);
  return LORA_OK;
}

inline lora_status check_head_dim(int dim) {
  if (dim > LORA_MAX_HEAD_DIM) return fail(LORA_ERR_SHAPE, "head_dim %d above %d", dim, LORA_MAX_HEAD_DIM);
  if (dim < 16 || dim % 16) return fail(LORA_ERR_ALIGN, "head_dim %d is not a positive multiple of 16", dim);
  return LORA_OK;
}

inline lora_status check_cache(const lora_kv_cache* c) {
  if (!c) return fail(LORA_ERR_INVALID_ARG, "cache must not be NULL");
  if (!c->k || !c->v) return fail(LORA_ERR_INVALID_ARG, "cache->k and cache->v must not be NULL");
  if (c->dtype != LORA_BF16 && c->dtype != LORA_F32 && c->dtype != LORA_FP8E4M3)
    return fail(LORA_ERR_DTYPE, "unknown cache dtype %d", (int)c->dtype);
  if (c->dtype == LORA_FP8E4M3 &&
      !(std::isfinite(c->k_scale) && std::isfinite(c->v_scale) && c->k_scale > 0 && c->v_scale > 0))
    return fail(LORA_ERR_INVALID_ARG, "k_scale and v_scale must be positive and finite");
  lora_status st = check_pages(c->page_size, c->num_pages);
  if (st != LORA_OK) return st;
  if (c->num_heads < 1 || c->num_heads > 1024) return fail(LORA_ERR_SHAPE, "num_heads %d outside [1, 1024]", c->num_heads);
  if ((st = check_head_dim(c->head_dim)) != LORA_OK) return st;
  // strides: no two elements share an address (each stride spans everything that varies faster)
  struct Axis {
    long long stride, n;
  } ax[3] = {{c->page_stride, c->num_pages}, {c->token_stride, c->page_size}, {c->head_stride, c->num_heads}};
  std::sort(ax, ax + 3, [](const Axis& a, const Axis& b) { return a.stride < b.stride; });
  long long span = c->head_dim;
  for (const Axis& x : ax) {
    if (x.n == 1 && x.stride >= 0) continue;
    if (x.stride < span) return fail(LORA_ERR_SHAPE, "cache strides overlap (stride %lld below %lld)", x.stride, span);
    if (x.stride > (1LL << 60) / x.n) return fail(LORA_ERR_SHAPE, "cache stride %lld too large", x.stride);
    span = x.stride * (x.n - 1) + span;
  }
  if (c->token_stride >= (1LL << 25)) return fail(LORA_ERR_SHAPE, "token_stride %lld is not below 2^25", (long long)c->token_stride);
  if (c->page_stride % 16 || c->token_stride % 16 || c->head_stride % 16 || !aligned16(c->k) || !aligned16(c->v))
    return fail(LORA_ERR_ALIGN, "cache strides must be multiples of 16 elements and k, v 16-byte aligned");
  return LORA_OK;
}

inline lora_status check_act(lora_dtype dtype, const lora_kv_cache* c) {
  if (dtype != LORA_BF16 && dtype != LORA_F32) return fail(LORA_ERR_DTYPE, "activations must be bfloat16 or float32");
  if ((dtype == LORA_F32) != (c->dtype == LORA_F32))
    return fail(LORA_ERR_DTYPE, "float32 activations take a float32 cache, bfloat16 ones a bfloat16 or e4m3 cache");
  return LORA_OK;
}

inline lora_status check_rows(const char* what, const void* p, int ld, long long width, int rows) {
  if (rows > 0 && !p) return fail(LORA_ERR_INVALID_ARG, "%s is NULL", what);
  if (ld < width) return fail(LORA_ERR_SHAPE, "%s: row stride %d below its width %lld", what, ld, width);
  if (ld % 8 || !aligned16(p)) return fail(LORA_ERR_ALIGN, "%s must be 16-byte aligned with a row stride a multiple of 8", what);
  return LORA_OK;
}

inline CacheView cache_view(const lora_kv_cache* c) {
  CacheView v{};
  v.k = c->k;
  v.v = c->v;
  v.page_stride = c->page_stride;
  v.token_stride = c->token_stride;
  v.head_stride = c->head_stride;
  v.num_pages = c->num_pages;
  v.page_shift = log2_of(c->page_size);
  v.heads = c->num_heads;
  v.dim = c->head_dim;
  v.dtype = c->dtype;
  const bool f8 = c->dtype == LORA_FP8E4M3;
  v.k_scale = f8 ? c->k_scale : 1.f;
  v.v_scale = f8 ? c->v_scale : 1.f;
  return v;
}

}  // namespace rax
