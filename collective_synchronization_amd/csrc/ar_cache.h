// ar_cache.h -- the paged key-value cache of ar_kv_cache: host-side checks and
// the view of it that kernels take.  Internal; not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "ar_host.h"
#include "ar_rows.h"

namespace ar {

// Strides in bytes for the rows, in floats for the scales.
struct CacheView {
  uint8_t* k;
  uint8_t* v;
  int64_t page_stride, token_stride, head_stride;
  float* k_scales;
  float* v_scales;
  int64_t scale_page_stride, scale_token_stride, scale_head_stride;
  int32_t pages, page, page_shift, kv_heads, dim;
};

inline CacheView cache_view(const ar_kv_cache* c) {
  const int64_t size = c->format == AR_E4M3_ROW ? 1 : 2;
  CacheView v{};
  v.k = static_cast<uint8_t*>(c->k);
  v.v = static_cast<uint8_t*>(c->v);
  v.page_stride = c->page_stride * size;
  v.token_stride = c->token_stride * size;
  v.head_stride = c->head_stride * size;
  v.k_scales = c->k_scales;
  v.v_scales = c->v_scales;
  v.scale_page_stride = c->scale_page_stride;
  v.scale_token_stride = c->scale_token_stride;
  v.scale_head_stride = c->scale_head_stride;
  v.pages = (int32_t)c->pages;
  v.page = c->page;
  v.page_shift = __builtin_ctz((unsigned)c->page);
  v.kv_heads = c->kv_heads;
  v.dim = c->dim;
  return v;
}

// Sizes and formats of a cache.
inline int check_cache(const ar_kv_cache* c) {
  if (c->format != AR_BF16 && c->format != AR_F16 && c->format != AR_E4M3_ROW) return AR_EINVAL;
  if (c->kv_heads < 1 || c->dim < 16 || c->pages < 0) return AR_EINVAL;
  if (c->page < 16 || (c->page & (c->page - 1)) != 0) return AR_EINVAL;
  if (c->dim % 16 != 0) return AR_EALIGN;
  if (c->dim > AR_CACHE_MAX_DIM || c->pages >= (int64_t(1) << 31) || c->page > (1 << 20)) return AR_ESIZE;
  return AR_OK;
}

// Rows of `width` for every page, token and head that do not overlap: each
// dimension steps past all that the ones with smaller strides cover.
inline bool rows_apart(const ar_kv_cache* c, int64_t width, int64_t page_stride, int64_t token_stride,
                       int64_t head_stride) {
  struct Dim { int64_t count, stride; } d[3] = {
      {c->kv_heads, head_stride}, {c->page, token_stride}, {c->pages, page_stride}};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (d[j].stride > d[j + 1].stride) { const Dim t = d[j]; d[j] = d[j + 1]; d[j + 1] = t; }
  for (const Dim& x : d) {
    if (x.count == 1) continue;
    if (x.stride < width) return false;
    width += (x.count - 1) * x.stride;
  }
  return true;
}

// Its buffers and strides.
inline int check_cache_rows(const ar_kv_cache* c) {
  if (c->pages == 0) return AR_OK;
  if (!c->k || !c->v) return AR_EINVAL;
  if (c->page_stride < 0 || c->token_stride < 0 || c->head_stride < 0) return AR_EINVAL;
  const int64_t most = int64_t(1) << 30;       // a page's number times its stride stays within 2^62 bytes
  if (c->page_stride >= most || c->token_stride >= most || c->head_stride >= most) return AR_ESIZE;
  if (c->token_stride >= 1 << 26) return AR_ESIZE;      // 16 tokens' offsets stay 32-bit
  if (!rows_apart(c, c->dim, c->page_stride, c->token_stride, c->head_stride)) return AR_EINVAL;
  const int unit = c->format == AR_E4M3_ROW ? 16 : 8;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->page_stride % unit || c->token_stride % unit ||
      c->head_stride % unit)
    return AR_EALIGN;
  if (c->format != AR_E4M3_ROW) return AR_OK;
  if (!c->k_scales || !c->v_scales) return AR_EINVAL;
  if (c->scale_page_stride < 0 || c->scale_token_stride < 0 || c->scale_head_stride < 0) return AR_EINVAL;
  if (c->scale_page_stride >= most || c->scale_token_stride >= most || c->scale_head_stride >= most) return AR_ESIZE;
  if (!rows_apart(c, 1, c->scale_page_stride, c->scale_token_stride, c->scale_head_stride)) return AR_EINVAL;
  return aligned(c->k_scales, 4) && aligned(c->v_scales, 4) ? AR_OK : AR_EALIGN;
}

}  // namespace ar
