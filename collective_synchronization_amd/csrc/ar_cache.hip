// ar_cache.hip -- a step's keys and values into the paged cache (gfx950).
//
// Bound by the stores' way to memory, and for a step of single tokens by the
// launch.  A row is 8 elements a lane, of keys in the grid's first half and of
// values in its second, so that the rows' page numbers are read once each and a
// row's largest value is a maximum over its few lanes.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "../../include/ar.h"
#include "ar_cache.h"
#include "ar_host.h"
#include "ar_rows.h"

namespace ar {

// Strides in elements for k and v.
struct AppendArgs {
  CacheView kv;
  const uint16_t* k;
  const uint16_t* v;
  int64_t k_stride, k_head, v_stride, v_head;
  const int32_t* lengths;
  const int32_t* tables;
  int64_t table_stride;
  int32_t max_pages, queries;
  int64_t rows;                      // tokens * heads
  FastDiv heads, steps;              // of the cache, and `queries`
  int32_t lanes_shift;               // log2 of the lanes to a row
};

template <int F, bool C8>
__global__ __launch_bounds__(kBlock) void k_cache_append(AppendArgs a) {
  const int64_t at = ((int64_t)blockIdx.x * kBlock + threadIdx.x) >> a.lanes_shift;
  const int c = threadIdx.x & ((1 << a.lanes_shift) - 1);
  if (at >= 2 * a.rows) return;
  const bool values_half = at >= a.rows;
  const uint32_t r = (uint32_t)(values_half ? at - a.rows : at);
  const uint32_t token = div_by(r, a.heads), head = r - token * a.heads.d;
  const uint32_t seq = div_by(token, a.steps);
  const int64_t t = (int64_t)a.lengths[seq] - a.queries + (token - seq * a.steps.d);
  if (t < 0 || (t >> a.kv.page_shift) >= a.max_pages) return;
  const int page = a.tables[seq * a.table_stride + (t >> a.kv.page_shift)];
  if ((uint32_t)page >= (uint32_t)a.kv.pages) return;
  const int64_t in_page = t & (a.kv.page - 1);
  const uint16_t* src = values_half ? a.v + token * a.v_stride + head * a.v_head : a.k + token * a.k_stride + head * a.k_head;
  uint8_t* dst = (values_half ? a.kv.v : a.kv.k) + page * a.kv.page_stride + in_page * a.kv.token_stride +
                 head * a.kv.head_stride;
  const Raw<F> raw = load_raw<F>(src, a.kv.dim, c * 8);    // zeros for lanes past the row
  if constexpr (C8) {
    float v[8];
    values<F>(raw, a.kv.dim, c * 8, v);
    uint32_t m = max8_bits(v);
    for (int d = 1 << a.lanes_shift >> 1; d > 0; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
    const bool nan = m >= kInfBits;
    const float most = __uint_as_float(m), s = fmaxf(most / kE4m3Max, 0x1p-126f);
    // Codes of v over the scale before its rounding, 448 v / max|v|: the product
    // is exact and a quotient of two 16-bit numbers that is no code's border is
    // further from it than a rounding, so every code is the nearest.  (Large rows
    // are taken down first, where the product would overflow.)
    const bool tiny = most < 0x1p-126f * kE4m3Max, large = most >= 0x1p100f;
    const float by = tiny ? 0x1p-126f : (large ? most * 0x1p-32f : most);
    const float mul = tiny ? 1.0f : (large ? kE4m3Max * 0x1p-32f : kE4m3Max);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * mul / by;
    if (c * 8 < a.kv.dim) *reinterpret_cast<u32x2*>(dst + c * 8) = e4m3_codes(v, 1.0f, nan);
    if (c == 0)
      (values_half ? a.kv.v_scales : a.kv.k_scales)[page * a.kv.scale_page_stride + in_page * a.kv.scale_token_stride +
                                                    head * a.kv.scale_head_stride] =
          nan ? __builtin_nanf("") : s;
  } else {
    if (c * 8 < a.kv.dim) *reinterpret_cast<u32x4*>(dst + c * 16) = raw.a;
  }
}

}  // namespace ar

using namespace ar;

extern "C" {

int ar_cache_append(const ar_kv_cache* cache, const ar_append_params* p, void* stream) {
  if (!cache || !p || p->sequences < 0 || p->queries < 0 || p->max_pages < 0) return AR_EINVAL;
  int rc = check_cache(cache);
  if (rc) return rc;
  if (p->format != AR_BF16 && p->format != AR_F16) return AR_EINVAL;
  if (cache->format != AR_E4M3_ROW && cache->format != p->format) return AR_EINVAL;
  if (p->sequences == 0 || p->queries == 0 || p->max_pages == 0 || cache->pages == 0) return AR_OK;
  rc = check_cache_rows(cache);
  if (rc) return rc;
  const int64_t most = int64_t(1) << 30;
  if (!p->k || !p->v || !p->lengths || !p->pages) return AR_EINVAL;
  if (p->sequences > 1 && p->pages_stride < p->max_pages) return AR_EINVAL;
  if (p->k_stride < 0 || p->k_head_stride < 0 || p->v_stride < 0 || p->v_head_stride < 0) return AR_EINVAL;
  if (p->sequences >= most || p->max_pages >= most || p->pages_stride >= most || p->k_stride >= most ||
      p->k_head_stride >= most || p->v_stride >= most || p->v_head_stride >= most)
    return AR_ESIZE;
  if (p->sequences * p->queries >= most || p->sequences * p->queries * cache->kv_heads >= most) return AR_ESIZE;
  if (!aligned(p->k, 16) || !aligned(p->v, 16) || p->k_stride % 8 || p->k_head_stride % 8 || p->v_stride % 8 ||
      p->v_head_stride % 8 || !aligned(p->lengths, 4) || !aligned(p->pages, 4))
    return AR_EALIGN;
  AppendArgs a{};
  a.kv = cache_view(cache);
  a.k = static_cast<const uint16_t*>(p->k);
  a.v = static_cast<const uint16_t*>(p->v);
  a.k_stride = p->k_stride;
  a.k_head = p->k_head_stride;
  a.v_stride = p->v_stride;
  a.v_head = p->v_head_stride;
  a.lengths = p->lengths;
  a.tables = p->pages;
  a.table_stride = p->pages_stride;
  a.max_pages = (int32_t)p->max_pages;
  a.queries = p->queries;
  a.rows = p->sequences * p->queries * cache->kv_heads;
  a.heads = fast_div((uint32_t)cache->kv_heads);
  a.steps = fast_div((uint32_t)p->queries);
  while ((8 << a.lanes_shift) < cache->dim) ++a.lanes_shift;
  const int64_t blocks = ceil_div64((2 * a.rows) << a.lanes_shift, kBlock);
  if (blocks > most_blocks(kBlock)) return AR_ESIZE;
  const dim3 grid((unsigned)blocks), block(kBlock);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool c8 = cache->format == AR_E4M3_ROW;
  if (p->format == AR_BF16)
    return map_hip(c8 ? launch(k_cache_append<AR_BF16, true>, grid, block, s, a)
                      : launch(k_cache_append<AR_BF16, false>, grid, block, s, a));
  return map_hip(c8 ? launch(k_cache_append<AR_F16, true>, grid, block, s, a)
                    : launch(k_cache_append<AR_F16, false>, grid, block, s, a));
}

}  // extern "C"
