// ar_rows.h -- rows of values in the formats of ar_format: loads and stores
// of 8-element chunks, the conversions to 8- and 4-bit floats, and the
// host-side checks of row arguments.  Internal; not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>

#include "ar_host.h"

namespace ar {

constexpr int kMxBlock = 32;              // elements that share an e8m0 scale
constexpr int kE4m3Emax = 8;              // exponent of the largest power of two
constexpr int kE2m1Emax = 2;
constexpr float kE4m3Max = 448.0f;

__host__ __device__ constexpr bool is_float_format(int f) { return f >= AR_BF16 && f <= AR_F32; }
__host__ __device__ constexpr bool is_mx_format(int f) { return f == AR_E4M3_MX || f == AR_E2M1_MX; }

// ------------------------------------------------------------- chunks ---
// A chunk is 8 elements of one row, 16-byte aligned in a 16-bit row.  Rows
// are written below `count` only; a chunk that ends past it goes element by
// element.

template <int F> struct Elem;
template <> struct Elem<AR_BF16> { typedef uint16_t type; };
template <> struct Elem<AR_F16> { typedef _Float16 type; };
template <> struct Elem<AR_F32> { typedef float type; };

// Two bf16, nearest even, by the conversion instruction (NaNs stay quiet NaNs).
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

template <int F>
__device__ __forceinline__ typename Elem<F>::type elem_from_f32(float v) {
  if constexpr (F == AR_BF16) return (uint16_t)bf16_pair(v, 0.0f);
  else if constexpr (F == AR_F16) return (_Float16)v;
  else return v;
}

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// A chunk as it lies in memory.  Loading and converting are apart so that a
// thread can have all its loads under way before it waits for the first.
template <int F> struct Raw { u32x4 a; };
template <> struct Raw<AR_F32> { u32x4 a, b; };

// Elements [first, first + 8) of a row, up to the 16-byte boundary after
// element count - 1; zeros past that.
template <int F>
__device__ __forceinline__ Raw<F> load_raw(const void* row, int64_t count, int64_t first) {
  Raw<F> r{};
  const auto* p = static_cast<const typename Elem<F>::type*>(row) + first;
  if (first < count) r.a = *reinterpret_cast<const u32x4*>(p);
  if constexpr (F == AR_F32) {
    if (first + 4 < count) r.b = *reinterpret_cast<const u32x4*>(p + 4);
  }
  return r;
}

// The same through a buffer resource whose range is the row up to that
// boundary (raw_row below): no branch, so nothing waits on its way.
template <int F>
__device__ __forceinline__ Raw<F> load_raw(rsrc_t row, int64_t first) {
  Raw<F> r;
  const uint32_t off = (uint32_t)first * (F == AR_F32 ? 4u : 2u);
  r.a = __builtin_amdgcn_raw_buffer_load_b128(row, off, 0, 0);
  if constexpr (F == AR_F32) r.b = __builtin_amdgcn_raw_buffer_load_b128(row, off + 16u, 0, 0);
  return r;
}
// `row` the same for all lanes; null: an empty range, which reads as zeros.
__device__ __forceinline__ rsrc_t raw_row(const void* row, int64_t count, int size) {
  return make_rsrc(row, row ? (uint32_t)((count * size + 15) & ~int64_t(15)) : 0u);
}

// The chunk's values; zeros at and past count.
template <int F>
__device__ __forceinline__ void values(const Raw<F>& r, int64_t count, int64_t first, float (&v)[8]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (F == AR_BF16) {
      v[2 * k] = bf_lo(r.a[k]);
      v[2 * k + 1] = bf_hi(r.a[k]);
    } else if constexpr (F == AR_F16) {
      typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
      const uint32_t d = r.a[k];
      const f16x2 h = __builtin_bit_cast(f16x2, d);
      v[2 * k] = (float)h.x;
      v[2 * k + 1] = (float)h.y;
    } else {
      v[k] = __uint_as_float(r.a[k]);
      v[4 + k] = __uint_as_float(r.b[k]);
    }
  }
  if (first + 8 > count) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = first + k < count ? v[k] : 0.0f;
  }
}

// Float rows go past the caches: the next kernel reads them on any XCD, and the
// lines that they would displace are inputs still to be read.  8192 x 8192 from
// 4 bits to bf16: 28 us against 39 with ordinary stores (25 since, for other
// reasons); the norm of 16384 x 8192 to bf16 180 against 185, of 1000 x 4100 fp16
// 7.8 against 8.4.
template <typename V>
__device__ __forceinline__ void store_nt(void* p, V v) {
  __builtin_nontemporal_store(v, reinterpret_cast<V*>(p));
}

// One rounding to the row's type, nearest even.
template <int F>
__device__ __forceinline__ void store8(typename Elem<F>::type* __restrict__ row, int64_t count,
                                       int64_t first, const float (&v)[8]) {
  if (first + 8 <= count) {
    if constexpr (F == AR_BF16) {
      store_nt(row + first, u32x4{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]), bf16_pair(v[4], v[5]),
                                  bf16_pair(v[6], v[7])});
    } else if constexpr (F == AR_F16) {
      f16x8 d;
#pragma unroll
      for (int k = 0; k < 8; ++k) d[k] = (_Float16)v[k];
      store_nt(row + first, d);
    } else {
      store_nt(row + first, f32x4{v[0], v[1], v[2], v[3]});
      store_nt(row + first + 4, f32x4{v[4], v[5], v[6], v[7]});
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (first + k < count) row[first + k] = elem_from_f32<F>(v[k]);
  }
}

// --------------------------------------------------- 8- and 4-bit floats ---

// Unsigned division by a number known at launch: n / d for n < 2^31.
struct FastDiv {
  uint32_t d, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
  // ceil(2^(32 + shift) / d) with 2^shift >= d: exact for n < 2^32, and the
  // 33rd bit of the multiplier, always set, is added apart
  uint32_t s = 0;
  while ((uint64_t(1) << s) < d) ++s;
  const uint64_t m = ((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1;
  return {d, (uint32_t)m, s};
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, FastDiv f) {
  return (uint32_t)(((uint64_t)__umulhi(n, f.mul) + n) >> f.shift);
}

// The largest magnitude as its binary32 pattern: patterns order as the
// magnitudes do, infinities above every finite value and NaNs above those,
// so a maximum of patterns also says whether the block holds either.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
constexpr uint32_t kInfBits = 0x7F800000u;

__device__ __forceinline__ uint32_t max8_bits(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = max(m, abs_bits(v[k]));
  return m;
}

// e8m0 code of a block whose largest magnitude has the pattern `amax`: the
// block's exponent floor(log2 amax) less the format's own largest one, so
// the largest element lands in the format's top binade; 0 (2^-127) for
// blocks below that, zeros among them; 0xFF (NaN) for one that holds a NaN
// or an infinity.
template <int F>
__device__ __forceinline__ uint32_t mx_scale_code(uint32_t amax) {
  constexpr int emax = F == AR_E4M3_MX ? kE4m3Emax : kE2m1Emax;
  const int e = (int)(amax >> 23) - emax;
  return amax >= kInfBits ? 0xFFu : (uint32_t)max(e, 0);
}

// e4m3 codes of 8 values times `mul`, nearest even, saturated at 448 (the
// conversion itself makes NaN of larger values); `nan`: all codes NaN.
__device__ __forceinline__ u32x2 e4m3_codes(const float (&v)[8], float mul, bool nan) {
  uint32_t d[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    float t[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      t[k] = __builtin_amdgcn_fmed3f(v[4 * q + k] * mul, -kE4m3Max, kE4m3Max);
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(t[0], t[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(t[2], t[3], w, true);
    d[q] = nan ? 0x7F7F7F7Fu : (uint32_t)w;
  }
  return u32x2{d[0], d[1]};
}

// e2m1 codes of 8 values over the scale 2^(code - 127), two in a byte, the
// even element low; nearest even, saturated at 6 (the conversion's own
// behaviour).  The conversion reads the scale's exponent field alone, so
// code << 23 also stands for code 0.
__device__ __forceinline__ uint32_t e2m1_codes(const float (&v)[8], uint32_t code) {
  const float s = __uint_as_float(code << 23);
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], s, 3);
  return code == 0xFFu ? 0u : w;
}

// Maximum over the 4 lanes that hold one 32-element block.
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
  // quad permutations 1,0,3,2 and 2,3,0,1
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, true));
  return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, true));
}

// Quantise chunk `c` (8 elements) of a row to an MX format.  The 4 lanes of
// an aligned group hold the 4 chunks of one block and all reach this call.
// Chunks past the row's last element belong to its last block: zeros.
template <int F>
__device__ __forceinline__ void store8_mx(uint8_t* __restrict__ row, uint8_t* __restrict__ scales,
                                          int c, int chunks, const float (&v)[8]) {
  const uint32_t code = mx_scale_code<F>(block_max(max8_bits(v)));
  if (c >= chunks) return;
  if constexpr (F == AR_E4M3_MX) {
    const bool nan = code == 0xFFu;
    const float mul = __uint_as_float((254u - (nan ? 0u : code)) << 23);   // 2^(127 - code)
    *reinterpret_cast<u32x2*>(row + (int64_t)c * 8) = e4m3_codes(v, mul, nan);
  } else {
    *reinterpret_cast<uint32_t*>(row + (int64_t)c * 4) = e2m1_codes(v, code);
  }
  if ((c & 3) == 0) scales[c >> 2] = (uint8_t)code;
}

// ---------------------------------------------------------- host checks ---

inline int64_t mx_blocks(int64_t cols) { return ceil_div64(cols, kMxBlock); }

// Bytes of a stride in a format's units (elements, or bytes of codes).
inline int64_t format_bytes(int32_t f, int64_t stride) {
  return f == AR_F32 ? 4 * stride : (is_float_format(f) ? 2 * stride : stride);
}

// Bytes a row of `cols` elements takes in a format (its scales apart).
inline int64_t format_row_bytes(int32_t f, int64_t cols) {
  switch (f) {
    case AR_BF16:
    case AR_F16: return 2 * cols;
    case AR_F32: return 4 * cols;
    case AR_E4M3_ROW: return cols;
    case AR_E4M3_MX: return kMxBlock * mx_blocks(cols);
    default: return kMxBlock / 2 * mx_blocks(cols);
  }
}

// Rows of a format: 16-byte aligned, a stride of whole 16-byte steps (8
// elements of a 16-bit type, 8 of binary32, 16 bytes of codes) that holds a
// row, row offsets within 2^62 bytes.
inline int check_format_rows(int32_t f, const void* p, int64_t stride, int64_t rows, int64_t cols) {
  if (rows == 0 || cols == 0) return AR_OK;
  if (!p) return AR_EINVAL;
  if (stride <= 0 || stride >= (int64_t(1) << 40)) return stride <= 0 ? AR_EINVAL : AR_ESIZE;
  if (format_bytes(f, stride) < format_row_bytes(f, cols)) return AR_EINVAL;
  if (!aligned(p, 16) || stride % (is_float_format(f) ? 8 : 16) != 0) return AR_EALIGN;
  return AR_OK;
}

// Scales of a format's rows: e8m0 bytes with a row stride that is a multiple
// of 4 bytes, or one binary32 a row.
inline int check_scales(int32_t f, const void* p, int64_t stride, int64_t rows, int64_t cols) {
  if (is_float_format(f) || rows == 0 || cols == 0) return AR_OK;
  if (!p) return AR_EINVAL;
  if (!aligned(p, 4)) return AR_EALIGN;
  if (f == AR_E4M3_ROW) return AR_OK;
  if (stride < mx_blocks(cols)) return AR_EINVAL;
  if (stride >= (int64_t(1) << 40)) return AR_ESIZE;
  return stride % 4 ? AR_EALIGN : AR_OK;
}

}  // namespace ar
