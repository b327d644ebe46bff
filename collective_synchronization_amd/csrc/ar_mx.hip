// ar_mx.hip -- rows to and from the microscaled formats (gfx950): 32
// elements share one power-of-two scale.
//
// Both directions are one pass over memory and bound by it.  8 elements a
// thread: 16-byte loads of 16-bit rows, and the 4 lanes that hold a block find
// its largest magnitude with two lane exchanges, so nothing goes through shared
// memory.  8192 x 8192: bf16 to 4 bits 32 us, to 8 bits 38 us (5.3 and 5.4
// TB/s), fp32 to 4 bits 53 us (5.7); back to bf16 25 and 30 us (6.8 and 6.7).
// Two or four chunks a thread are no faster (31 to 32 us).
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "../../include/ar.h"
#include "ar_host.h"
#include "ar_rows.h"

namespace ar {

struct MxArgs {
  const void* in;
  int64_t in_stride;
  void* codes;
  int64_t codes_stride;
  uint8_t* scales;
  int64_t scale_stride;
  void* out;
  int64_t out_stride;
  int64_t cols;
  uint32_t total;                    // chunks of all rows, whole blocks a row
  FastDiv per_row;                   // chunks of one row
};

template <int F, int Q>
__global__ __launch_bounds__(kBlock) void k_quantize_mx(MxArgs a) {
  const uint32_t n = blockIdx.x * kBlock + threadIdx.x;
  if (n >= a.total) return;                                // whole blocks: total % 4 == 0
  const uint32_t row = div_by(n, a.per_row);
  const int c = (int)(n - row * a.per_row.d);
  float v[8];
  values<F>(load_raw<F>(static_cast<const typename Elem<F>::type*>(a.in) + (int64_t)row * a.in_stride,
                        a.cols, (int64_t)c * 8),
            a.cols, (int64_t)c * 8, v);
  store8_mx<Q>(static_cast<uint8_t*>(a.codes) + (int64_t)row * a.codes_stride,
               a.scales + (int64_t)row * a.scale_stride, c, (int)a.per_row.d, v);
}

// 8 values of an MX row: codes times their block's scale, exact in binary32
// except where the product leaves its range.
template <int Q>
__device__ __forceinline__ void values8(const uint8_t* __restrict__ row, const uint8_t* __restrict__ scales,
                                        int c, float (&v)[8]) {
  const uint32_t code = scales[c >> 2];
  // 2^(code - 127); code 0 is the subnormal 2^-127, code 255 NaN
  const float s = code == 0xFFu ? __uint_as_float(0x7FC00000u)
                                : __uint_as_float(code ? code << 23 : 0x00400000u);
  if constexpr (Q == AR_E4M3_MX) {
    const u32x2 d = *reinterpret_cast<const u32x2*>(row + (int64_t)c * 8);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int w = (int)(k ? d.y : d.x);
      v[4 * k + 0] = __builtin_amdgcn_cvt_f32_fp8(w, 0) * s;
      v[4 * k + 1] = __builtin_amdgcn_cvt_f32_fp8(w, 1) * s;
      v[4 * k + 2] = __builtin_amdgcn_cvt_f32_fp8(w, 2) * s;
      v[4 * k + 3] = __builtin_amdgcn_cvt_f32_fp8(w, 3) * s;
    }
  } else {
    const uint32_t d = *reinterpret_cast<const uint32_t*>(row + (int64_t)c * 4);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      typedef float f32x2 __attribute__((ext_vector_type(2)));
      const f32x2 p = k == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 0)
                      : k == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 1)
                      : k == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 2)
                               : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(d, 1.0f, 3);
      v[2 * k] = p.x * s;
      v[2 * k + 1] = p.y * s;
    }
  }
}

template <int Q, int F>
__global__ __launch_bounds__(kBlock) void k_dequantize_mx(MxArgs a) {
  const uint32_t n = blockIdx.x * kBlock + threadIdx.x;
  if (n >= a.total) return;
  const uint32_t row = div_by(n, a.per_row);
  const int c = (int)(n - row * a.per_row.d);
  if ((int64_t)c * 8 >= a.cols) return;
  float v[8];
  values8<Q>(static_cast<const uint8_t*>(a.codes) + (int64_t)row * a.codes_stride,
             a.scales + (int64_t)row * a.scale_stride, c, v);
  store8<F>(static_cast<typename Elem<F>::type*>(a.out) + (int64_t)row * a.out_stride, a.cols,
            (int64_t)c * 8, v);
}

static int mx_check(int64_t rows, int64_t cols, int32_t f, const void* p, int64_t stride, int32_t q,
                    const void* codes, int64_t codes_stride, const void* scales,
                    int64_t scale_stride) {
  if (rows < 0 || cols < 0) return AR_EINVAL;
  if (!is_float_format(f) || !is_mx_format(q)) return AR_EINVAL;
  if (rows == 0 || cols == 0) return AR_OK;
  if (rows > INT32_MAX || cols > INT32_MAX) return AR_ESIZE;
  if (rows * (mx_blocks(cols) * 4) > INT32_MAX) return AR_ESIZE;
  int rc = check_format_rows(f, p, stride, rows, cols);
  if (rc) return rc;
  rc = check_format_rows(q, codes, codes_stride, rows, cols);
  if (rc) return rc;
  return check_scales(q, scales, scale_stride, rows, cols);
}

static MxArgs mx_args(int64_t rows, int64_t cols) {
  MxArgs a{};
  a.cols = cols;
  a.per_row = fast_div((uint32_t)(mx_blocks(cols) * 4));
  a.total = (uint32_t)(rows * a.per_row.d);
  return a;
}

template <int F>
static hipError_t launch_quantize(const MxArgs& a, int q, hipStream_t s) {
  const dim3 grid((a.total + kBlock - 1) / kBlock), block(kBlock);
  return q == AR_E4M3_MX ? launch(k_quantize_mx<F, AR_E4M3_MX>, grid, block, s, a)
                         : launch(k_quantize_mx<F, AR_E2M1_MX>, grid, block, s, a);
}

template <int Q>
static hipError_t launch_dequantize(const MxArgs& a, int f, hipStream_t s) {
  const dim3 grid((a.total + kBlock - 1) / kBlock), block(kBlock);
  switch (f) {
    case AR_BF16: return launch(k_dequantize_mx<Q, AR_BF16>, grid, block, s, a);
    case AR_F16: return launch(k_dequantize_mx<Q, AR_F16>, grid, block, s, a);
    default: return launch(k_dequantize_mx<Q, AR_F32>, grid, block, s, a);
  }
}

}  // namespace ar

using namespace ar;

extern "C" {

int ar_quantize_mx(int64_t rows, int64_t cols, int32_t in_format, const void* in, int64_t in_stride,
                   int32_t out_format, void* codes, int64_t codes_stride, void* scales,
                   int64_t scale_stride, void* stream) {
  const int rc = mx_check(rows, cols, in_format, in, in_stride, out_format, codes, codes_stride,
                          scales, scale_stride);
  if (rc) return rc;
  if (rows == 0 || cols == 0) return AR_OK;
  MxArgs a = mx_args(rows, cols);
  a.in = in;
  a.in_stride = in_stride;
  a.codes = codes;
  a.codes_stride = codes_stride;
  a.scales = static_cast<uint8_t*>(scales);
  a.scale_stride = scale_stride;
  hipStream_t s = static_cast<hipStream_t>(stream);
  switch (in_format) {
    case AR_BF16: return map_hip(launch_quantize<AR_BF16>(a, out_format, s));
    case AR_F16: return map_hip(launch_quantize<AR_F16>(a, out_format, s));
    default: return map_hip(launch_quantize<AR_F32>(a, out_format, s));
  }
}

int ar_dequantize_mx(int64_t rows, int64_t cols, int32_t in_format, const void* codes,
                     int64_t codes_stride, const void* scales, int64_t scale_stride,
                     int32_t out_format, void* out, int64_t out_stride, void* stream) {
  const int rc = mx_check(rows, cols, out_format, out, out_stride, in_format, codes, codes_stride,
                          scales, scale_stride);
  if (rc) return rc;
  if (rows == 0 || cols == 0) return AR_OK;
  MxArgs a = mx_args(rows, cols);
  a.codes = const_cast<void*>(codes);
  a.codes_stride = codes_stride;
  a.scales = static_cast<uint8_t*>(const_cast<void*>(scales));
  a.scale_stride = scale_stride;
  a.out = out;
  a.out_stride = out_stride;
  hipStream_t s = static_cast<hipStream_t>(stream);
  return map_hip(in_format == AR_E4M3_MX ? launch_dequantize<AR_E4M3_MX>(a, out_format, s)
                                         : launch_dequantize<AR_E2M1_MX>(a, out_format, s));
}

}  // extern "C"
