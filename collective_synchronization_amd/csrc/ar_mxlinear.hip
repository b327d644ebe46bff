// ar_mxlinear.hip -- row-parallel linear layer shards on microscaled 4-bit
// weights (gfx950):
//     y_r[m][n] = sum over k of x_r[m][k] * w_r[n][k]
// for every simulated rank r, with binary32 accumulation in the matrix cores.
//
// 8- and 4-bit inputs go through the block-scaled matrix instruction, which
// takes the e8m0 scales of both operands as they are; bf16 inputs through
// the bf16 one, the weights converted in registers (every e2m1 value times a
// power of two is a bf16 value).  The weights are the first operand, so a
// lane ends with 4 consecutive outputs of one token.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "../../include/ar.h"
#include "ar_host.h"
#include "ar_rows.h"

namespace ar {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// Strides in bytes for x, w and the scales, in elements for y.
struct MxLinArgs {
  const uint8_t* x;
  int64_t x_stride, x_rank;
  const uint8_t* xs;
  int64_t xs_stride, xs_rank;
  const uint8_t* w;
  int64_t w_stride, w_rank;
  const uint8_t* ws;
  int64_t ws_stride, ws_rank;
  void* y;
  int64_t y_stride, y_rank;
  int32_t M, N, K;
  int32_t nb;                        // 32-element blocks of K, the last maybe partial
  int32_t n_groups, m_groups;
  int32_t vec;                       // y rows take 4 elements in one store
};

__device__ __forceinline__ u32x4 ldg16(const uint8_t* p) { return *reinterpret_cast<const u32x4*>(p); }

// Scale dword of blocks b..b+3 with every block at or past `nb` set to 1
// (its codes are zeros; what lies past a row's scales may be anything).
__device__ __forceinline__ uint32_t scale_dword(const uint8_t* row, int b, int nb) {
  if (b + 4 <= nb) return *reinterpret_cast<const uint32_t*>(row + b);
  if (b >= nb) return 0x7F7F7F7Fu;
  const uint32_t keep = (1u << (8 * (nb - b))) - 1u;
  return (*reinterpret_cast<const uint32_t*>(row + b) & keep) | (0x7F7F7F7Fu & ~keep);
}

// The first `keep` bytes of 16, zeros after them.
__device__ __forceinline__ u32x4 keep_bytes(u32x4 v, int keep) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const int k = keep - 4 * d;
    v[d] &= k >= 4 ? 0xFFFFFFFFu : (k <= 0 ? 0u : (1u << (8 * k)) - 1u);
  }
  return v;
}

template <int XF>
struct XFrag;                        // one lane's inputs of a 512-element step
template <> struct XFrag<AR_E4M3_MX> { u32x4 d[4][2]; uint32_t s; };
template <> struct XFrag<AR_E4M3_ROW> { u32x4 d[4][2]; };
template <> struct XFrag<AR_E2M1_MX> { u32x4 d[4]; uint32_t s; };
template <> struct XFrag<AR_BF16> { u32x4 d[4][4]; };

struct WFrag {
  u32x4 d[4];
  uint32_t s;
};

// A step is 16 blocks of K.  Sums over k may go in any order that both
// operands share, so the four lane groups g = lane / 16 of a wave take blocks
// 4g .. 4g+3 of it, one in each of 4 matrix instructions: a lane's 64 bytes of
// weights lie together, and its four scales in one dword.
// The instruction wants 4-bit operands as block g's 32 values in group g, but
// 8-bit ones as values [16g', 16g' + 16) of the 128, for g' = g and g + 4: half
// (g & 1) of blocks g/2 and g/2 + 2 -- while group g still gives the scale of
// block g.
template <bool TAIL>
__device__ __forceinline__ void load_w(const uint8_t* row, const uint8_t* srow, int step, int g, int nb,
                                       WFrag& f) {
  const int b = 16 * step + 4 * g;
#pragma unroll
  for (int s = 0; s < 4; ++s)
    f.d[s] = !TAIL || b + s < nb ? ldg16(row + (int64_t)(b + s) * 16) : u32x4{0u, 0u, 0u, 0u};
  f.s = TAIL ? scale_dword(srow, b, nb) : *reinterpret_cast<const uint32_t*>(srow + b);
}

template <int XF, bool TAIL>
__device__ __forceinline__ void load_x(const uint8_t* row, const uint8_t* srow, int step, int g, int nb,
                                       int K, XFrag<XF>& f) {
  if constexpr (XF == AR_E2M1_MX) {
    const int b = 16 * step + 4 * g;
#pragma unroll
    for (int s = 0; s < 4; ++s)
      f.d[s] = !TAIL || b + s < nb ? ldg16(row + (int64_t)(b + s) * 16) : u32x4{0u, 0u, 0u, 0u};
    f.s = TAIL ? scale_dword(srow, b, nb) : *reinterpret_cast<const uint32_t*>(srow + b);
  } else if constexpr (XF == AR_BF16) {
    const int b = 16 * step + 4 * g;
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int at = (b + s) * 32 + 8 * j;               // element
        if (!TAIL) {
          f.d[s][j] = ldg16(row + (int64_t)at * 2);
        } else {
          f.d[s][j] = at < K ? keep_bytes(ldg16(row + (int64_t)at * 2), 2 * (K - at))
                             : u32x4{0u, 0u, 0u, 0u};
        }
      }
  } else {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int b = 16 * step + 4 * ((g >> 1) + 2 * h) + s;
        const int at = b * 32 + 16 * (g & 1);
        if (!TAIL) {
          f.d[s][h] = ldg16(row + at);
        } else if (XF == AR_E4M3_MX) {
          f.d[s][h] = b < nb ? ldg16(row + at) : u32x4{0u, 0u, 0u, 0u};
        } else {
          f.d[s][h] = at < K ? keep_bytes(ldg16(row + at), K - at) : u32x4{0u, 0u, 0u, 0u};
        }
      }
    if constexpr (XF == AR_E4M3_MX) {
      const int b = 16 * step + 4 * g;
      f.s = TAIL ? scale_dword(srow, b, nb) : *reinterpret_cast<const uint32_t*>(srow + b);
    }
  }
}

__device__ __forceinline__ i32x8 operand(u32x4 lo, u32x4 hi) {
  return i32x8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// 8 weights (one dword of codes) as bf16; the conversion reads the scale's
// exponent field alone.
__device__ __forceinline__ bf16x8 weights_bf16(uint32_t codes, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
  return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// One block of each lane group: S is the scales' byte and the block's place.
template <int XF, int S>
__device__ __forceinline__ f32x4 multiply(const WFrag& w, const XFrag<XF>& x, f32x4 acc) {
  constexpr u32x4 none = u32x4{0u, 0u, 0u, 0u};
  if constexpr (XF == AR_BF16) {
    const uint32_t code = (w.s >> (8 * S)) & 0xFFu;
    const float scale = __uint_as_float(code << 23);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          weights_bf16(w.d[S][j], scale), __builtin_bit_cast(bf16x8, x.d[S][j]), acc, 0, 0, 0);
    return acc;
  } else if constexpr (XF == AR_E2M1_MX) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        operand(w.d[S], none), operand(x.d[S], none), acc, 4, 4, S, (int)w.s, S, (int)x.s);
  } else if constexpr (XF == AR_E4M3_MX) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        operand(w.d[S], none), operand(x.d[S][0], x.d[S][1]), acc, 4, 0, S, (int)w.s, S, (int)x.s);
  } else {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        operand(w.d[S], none), operand(x.d[S][0], x.d[S][1]), acc, 4, 0, S, (int)w.s, 0, 127);
  }
}

template <int YF>
__device__ __forceinline__ void store_out4(void* y, int64_t at, int n, int N, bool vec, f32x4 v) {
  typename Elem<YF>::type* p = static_cast<typename Elem<YF>::type*>(y) + at;
  if (vec && n + 4 <= N) {
    if constexpr (YF == AR_BF16) {
      *reinterpret_cast<u32x2*>(p) =
          u32x2{pack2(to_bf16(v[0]), to_bf16(v[1])), pack2(to_bf16(v[2]), to_bf16(v[3]))};
    } else {
      *reinterpret_cast<f32x4*>(p) = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) p[i] = elem_from_f32<YF>(v[i]);
  }
}

// Few tokens: bound by the stream of weights.  A wave holds 16 outputs and
// 16 * MT tokens; WK waves split K step by step and join their sums, in
// order, in shared memory.
template <int XF, int YF, int MT, int WN, int WK>
__global__ __launch_bounds__(kWave * WN * WK) void k_mx_linear_rows(MxLinArgs a) {
  __shared__ f32x4 part[WK > 1 ? WK * WN * MT * kWave : 1];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wk = wave % WK, wn = wave / WK;
  const int c = lane & 15, g = lane >> 4;
  int b = blockIdx.x;
  const int mg = b % a.m_groups;
  b /= a.m_groups;
  const int ng = b % a.n_groups;
  const int r = b / a.n_groups;
  const int n0 = (ng * WN + wn) * 16, m0 = mg * MT * 16;
  const int n = min(n0 + c, a.N - 1);
  const uint8_t* wrow = a.w + r * a.w_rank + n * a.w_stride;
  const uint8_t* wsrow = a.ws + r * a.ws_rank + n * a.ws_stride;
  const uint8_t* xrow[MT];
  const uint8_t* xsrow[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int m = min(m0 + i * 16 + c, a.M - 1);
    xrow[i] = a.x + r * a.x_rank + m * a.x_stride;
    xsrow[i] = a.xs + r * a.xs_rank + m * a.xs_stride;
  }
  f32x4 acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // steps that hold whole blocks only
  const int full = (is_mx_format(XF) ? a.nb : a.K / 32) / 16;
  const int steps = (a.nb + 15) / 16;
  for (int st = wk; st < steps; st += WK) {
    WFrag w;
    XFrag<XF> x[MT];
    if (st < full) {
      load_w<false>(wrow, wsrow, st, g, a.nb, w);
#pragma unroll
      for (int i = 0; i < MT; ++i) load_x<XF, false>(xrow[i], xsrow[i], st, g, a.nb, a.K, x[i]);
    } else {
      load_w<true>(wrow, wsrow, st, g, a.nb, w);
#pragma unroll
      for (int i = 0; i < MT; ++i) load_x<XF, true>(xrow[i], xsrow[i], st, g, a.nb, a.K, x[i]);
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      acc[i] = multiply<XF, 0>(w, x[i], acc[i]);
      acc[i] = multiply<XF, 1>(w, x[i], acc[i]);
      acc[i] = multiply<XF, 2>(w, x[i], acc[i]);
      acc[i] = multiply<XF, 3>(w, x[i], acc[i]);
    }
  }
  if constexpr (WK > 1) {
#pragma unroll
    for (int i = 0; i < MT; ++i) part[((wk * WN + wn) * MT + i) * kWave + lane] = acc[i];
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    if (i % WK != wk) continue;                            // the waves of a group share the tiles
    f32x4 v = acc[i];
    if constexpr (WK > 1) {
      v = part[(wn * MT + i) * kWave + lane];
#pragma unroll
      for (int k = 1; k < WK; ++k) v += part[((k * WN + wn) * MT + i) * kWave + lane];
    }
    const int m = m0 + i * 16 + c;
    if (m >= a.M || n0 + 4 * g >= a.N) continue;
    if constexpr (XF == AR_E4M3_ROW) {
      if (a.K > 0) v *= *reinterpret_cast<const float*>(xsrow[i]);
    }
    store_out4<YF>(a.y, r * a.y_rank + m * a.y_stride + n0 + 4 * g, n0 + 4 * g, a.N, a.vec != 0, v);
  }
}

// ================================================================ host side

static int check_linear(const ar_linear_params* p) {
  if (!p) return AR_EINVAL;
  if (p->nranks < 1 || p->nranks > AR_MAX_RANKS || p->reserved != 0) return AR_EINVAL;
  if (p->rows < 0 || p->outputs < 0 || p->inputs < 0) return AR_EINVAL;
  if (p->x_format != AR_BF16 && (p->x_format < AR_E4M3_ROW || p->x_format > AR_E2M1_MX))
    return AR_EINVAL;
  if (p->y_format != AR_BF16 && p->y_format != AR_F32) return AR_EINVAL;
  if (p->rows == 0 || p->outputs == 0) return AR_OK;
  if (p->rows > (1 << 30) || p->outputs > (1 << 30) || p->inputs > (1 << 30)) return AR_ESIZE;
  if (!p->y || p->y_stride < p->outputs) return AR_EINVAL;
  if (p->x_rank_stride < 0 || p->x_scale_rank_stride < 0 || p->w_rank_stride < 0 ||
      p->w_scale_rank_stride < 0 || p->y_rank_stride < 0)
    return AR_EINVAL;
  const int64_t most = int64_t(1) << 40;
  if (p->y_stride >= most || p->x_rank_stride >= most || p->x_scale_rank_stride >= most ||
      p->w_rank_stride >= most || p->w_scale_rank_stride >= most || p->y_rank_stride >= most)
    return AR_ESIZE;
  if (!aligned(p->y, p->y_format == AR_F32 ? 4 : 2)) return AR_EALIGN;
  int rc = check_format_rows(p->x_format, p->x, p->x_stride, p->rows, p->inputs);
  if (rc) return rc;
  rc = check_scales(p->x_format, p->x_scales, p->x_scale_stride, p->rows, p->inputs);
  if (rc) return rc;
  rc = check_format_rows(AR_E2M1_MX, p->w, p->w_stride, p->outputs, p->inputs);
  if (rc) return rc;
  rc = check_scales(AR_E2M1_MX, p->w_scales, p->w_scale_stride, p->outputs, p->inputs);
  if (rc) return rc;
  if (p->nranks > 1 && p->inputs > 0) {
    if (p->x_rank_stride % (p->x_format == AR_BF16 ? 8 : 16) || p->w_rank_stride % 16 ||
        p->w_scale_rank_stride % 4 ||
        (is_mx_format(p->x_format) && p->x_scale_rank_stride % 4))
      return AR_EALIGN;
  }
  return AR_OK;
}

template <int XF, int YF, int MT>
static hipError_t launch_rows(const MxLinArgs& a0, int nranks, int mt_groups, hipStream_t s) {
  MxLinArgs a = a0;
  a.m_groups = mt_groups;
  const int steps = (a.nb + 15) / 16;
  const int tiles = (a.N + 15) / 16;
  auto go = [&](auto kernel, int wn, int waves) {
    a.n_groups = (tiles + wn - 1) / wn;
    return launch(kernel, dim3((unsigned)((int64_t)nranks * a.n_groups * a.m_groups)),
                  dim3(kWave * waves), s, a);
  };
  if (steps >= 4) return go(k_mx_linear_rows<XF, YF, MT, 1, 4>, 1, 4);
  if (steps >= 2) return go(k_mx_linear_rows<XF, YF, MT, 2, 2>, 2, 4);
  return go(k_mx_linear_rows<XF, YF, MT, 4, 1>, 4, 4);
}

template <int XF, int YF>
static hipError_t launch_linear(const MxLinArgs& a, int nranks, hipStream_t s) {
  if (a.M <= 16) return launch_rows<XF, YF, 1>(a, nranks, 1, s);
  if (a.M <= 32) return launch_rows<XF, YF, 2>(a, nranks, 1, s);
  return launch_rows<XF, YF, 4>(a, nranks, (a.M + 63) / 64, s);
}

template <int XF>
static hipError_t launch_linear_y(const MxLinArgs& a, int yf, int nranks, hipStream_t s) {
  return yf == AR_F32 ? launch_linear<XF, AR_F32>(a, nranks, s)
                      : launch_linear<XF, AR_BF16>(a, nranks, s);
}

}  // namespace ar

using namespace ar;

extern "C" {

int ar_mx4_linear(const ar_linear_params* p, void* stream) {
  const int rc = check_linear(p);
  if (rc) return rc;
  if (p->rows == 0 || p->outputs == 0) return AR_OK;
  // workgroups of the kernel with the smallest tiles (64 outputs or 16, 64 tokens or all)
  const int64_t tiles = ceil_div64(p->outputs, 16) * ceil_div64(p->rows, 64) * p->nranks;
  if (tiles > INT32_MAX) return AR_ESIZE;
  MxLinArgs a{};
  const int64_t xe = p->x_format == AR_BF16 ? 2 : 1;
  const int64_t xse = p->x_format == AR_E4M3_ROW ? 4 : 1;
  a.x = static_cast<const uint8_t*>(p->x);
  a.x_stride = p->x_stride * xe;
  a.x_rank = p->x_rank_stride * xe;
  a.xs = static_cast<const uint8_t*>(p->x_scales);
  a.xs_stride = p->x_format == AR_E4M3_ROW ? 4 : p->x_scale_stride;
  a.xs_rank = p->x_scale_rank_stride * xse;
  a.w = static_cast<const uint8_t*>(p->w);
  a.w_stride = p->w_stride;
  a.w_rank = p->w_rank_stride;
  a.ws = static_cast<const uint8_t*>(p->w_scales);
  a.ws_stride = p->w_scale_stride;
  a.ws_rank = p->w_scale_rank_stride;
  a.y = p->y;
  a.y_stride = p->y_stride;
  a.y_rank = p->y_rank_stride;
  a.M = (int32_t)p->rows;
  a.N = (int32_t)p->outputs;
  a.K = (int32_t)p->inputs;
  a.nb = (int32_t)mx_blocks(p->inputs);
  a.vec = aligned(p->y, p->y_format == AR_F32 ? 16 : 8) && p->y_stride % 4 == 0 &&
          (p->nranks == 1 || p->y_rank_stride % 4 == 0);
  hipStream_t s = static_cast<hipStream_t>(stream);
  switch (p->x_format) {
    case AR_BF16: return map_hip(launch_linear_y<AR_BF16>(a, p->y_format, p->nranks, s));
    case AR_E4M3_ROW: return map_hip(launch_linear_y<AR_E4M3_ROW>(a, p->y_format, p->nranks, s));
    case AR_E4M3_MX: return map_hip(launch_linear_y<AR_E4M3_MX>(a, p->y_format, p->nranks, s));
    default: return map_hip(launch_linear_y<AR_E2M1_MX>(a, p->y_format, p->nranks, s));
  }
}

}  // extern "C"
