// ar_mxlinear.h -- row-parallel linear layer shards on microscaled 4-bit
// weights (gfx950):
//     y_r[m][n] = sum over k of x_r[m][k] * w_r[n][k]
// for every simulated rank r, accumulated in binary32 in the matrix cores: the
// kernels, alone (ar_mxlinear.hip) and with the low-rank adapters of each token
// in their epilogue (ar_adapters.hip).  Internal; not part of the C ABI.
//
// 8- and 4-bit inputs go through the block-scaled matrix instruction, which
// takes the e8m0 scales of both operands as they are.  It adds 8 neighbouring
// products, cut at 13 bits below the largest one's exponent (measured: beside 256,
// products of 2^-5 and its multiples stay); 4-bit products all fit above that,
// of 8-bit ones those far below their neighbours lose bits.  bf16 inputs through
// the bf16 one, the weights converted in registers.  That is exact but at the top
// of the scales: 4 and 6 under 2^127 and 6 under 2^126, 2^128 and more, are past
// bf16's range (and binary32's) and become infinities.  The weights are the first
// operand, so a lane ends with 4 consecutive outputs of one token.
#pragma once

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

// No adapters.
struct NoAdapters {};

template <class A, class B> constexpr bool is_same = false;
template <class A> constexpr bool is_same<A, A> = true;

// Low-rank adapters: token m's is index[m] (none outside 0 .. count - 1), its
// products with the adapter's first matrix are the binary32 row t[m], with zeros
// from `rank` on up to a multiple of 16, and what they add to output n is sum
// over j of t[m][j] * b[n][j].  Strides in bytes.
struct Adapters {
  const int32_t* index;
  const uint8_t* t;
  int64_t t_stride, t_rank;
  const uint8_t* b;
  int64_t b_stride, b_adapter, b_rank;
  // not null: these sums, ready in binary32, element [m][n] of rank r at delta +
  // r * delta_rank + m * delta_stride + n, for tokens with an adapter (never
  // where large_tiles holds)
  const float* delta;
  int64_t delta_stride, delta_rank;
  int32_t count, rank;
};

// Scales of blocks b .. b+15 of a row of `nb`; TAIL: the row's last dword in the
// place of those past its end.
template <bool TAIL>
__device__ __forceinline__ u32x4 load_scales16(const uint8_t* row, int b, int nb) {
  const uint32_t* p = reinterpret_cast<const uint32_t*>(row);
  u32x4 v;
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = p[TAIL ? min(b / 4 + q, (nb - 1) / 4) : b / 4 + q];
  return v;
}

// ... with the scale 1 for every block past the end: what lies there may be
// anything, a NaN too.
__device__ __forceinline__ u32x4 keep_scales(u32x4 v, int b, int nb) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int n = nb - b - 4 * q;
    const uint32_t keep = n >= 4 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << (8 * n)) - 1u);
    v[q] = (v[q] & keep) | (0x7F7F7F7Fu & ~keep);
  }
  return v;
}

// The first `keep` bits of 128, zeros after them.
__device__ __forceinline__ u32x4 keep_bits(u32x4 v, int64_t keep) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const int64_t k = keep - 32 * d;
    v[d] &= k >= 32 ? 0xFFFFFFFFu : (k <= 0 ? 0u : (1u << k) - 1u);
  }
  return v;
}

// Bits of one element of an input row.
template <int XF>
constexpr int elem_bits() { return XF == AR_BF16 ? 16 : (XF == AR_E2M1_MX ? 4 : 8); }

// 16 bytes of an input row from element `at` on, with zeros at and past element
// K: what lies there in x does not count, and then neither does what lies there
// in w, whose values are finite but for bf16 tokens (keep_weights).
template <int XF>
__device__ __forceinline__ u32x4 keep_inputs(u32x4 v, int64_t at, int64_t K) {
  return keep_bits(v, (K - at) * elem_bits<XF>());
}

// The same for 32 weights, which as bf16 may be infinite.
__device__ __forceinline__ u32x4 keep_weights(u32x4 v, int64_t at, int64_t K) {
  return keep_bits(v, (K - at) * 4);
}

// 8 e4m3 codes times a scale as bf16, without loss in its range.
__device__ __forceinline__ bf16x8 tokens_bf16(uint32_t lo, uint32_t hi, float scale) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// Whether 8-bit tokens go through the bf16 instruction (as bf16, converted in
// registers), which loses nothing: for binary32 outputs with adapters.
template <int XF, int YF, class AD>
constexpr bool exact8() {
  return !is_same<AD, NoAdapters> && YF == AR_F32 && (XF == AR_E4M3_ROW || XF == AR_E4M3_MX);
}

// One lane's operands of a 512-element step: 4 blocks of K, one in each of 4
// matrix instructions, and the row's 16 scales.
template <int XF>
struct XFrag;
template <> struct XFrag<AR_E4M3_MX> { u32x4 d[4][2]; u32x4 s; };
template <> struct XFrag<AR_E4M3_ROW> { u32x4 d[4][2]; };
template <> struct XFrag<AR_E2M1_MX> { u32x4 d[4]; u32x4 s; };
template <> struct XFrag<AR_BF16> { u32x4 d[4][4]; };

struct WFrag {
  u32x4 d[4];
  u32x4 s;
};

// Group g = lane / 16 of a wave holds block 4s + g of the step in instruction
// s, so that the four groups read 64 bytes of a row together.  (With blocks
// 4g .. 4g + 3 to group g the four scales of a lane share a dword, but each
// load then touches all the step's lines and they do not stay in the L1: 4
// ranks of 16 x 8192 x 2048 took 15.2 us.)
// The instruction wants 4-bit operands as block g's 32 values in group g, but
// 8-bit ones as values [16g', 16g' + 16) of the 128, for g' = g and g + 4 --
// while group g gives the scale of block g in either case.
// TAIL: a step that K ends in, which reads the row's last piece again in the
// place of those past its end; keep_step then takes out what does not count.
template <bool TAIL>
__device__ __forceinline__ void load_w(const uint8_t* row, const uint8_t* srow, int step, int g, int nb,
                                       WFrag& f) {
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int b = 16 * step + 4 * s + g;
    f.d[s] = ldg16(row + (int64_t)(TAIL ? min(b, nb - 1) : b) * 16);
  }
  f.s = load_scales16<TAIL>(srow, 16 * step, nb);
}

// First element of piece q of instruction s in group g's operand of a step.
template <int XF, bool EX = false>
__device__ __forceinline__ int64_t input_at(int step, int s, int g, int q) {
  if constexpr (EX) return (int64_t)(16 * step + 4 * s + g) * 32 + 16 * q;
  else if constexpr (XF == AR_E2M1_MX) return (int64_t)(16 * step + 4 * s + g) * 32;
  else if constexpr (XF == AR_BF16) return (int64_t)(16 * step + 4 * s + g) * 32 + 8 * q;
  else return (int64_t)(16 * step + 4 * s) * 32 + 64 * q + 16 * g;
}
template <int XF> constexpr int input_pieces() { return XF == AR_E2M1_MX ? 1 : (XF == AR_BF16 ? 4 : 2); }

template <int XF>
__device__ __forceinline__ u32x4& input_piece(XFrag<XF>& f, int s, int q) {
  if constexpr (XF == AR_E2M1_MX) return f.d[s];
  else return f.d[s][q];
}

template <int XF, bool TAIL, bool EX>
__device__ __forceinline__ void load_x(const uint8_t* row, const uint8_t* srow, int step, int g, int nb,
                                       int K, XFrag<XF>& f) {
  constexpr int per = 128 / elem_bits<XF>();               // elements of 16 bytes
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int q = 0; q < input_pieces<XF>(); ++q) {
      int64_t at = input_at<XF, EX>(step, s, g, q);
      if (TAIL) at = min(at, (int64_t)((K - 1) / per) * per);
      input_piece<XF>(f, s, q) = ldg16(row + at * elem_bits<XF>() / 8);
    }
  if constexpr (is_mx_format(XF)) f.s = load_scales16<TAIL>(srow, 16 * step, nb);
}

template <int XF, bool EX>
__device__ __forceinline__ void keep_step(int step, int g, int nb, int K, XFrag<XF>& f) {
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int q = 0; q < input_pieces<XF>(); ++q)
      input_piece<XF>(f, s, q) = keep_inputs<XF>(input_piece<XF>(f, s, q), input_at<XF, EX>(step, s, g, q), K);
  if constexpr (is_mx_format(XF)) f.s = keep_scales(f.s, 16 * step, nb);
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

// Instruction S of a step; `shift` brings block 4S + g's scale to the lowest
// byte, the one the instruction reads.
template <int XF, int S, bool EX>
__device__ __forceinline__ f32x4 multiply(const WFrag& w, const XFrag<XF>& x, int shift, f32x4 acc) {
  constexpr u32x4 none = u32x4{0u, 0u, 0u, 0u};
  const uint32_t ws = w.s[S] >> shift;
  if constexpr (EX) {
    const float scale = __uint_as_float((ws & 0xFFu) << 23);
    float xscale = 1.0f;
    if constexpr (is_mx_format(XF)) xscale = __uint_as_float((x.s[S] >> shift & 0xFFu) << 23);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const u32x4 d = x.d[S][j / 2];
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          weights_bf16(w.d[S][j], scale),
          j % 2 ? tokens_bf16(d.z, d.w, xscale) : tokens_bf16(d.x, d.y, xscale), acc, 0, 0, 0);
    }
    return acc;
  } else if constexpr (XF == AR_BF16) {
    const float scale = __uint_as_float((ws & 0xFFu) << 23);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
          weights_bf16(w.d[S][j], scale), __builtin_bit_cast(bf16x8, x.d[S][j]), acc, 0, 0, 0);
    return acc;
  } else if constexpr (XF == AR_E2M1_MX) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        operand(w.d[S], none), operand(x.d[S], none), acc, 4, 4, 0, (int)ws, 0, (int)(x.s[S] >> shift));
  } else if constexpr (XF == AR_E4M3_MX) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        operand(w.d[S], none), operand(x.d[S][0], x.d[S][1]), acc, 4, 0, 0, (int)ws, 0,
        (int)(x.s[S] >> shift));
  } else {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        operand(w.d[S], none), operand(x.d[S][0], x.d[S][1]), acc, 4, 0, 0, (int)ws, 0, 127);
  }
}

template <int YF>
__device__ __forceinline__ void store_out4(void* y, int64_t at, int n, int N, bool vec, f32x4 v) {
  typename Elem<YF>::type* p = static_cast<typename Elem<YF>::type*>(y) + at;
  if (vec && n + 4 <= N) {
    if constexpr (YF == AR_BF16) {
      *reinterpret_cast<u32x2*>(p) = u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    } else {
      *reinterpret_cast<f32x4*>(p) = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (n + i < N) p[i] = elem_from_f32<YF>(v[i]);
  }
}

// A binary32 value as P bf16 values whose sum it is, to 16 bits for 2 and to all
// 24 for 3: the leading ones cut, so none of them overflows, the last rounded.
// Infinities and NaNs are in the first alone.
template <int P>
__device__ __forceinline__ void bf16_parts(float v, uint32_t (&p)[P]) {
  const uint32_t bits = __float_as_uint(v);
  const bool fine = abs_bits(v) < kInfBits;
  p[0] = abs_bits(v) > kInfBits ? 0x7FC0u : bits >> 16;
  float rest = fine ? v - __uint_as_float(bits & 0xFFFF0000u) : 0.0f;
  if constexpr (P == 3) {
    const uint32_t next = __float_as_uint(rest) & 0xFFFF0000u;
    p[1] = next >> 16;
    rest -= __uint_as_float(next);
  }
  p[P - 1] = bf16_pair(rest, 0.0f) & 0xFFFFu;
}

// Sums that are ready, for TI x TJ tiles of 16 outputs by 16 tokens.
template <int TI, int TJ, class Acc>
__device__ __forceinline__ void add_delta(const Adapters& ad, const MxLinArgs& a, int r, int m0, int n0, Acc acc) {
  const int c = threadIdx.x & 15, g = threadIdx.x >> 4 & 3;
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    const int m = m0 + 16 * j + c;
    const bool has = m < a.M && (uint32_t)ad.index[min(m, a.M - 1)] < (uint32_t)ad.count;
    const float* row = ad.delta + r * ad.delta_rank + (int64_t)min(m, a.M - 1) * ad.delta_stride;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int n = n0 + 16 * i + 4 * g;
      if (has && n < a.N) acc(i, j) += *reinterpret_cast<const f32x4*>(row + n);
    }
  }
}

// 8 values of an adapter's row of b from dimension `at` on, zeros from `rank` on.
__device__ __forceinline__ u32x4 load_b8(const uint8_t* row, int at, int rank) {
  u32x4 v = u32x4{0u, 0u, 0u, 0u};
  if (at < rank) v = ldg16(row + at * 2);
  return v;
}
__device__ __forceinline__ u32x4 keep_b8(u32x4 v, int at, int rank) {
  return at + 8 > rank ? keep_inputs<AR_BF16>(v, at, rank) : v;
}

// What adapters add to TI x TJ tiles of 16 outputs by 16 tokens where there are
// few: every lane by itself, for its token (lane % 16 of each group) and the 4
// outputs of its group, in binary32 products and sums.  No two tokens need the
// same adapter for it, there is nothing to find out, and the loads do not wait for
// each other.  ROOM: registers for the first 16 dimensions' operands beside
// the layer's own, so that they are loaded before its products.
template <int TI, int TJ, bool ROOM>
struct AdapterLanes {
  int mine[TJ];                      // -1: none
  const uint8_t* t[TJ];
  const uint8_t* b[TJ];              // of the first output, this token's adapter
  int n, last;                       // this lane's first output, and the last there is
  f32x4 tv[ROOM ? TJ : 1][4];
  u32x4 w[ROOM ? TI * TJ : 1][4][2];

  // m0: the first token, n0: the first output.
  __device__ __forceinline__ void find(const Adapters& ad, const MxLinArgs& a, int r, int m0, int n0) {
    const int c = threadIdx.x & 15, g = threadIdx.x >> 4 & 3;
    n = n0 + 4 * g;
    last = a.N - 1;
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int m = m0 + 16 * j + c;
      mine[j] = m < a.M ? ad.index[m] : -1;
      t[j] = ad.t + r * ad.t_rank + (int64_t)min(m, a.M - 1) * ad.t_stride;
    }
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      if ((uint32_t)mine[j] >= (uint32_t)ad.count) mine[j] = -1;
      b[j] = ad.b + r * ad.b_rank + mine[j] * ad.b_adapter;
    }
  }
  // Dimensions q .. q + 15.
  __device__ __forceinline__ void load_t(int j, int q, f32x4 (&v)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (mine[j] >= 0) v[k] = *reinterpret_cast<const f32x4*>(t[j] + (q + 4 * k) * 4);
    }
  }
  __device__ __forceinline__ void load_b(const Adapters& ad, int i, int j, int q, u32x4 (&v)[4][2]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint8_t* row = b[j] + min(n + 16 * i + e, last) * ad.b_stride;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        v[e][k] = u32x4{0u, 0u, 0u, 0u};
        if (mine[j] >= 0) v[e][k] = load_b8(row, q + 8 * k, ad.rank);
      }
    }
  }
  static __device__ __forceinline__ void add(const Adapters& ad, int q, const f32x4 (&x)[4], const u32x4 (&v)[4][2],
                                             f32x4& sum) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const u32x4 y = keep_b8(v[e][k], q + 8 * k, ad.rank);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          s = __builtin_fmaf(x[2 * k + u / 2][u % 2 * 2], bf_lo(y[u]), s);
          s = __builtin_fmaf(x[2 * k + u / 2][u % 2 * 2 + 1], bf_hi(y[u]), s);
        }
      }
      sum[e] += s;
    }
  }
  // Where the layer's first loads are under way.
  __device__ __forceinline__ void start(const Adapters& ad, const MxLinArgs& a, int r, int m0, int n0) {
    find(ad, a, r, m0, n0);
    if constexpr (ROOM) {
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        load_t(j, 0, tv[j]);
#pragma unroll
        for (int i = 0; i < TI; ++i) load_b(ad, i, j, 0, w[i * TJ + j]);
      }
    }
  }
  template <class Acc>
  __device__ __forceinline__ void finish(const Adapters& ad, Acc acc) {
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      if (!__any(mine[j] >= 0)) continue;
      f32x4 sum[TI];
#pragma unroll
      for (int i = 0; i < TI; ++i) sum[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if constexpr (ROOM) {
#pragma unroll
        for (int i = 0; i < TI; ++i) add(ad, 0, tv[j], w[i * TJ + j], sum[i]);
      }
      for (int q = ROOM ? 16 : 0; q < ad.rank; q += 16) {
        f32x4 x[4];
        u32x4 v[TI][4][2];
        load_t(j, q, x);
#pragma unroll
        for (int i = 0; i < TI; ++i) load_b(ad, i, j, q, v[i]);
#pragma unroll
        for (int i = 0; i < TI; ++i) add(ad, q, x, v[i], sum[i]);
      }
      if (mine[j] >= 0) {
#pragma unroll
        for (int i = 0; i < TI; ++i) acc(i, j) += sum[i];
      }
    }
  }
};

// Up to 16 tokens: bound by the stream of weights.  A wave holds 16 * NT outputs
// and the tokens; WK waves split K step by step and join their sums, in order,
// in shared memory.  The next step's operands are on their way while one is
// multiplied.  4 shards of 8192 x 2048, 8-bit: one token 10.3 us with the weights
// in HBM, 3.5 TB/s with the launch, which takes 2, and 8.7 with them in the last
// cache; 8 tokens 11.4 and 10.0; 8 shards of 4096 x 512, bf16: 5.3 and 4.3.
template <int XF, int YF, int NT, int WN, int WK, class AD>
__global__ __launch_bounds__(kWave * WN * WK) void k_mx_linear_rows(MxLinArgs a, AD ad) {
  __shared__ f32x4 part[WK > 1 ? WK * WN * NT * kWave : 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wk = wave % WK, wn = wave / WK;
  const int c = lane & 15, g = lane >> 4, shift = 8 * g;
  constexpr bool EX = exact8<XF, YF, AD>();
  int b = blockIdx.x;
  const int mg = b % a.m_groups;
  b /= a.m_groups;
  const int ng = b % a.n_groups;
  const int r = b / a.n_groups;
  const int n0 = (ng * WN + wn) * 16 * NT, m = mg * 16 + c;
  const uint8_t *wrow[NT], *wsrow[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {                           // rows past the end read the last one
    const int n = min(n0 + i * 16 + c, a.N - 1);
    wrow[i] = a.w + r * a.w_rank + n * a.w_stride;
    wsrow[i] = a.ws + r * a.ws_rank + n * a.ws_stride;
  }
  const uint8_t* xrow = a.x + r * a.x_rank + min(m, a.M - 1) * a.x_stride;
  const uint8_t* xsrow = a.xs + r * a.xs_rank + min(m, a.M - 1) * a.xs_stride;
  // this wave's output tiles: all, or one of those that the group shares
  constexpr int own = WK == 1 ? NT : 1;
  AdapterLanes<own, 1, true> tiles;
  f32x4 acc[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  struct Step {
    WFrag w[NT];
    XFrag<XF> x;
  };
  const int full = a.K / 512, steps = (a.nb + 15) / 16;    // the last step may be one that K ends in
  auto load = [&](int st, Step& f) {
    if (st < full) {
#pragma unroll
      for (int i = 0; i < NT; ++i) load_w<false>(wrow[i], wsrow[i], st, g, a.nb, f.w[i]);
      load_x<XF, false, EX>(xrow, xsrow, st, g, a.nb, a.K, f.x);
    } else {
#pragma unroll
      for (int i = 0; i < NT; ++i) load_w<true>(wrow[i], wsrow[i], st, g, a.nb, f.w[i]);
      load_x<XF, true, EX>(xrow, xsrow, st, g, a.nb, a.K, f.x);
    }
  };
  auto keep = [&](int st, Step& f) {
    if (st < full) return;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      f.w[i].s = keep_scales(f.w[i].s, 16 * st, a.nb);
      if constexpr (XF == AR_BF16 || EX) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          f.w[i].d[q] = keep_weights(f.w[i].d[q], (int64_t)(16 * st + 4 * q + g) * 32, a.K);
      }
    }
    keep_step<XF, EX>(st, g, a.nb, a.K, f.x);
  };
  auto compute = [&](const Step& f) {
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = multiply<XF, 0, EX>(f.w[i], f.x, shift, acc[i]);
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = multiply<XF, 1, EX>(f.w[i], f.x, shift, acc[i]);
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = multiply<XF, 2, EX>(f.w[i], f.x, shift, acc[i]);
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = multiply<XF, 3, EX>(f.w[i], f.x, shift, acc[i]);
  };
  auto start = [&]() {                                     // beside the layer's first loads
    if constexpr (!is_same<AD, NoAdapters>) {
      if (!ad.delta && wk < NT) tiles.start(ad, a, r, mg * 16, n0 + (WK == 1 ? 0 : 16 * wk));
    }
  };
  if (wk < steps) {
    Step cur;
    int st = wk;
    load(st, cur);
    start();
    for (; st + WK < steps; st += WK) {
      Step next;
      load(st + WK, next);
      compute(cur);                                        // never the last step
      cur = next;
    }
    keep(st, cur);
    compute(cur);
  } else {
    start();
  }
  if constexpr (WK > 1) {
#pragma unroll
    for (int i = 0; i < NT; ++i) part[((wk * WN + wn) * NT + i) * kWave + lane] = acc[i];
    __syncthreads();
  }
  f32x4 sums[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    if (i % WK != wk) continue;                            // the waves of a group share the tiles
    f32x4 v = acc[i];
    if constexpr (WK > 1) {
      v = part[(wn * NT + i) * kWave + lane];
#pragma unroll
      for (int k = 1; k < WK; ++k) v += part[((k * WN + wn) * NT + i) * kWave + lane];
    }
    if constexpr (XF == AR_E4M3_ROW) {
      if (a.K > 0) v *= *reinterpret_cast<const float*>(xsrow);
    }
    sums[i] = v;
  }
  if constexpr (!is_same<AD, NoAdapters>) {
    if (ad.delta) {
#pragma unroll
      for (int i = 0; i < NT; ++i)
        if (i % WK == wk) add_delta<1, 1>(ad, a, r, mg * 16, n0 + 16 * i, [&](int, int) -> f32x4& { return sums[i]; });
    } else if constexpr (WK == 1) {
      tiles.finish(ad, [&](int i, int) -> f32x4& { return sums[i]; });
    } else {
#pragma unroll
      for (int i = 0; i < NT; ++i)
        if (i == wk) tiles.finish(ad, [&](int, int) -> f32x4& { return sums[i]; });
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    if (i % WK != wk) continue;
    const int n = n0 + i * 16 + 4 * g;
    if (m >= a.M || n >= a.N) continue;
    store_out4<YF>(a.y, r * a.y_rank + m * a.y_stride + n, n, a.N, a.vec != 0, sums[i]);
  }
}

// ---------------------------------------------------------- many tokens ---
//
// Bound by the matrix cores.  A workgroup holds BN outputs by BM tokens; K goes by
// in steps, NS steps' codes in shared memory: while one is multiplied the ones
// after it are on their way, loaded straight into shared memory, and one barrier
// a step is enough.  Rows lie there as they come, 16-byte pieces permuted by the
// row so that the lanes that read at once meet different banks; the loads apply
// the permutation to their addresses.  Scales come 512 elements of K at a time,
// one row a lane.
// 4096 x 8192 x 8192: 8-bit tokens 198 to 217 us from run to run (2.5 to 2.8
// PFLOP/s), 4-bit 162 to 180 (3.1 to 3.4), bf16 375 to 405 (1.36 to 1.46); the
// instructions alone, on registers, do 4.6, 8.3 and 2.2.  With 8-bit tokens the
// matrix cores are busy 62% of the time.  In a form of 208 us, the operands' way
// into shared memory and registers took 178 us without any product, the products
// 141 without operands: they overlap in part only, and the two steps on their way
// are all that shared memory holds.

// 16 bytes a lane from the buffer straight into shared memory, at `lds` (the
// wave's own address) + 16 * lane.
__device__ __forceinline__ void load_to_lds(rsrc_t r, uint8_t* lds, uint32_t lane_off) {
  typedef __attribute__((address_space(3))) void lds_void;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, lane_off, 0, 0, 0);
}

__device__ __forceinline__ void load_to_lds(const uint8_t* p, uint8_t* lds) {
  typedef __attribute__((address_space(3))) void lds_void;
  typedef const __attribute__((address_space(1))) void global_void;
  __builtin_amdgcn_global_load_lds((global_void*)p, (lds_void*)lds, 16, 0, 0);
}

template <int XF, int BK_, bool EX>
struct TileShape {
  static constexpr int BK = BK_;                           // elements of K a step
  static constexpr int BI = XF == AR_BF16 || EX ? 64 : 128; // and of one round of instructions
  static constexpr int rounds = BK / BI;
  static constexpr int XB = XF == AR_BF16 ? 2 * BK : (XF == AR_E2M1_MX ? BK / 2 : BK);  // bytes of an x row
  static constexpr int WB = BK / 2;                        // bytes of a weight row
  static constexpr int XC = XB / 16, WC = WB / 16;         // 16-byte pieces
  static constexpr int steps_scales = 512 / BK;            // steps that share 16 scales a row
};

// Where piece `c` of row `r` lies among the row's C pieces: 8 rows that are
// read together cover every 16-byte column of 128 bytes.
template <int C>
__device__ __forceinline__ int place(int r, int c) {
  if constexpr (C >= 8) return c ^ (r & 7);
  else if constexpr (C == 4) return c ^ ((r >> 1) & 3);
  else return c ^ ((r >> 2) & 1);
}

__device__ __forceinline__ void barrier_only() {
  compiler_barrier();
  __builtin_amdgcn_s_barrier();
  compiler_barrier();
}

// KG groups of waves share a step's rounds among them and join their sums at
// the end: more waves, and fewer steps one after the other, where there are few
// tiles.
template <int XF_, int YF_, bool EX_, int BK_, int BM_, int BN_, int WM_, int WN_, int NS_, int KG_ = 1>
struct Tile {
  static constexpr int XF = XF_, YF = YF_, BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_,
                       KG = KG_;
  static constexpr bool EX = EX_;
  using T = TileShape<XF, BK_, EX>;
  static constexpr int tile_waves = (BM / WM) * (BN / WN), waves = tile_waves * KG;
  static constexpr int threads = waves * kWave;
  static constexpr int xbytes = BM * T::XB, wbytes = BN * T::WB;
  static constexpr int stage = xbytes + wbytes;
  // 16-byte pieces of a step, and loads of a thread (where there are fewer
  // pieces than threads, some load a piece that another one loads too)
  static constexpr int px = xbytes / 16, pw = wbytes / 16;
  static constexpr int nx = (px + threads - 1) / threads, nw = (pw + threads - 1) / threads;
  // rows of scales: the weights', then the tokens' where they have some
  static constexpr int srows = is_mx_format(XF) ? BM + BN : BN;
  static constexpr int swaves = (srows + kWave - 1) / kWave;
  static constexpr int ns = (swaves + waves - 1) / waves;
  static constexpr int scales = swaves * kWave * 16;
  // runs of scales held: the one in use and the next, or one a step
  static constexpr int runs = T::steps_scales > 1 ? 2 : NS;
  static constexpr int lds = NS * stage + runs * scales;
  static_assert(px % kWave == 0 && pw % kWave == 0, "whole waves load");
  static_assert(threads % px == 0 || px % threads == 0, "");
  static_assert(threads % pw == 0 || pw % threads == 0, "");
  static_assert(waves % swaves == 0 || swaves % waves == 0, "");
  static_assert(NS - 1 <= T::steps_scales || T::steps_scales == 1, "scales of two runs of steps at a time");
  static_assert(KG == 1 || KG == T::rounds, "a round for each group");
  static_assert(KG == 1 || tile_waves * WM * WN * 4 * KG <= lds, "room to join the sums");
  static_assert((NS - 2) * (nx + nw) < 64, "loads on their way that a wait can name");
};

// Whether one of two bf16 values is an infinity or a NaN.
__device__ __forceinline__ bool bf16_odd(uint32_t v) {
  return (v & 0x7F80u) == 0x7F80u || (v & 0x7F800000u) == 0x7F800000u;
}

// What adapters add to a workgroup's BM tokens by BN outputs: one adapter after the other, for the tokens that have it (those of a
// request stand together, so most often there are one or two), and two at a time
// where their dimensions fit into one matrix instruction.  The layer's operands are
// done with, so t and the adapter's rows of b go through shared memory, 32 dimensions
// at a time, the next adapter's rows on their way in registers.  Tokens with other
// adapters have zeros for t there, so their sums stay as they are (but for a zero's
// sign); where rows of b have infinities or NaNs, which zeros would make NaN, the sums
// are taken for their own tokens alone.
// t's values go as 2 bf16 parts for bf16 outputs, as 3, which is all of them, for
// binary32 ones.
// Bound by its own chain of loads (index, t, rows) where there are few adapters, by
// the products of all tiles of 16 tokens with every adapter that one of them has
// where there are many: 4096 x 8192 x 8192, 8-bit tokens, 196 us without adapters, 8
// requests with one of rank 16 each 219, of rank 64 235 (23 and 4 of them t), 16
// adapters of rank 16 in any order 265.  Rows of three adapters on their way, and
// t in registers, changed nothing.
template <class G, class Acc>
__device__ __forceinline__ void add_adapters(const Adapters& ad, const MxLinArgs& a, int r, int m0, int n0, int wm,
                                             int wn, uint8_t* smem, Acc acc) {
  constexpr int P = G::YF == AR_F32 ? 3 : 2, TI = G::WN / 16, TJ = G::WM / 16, threads = G::threads;
  constexpr int TS = 64 * P + 16, BS = 64 + 16;            // 16 rows' reads meet different banks
  constexpr int pieces = G::BN * 4 / threads, sets = G::BM / kWave;
  static_assert(G::KG == 1 && TI % 4 == 0 && G::BM % kWave == 0 && G::BN * 4 % threads == 0, "");
  static_assert(G::BM * (4 + TS) + 2 * G::BN * BS + 8 <= G::lds, "room for t and b");
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, g = lane >> 4;
  int* ids = reinterpret_cast<int*>(smem);
  uint8_t *ts = smem + G::BM * 4, *bs = ts + G::BM * TS;
  int* odd = reinterpret_cast<int*>(bs + 2 * G::BN * BS);   // the last turn whose rows were odd, of each buffer
  __syncthreads();
  for (int i = tid; i < G::BM; i += threads) {
    const int which = m0 + i < a.M ? ad.index[m0 + i] : -1;
    ids[i] = (uint32_t)which < (uint32_t)ad.count ? which : -1;
  }
  if (tid < 2) odd[tid] = -1;
  __syncthreads();
  int mine[sets], of[TJ];            // adapters of the workgroup's tokens, and of this lane's
  uint64_t all[sets], left[sets], any = 0;
#pragma unroll
  for (int j = 0; j < TJ; ++j) of[j] = ids[wm + 16 * j + c];
#pragma unroll
  for (int k = 0; k < sets; ++k) {
    mine[k] = ids[64 * k + lane];
    all[k] = __ballot(mine[k] >= 0);
    any |= all[k];
  }
  auto next = [&]() {
    int which = -1;
#pragma unroll
    for (int k = 0; k < sets; ++k)
      if (which < 0 && left[k] != 0) which = __builtin_amdgcn_readlane(mine[k], __builtin_ctzll(left[k]));
#pragma unroll
    for (int k = 0; k < sets; ++k) left[k] &= ~__ballot(mine[k] == which);
    return which;
  };
  if (any == 0) return;
  const bool two = ad.rank <= 16;                          // adapters at a time: dimensions 16 on are the second one's
  int turn = 0;
  for (int q = 0; q < ad.rank; q += 32) {
    int which[2];
    u32x4 w[pieces];
    auto load_rows = [&]() {
      which[0] = next();
      which[1] = two ? next() : which[0];
      if (which[0] < 0) return;
#pragma unroll
      for (int i = 0; i < pieces; ++i) {
        const int s = i * threads + tid, row = s / 4, at = two ? 8 * (s % 2) : q + 8 * (s % 4);
        const uint8_t* b = ad.b + r * ad.b_rank + (s % 4 < 2 || which[1] < 0 ? which[0] : which[1]) * ad.b_adapter;
        w[i] = load_b8(b + min(n0 + row, a.N - 1) * ad.b_stride, at, ad.rank);
      }
    };
#pragma unroll
    for (int k = 0; k < sets; ++k) left[k] = all[k];
    load_rows();
    for (int s = tid; s < G::BM * 4; s += threads) {
      const int row = s / 4, at = two ? 8 * (s % 2) : q + 8 * (s % 4);
      f32x4 v[2] = {f32x4{0.0f, 0.0f, 0.0f, 0.0f}, f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
      if (ids[row] >= 0 && at < ad.rank) {
        const uint8_t* t = ad.t + r * ad.t_rank + (m0 + row) * ad.t_stride + at * 4;
        v[0] = *reinterpret_cast<const f32x4*>(t);
        v[1] = *reinterpret_cast<const f32x4*>(t + 16);
      }
      u32x4 p[P];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t lo[P], hi[P];
        bf16_parts<P>(v[e / 2][e % 2 * 2], lo);
        bf16_parts<P>(v[e / 2][e % 2 * 2 + 1], hi);
#pragma unroll
        for (int k = 0; k < P; ++k) p[k][e] = pack2(lo[k], hi[k]);
      }
#pragma unroll
      for (int k = 0; k < P; ++k) *reinterpret_cast<u32x4*>(ts + row * TS + s % 4 * (16 * P) + 16 * k) = p[k];
    }
    while (which[0] >= 0) {
      const int buf = turn & 1, now[2] = {which[0], which[1]};
      uint8_t* rows = bs + buf * G::BN * BS;
      bool some = false;
#pragma unroll
      for (int i = 0; i < pieces; ++i) {
        const int s = i * threads + tid;
        const u32x4 v = keep_b8(w[i], two ? 8 * (s % 2) : q + 8 * (s % 4), ad.rank);
        some |= bf16_odd(v.x) || bf16_odd(v.y) || bf16_odd(v.z) || bf16_odd(v.w);
        *reinterpret_cast<u32x4*>(rows + s / 4 * BS + s % 4 * 16) = v;
      }
      if (some) odd[buf] = turn;
      __syncthreads();                                   // the other buffer's readers are through, too
      load_rows();
      const bool apart = odd[buf] == turn;
      ++turn;
      const int want = g < 2 ? now[0] : now[1];
      // this wave's rows of b, 4 tiles of outputs at a time
#pragma unroll
      for (int i0 = 0; i0 < TI; i0 += 4) {
        u32x4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = *reinterpret_cast<const u32x4*>(rows + (wn + 16 * (i0 + i) + c) * BS + g * 16);
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
          const bool take = of[j] >= 0 && of[j] == want;
          if (!__any(take)) continue;
          u32x4 t[P];
#pragma unroll
          for (int k = 0; k < P; ++k) {
            t[k] = *reinterpret_cast<const u32x4*>(ts + (wm + 16 * j + c) * TS + g * (16 * P) + 16 * k);
#pragma unroll
            for (int e = 0; e < 4; ++e) t[k][e] = take ? t[k][e] : 0u;
          }
          if (!apart) {
#pragma unroll
            for (int k = 0; k < P; ++k)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                acc(i0 + i, j) = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8, x[i]), __builtin_bit_cast(bf16x8, t[k]), acc(i0 + i, j), 0, 0, 0);
          } else {
            for (int half = 0; half < (two ? 2 : 1); ++half) {
              const bool part = !two || (g >= 2) == (half == 1), own = of[j] >= 0 && of[j] == now[half];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                f32x4 v = acc(i0 + i, j);
#pragma unroll
                for (int k = 0; k < P; ++k)
                  v = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                      __builtin_bit_cast(bf16x8, part ? x[i] : u32x4{0u, 0u, 0u, 0u}),
                      __builtin_bit_cast(bf16x8, t[k]), v, 0, 0, 0);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc(i0 + i, j)[e] = own ? v[e] : acc(i0 + i, j)[e];
              }
            }
          }
          __builtin_amdgcn_sched_barrier(0);               // one tile's operands at a time: the sums fill the registers
        }
      }
    }
    __syncthreads();                                       // t may be written over
  }
}

template <class G, class AD>
__global__ __launch_bounds__(G::threads) void k_mx_linear_tiles(MxLinArgs a, AD ad) {
  using T = typename G::T;
  constexpr int XF = G::XF, YF = G::YF, BM = G::BM, BN = G::BN, WM = G::WM, WN = G::WN, NS = G::NS;
  constexpr bool EX = G::EX;
  constexpr int TI = WN / 16, TJ = WM / 16;                // matrix tiles of a wave
  __shared__ __align__(256) uint8_t smem[G::lds];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int kg = wave / G::tile_waves, tw = wave % G::tile_waves;
  const int wi = tw % (BN / WN), wj = tw / (BN / WN);

  // Workgroups go round the 8 XCDs one by one; each XCD takes a run of tiles
  // that walks down strips of 8 tiles of outputs, so that the 32 tiles it
  // holds at a time share few rows of either operand in its own L2.
  const int total = gridDim.x;
  int b = blockIdx.x;
  {
    const int per = total / 8, extra = total % 8, xcd = b % 8, k = b / 8;
    b = xcd * per + min(xcd, extra) + k;
  }
  const int per_rank = a.n_groups * a.m_groups;
  const int r = b / per_rank;
  b -= r * per_rank;
  constexpr int strip = 8;
  const int s0 = b / (strip * a.m_groups) * strip;         // first output tile of the strip
  const int width = min(strip, a.n_groups - s0);
  b -= s0 * a.m_groups;
  const int n0 = (s0 + b % width) * BN, m0 = b / width * BM;

  const uint8_t* xbase = a.x + r * a.x_rank + m0 * a.x_stride;
  const uint8_t* wbase = a.w + r * a.w_rank + n0 * a.w_stride;
  const int mlast = a.M - 1 - m0, nlast = a.N - 1 - n0;    // rows past the end read the last one
  // ranges to the 16-byte boundary after the tile's last row
  const int64_t xrange = min(mlast, BM - 1) * a.x_stride + ((int64_t)a.K * elem_bits<XF>() + 127) / 128 * 16;
  const int64_t wrange = min(nlast, BN - 1) * a.w_stride + (int64_t)a.nb * 16;
  const rsrc_t xr = make_rsrc(xbase, (uint32_t)xrange), wr = make_rsrc(wbase, (uint32_t)wrange);

  // This thread's pieces: source offsets in the next step to be loaded.  The step
  // is part of them, not a scalar offset beside them: what ends a read at the
  // buffer's range is sure to look at this one.
  uint32_t xo[G::nx], wo[G::nw];
#pragma unroll
  for (int i = 0; i < G::nx; ++i) {
    const int at = (i * G::threads + tid) % G::px, row = at / T::XC;
    xo[i] = (uint32_t)min(row, mlast) * (uint32_t)a.x_stride + place<T::XC>(row, at % T::XC) * 16;
  }
#pragma unroll
  for (int i = 0; i < G::nw; ++i) {
    const int at = (i * G::threads + tid) % G::pw, row = at / T::WC;
    wo[i] = (uint32_t)min(row, nlast) * (uint32_t)a.w_stride + place<T::WC>(row, at % T::WC) * 16;
  }
  auto load_next = [&](int buf) {
    uint8_t* at = smem + buf * G::stage;
#pragma unroll
    for (int i = 0; i < G::nx; ++i) {
      load_to_lds(xr, at + (i * G::threads + wave * kWave) % G::px * 16, xo[i]);
      xo[i] += T::XB;
    }
#pragma unroll
    for (int i = 0; i < G::nw; ++i) {
      load_to_lds(wr, at + G::xbytes + (i * G::threads + wave * kWave) % G::pw * 16, wo[i]);
      wo[i] += T::WB;
    }
  };
  // In a step that K ends in, once it has arrived: zeros past K.  (What
  // was read there lies in the row, or in the next one, or is the zeros that a
  // read past the buffer's range gives.)
  auto keep_step = [&](int k, int buf) {
    uint8_t* at = smem + buf * G::stage;
#pragma unroll
    for (int i = 0; i < (G::px + G::threads - 1) / G::threads; ++i) {
      const int slot = i * G::threads + tid;
      if (slot >= G::px) break;
      const int row = slot / T::XC;
      const int64_t first = (int64_t)k * T::XB + place<T::XC>(row, slot % T::XC) * 16;  // byte of the row
      u32x4* p = reinterpret_cast<u32x4*>(at + slot * 16);
      *p = keep_inputs<XF>(*p, first * 8 / elem_bits<XF>(), a.K);
    }
    if constexpr (XF == AR_BF16 || EX) {
#pragma unroll
      for (int i = 0; i < (G::pw + G::threads - 1) / G::threads; ++i) {
        const int slot = i * G::threads + tid;
        if (slot >= G::pw) break;
        const int row = slot / T::WC;
        const int64_t first = (int64_t)k * T::WB + place<T::WC>(row, slot % T::WC) * 16;
        u32x4* p = reinterpret_cast<u32x4*>(at + G::xbytes + slot * 16);
        *p = keep_weights(*p, first * 2, a.K);
      }
    }
  };
  // Scales of the run of steps that begins with step k: 16 of each row, those
  // of the tokens after those of the weights.
  const uint8_t* srow[G::ns];
#pragma unroll
  for (int i = 0; i < G::ns; ++i) {
    const int row = (i * G::threads + tid) % (G::swaves * kWave);
    srow[i] = !is_mx_format(XF) || row < BN
                  ? a.ws + r * a.ws_rank + (n0 + min(row, nlast)) * a.ws_stride
                  : a.xs + r * a.xs_rank + (m0 + min(row - BN, mlast)) * a.xs_stride;
  }
  auto load_scales = [&](int k) {
    uint8_t* at = smem + NS * G::stage + k / T::steps_scales % G::runs * G::scales;
    const int blk = k * (T::BK / 32);
#pragma unroll
    for (int i = 0; i < G::ns; ++i) {
      if (blk + 16 <= a.nb)
        load_to_lds(srow[i] + blk, at + (i * G::threads + wave * kWave) % (G::swaves * kWave) * 16);
      else                                                 // K ends in these
        *reinterpret_cast<u32x4*>(at + (i * G::threads + tid) % (G::swaves * kWave) * 16) =
            keep_scales(load_scales16<true>(srow[i], blk, a.nb), blk, a.nb);
    }
  };

  f32x4 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  constexpr bool few = TI * TJ <= 4;
  AdapterLanes<few ? TI : 1, few ? TJ : 1, (TI * TJ <= 2 && G::threads <= 256)> tiles;

  // Operands of one round (round h of a step) in registers.  8- and 4-bit
  // tokens: one matrix instruction a tile; bf16: two, group g with elements
  // 16g .. 16g + 15 of the 64.
  struct Tokens {
    u32x4 d[TJ][2];
    int s[TJ];
  };
  struct Weights {
    u32x4 d;
    int s;
  };
  auto scales_at = [&](int k, int h) {
    return smem + NS * G::stage + k / T::steps_scales % G::runs * G::scales + (k % T::steps_scales) * (T::BK / 32) +
           h * (T::BI / 32);
  };
  auto read_tokens = [&](int k, int h, int buf, Tokens& f) {
    const uint8_t* xs = smem + buf * G::stage;
    const uint8_t* sc = scales_at(k, h);
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int row = wj * WM + j * 16 + c;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        if ((XF == AR_E2M1_MX || EX) && q == 1) continue;
        const int piece = h * (T::XC / T::rounds) + (XF == AR_BF16 ? 2 * g + q : 4 * q + g);
        f.d[j][q] = *reinterpret_cast<const u32x4*>(xs + row * T::XB + place<T::XC>(row, piece) * 16);
      }
      if constexpr (is_mx_format(XF)) f.s[j] = (int)sc[(BN + row) * 16 + (EX ? g >> 1 : g)];
    }
  };
  auto read_weights = [&](int k, int h, int buf, int i, Weights& f) {
    const uint8_t* ws = smem + buf * G::stage + G::xbytes;
    const uint8_t* sc = scales_at(k, h);
    const int first = h * (T::WC / T::rounds);
    const int row = wi * WN + i * 16 + c;
    if constexpr (XF == AR_BF16 || EX) {
      const u32x2 d = *reinterpret_cast<const u32x2*>(ws + row * T::WB +
                                                      place<T::WC>(row, first + (g >> 1)) * 16 + (g & 1) * 8);
      f.d.x = d.x;
      f.d.y = d.y;
      f.s = (int)sc[row * 16 + (g >> 1)];
    } else {
      f.d = *reinterpret_cast<const u32x4*>(ws + row * T::WB + place<T::WC>(row, first + g) * 16);
      f.s = (int)sc[row * 16 + g];
    }
  };
  auto multiply_row = [&](int i, const Weights& w, const Tokens& x) {
    if constexpr (EX) {
      const float scale = __uint_as_float((uint32_t)w.s << 23);
      const bf16x8 w0 = weights_bf16(w.d.x, scale), w1 = weights_bf16(w.d.y, scale);
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        float xscale = 1.0f;
        if constexpr (is_mx_format(XF)) xscale = __uint_as_float((uint32_t)x.s[j] << 23);
        const u32x4 d = x.d[j][0];
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w0, tokens_bf16(d.x, d.y, xscale), acc[i][j], 0, 0, 0);
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w1, tokens_bf16(d.z, d.w, xscale), acc[i][j], 0, 0, 0);
      }
    } else if constexpr (XF == AR_BF16) {
      const float scale = __uint_as_float((uint32_t)w.s << 23);
      const bf16x8 w0 = weights_bf16(w.d.x, scale), w1 = weights_bf16(w.d.y, scale);
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w0, __builtin_bit_cast(bf16x8, x.d[j][0]),
                                                            acc[i][j], 0, 0, 0);
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w1, __builtin_bit_cast(bf16x8, x.d[j][1]),
                                                            acc[i][j], 0, 0, 0);
      }
    } else {
      constexpr u32x4 none = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const i32x8 b = operand(x.d[j][0], XF == AR_E2M1_MX ? none : x.d[j][1]);
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
            operand(w.d, none), b, acc[i][j], 4, XF == AR_E2M1_MX ? 4 : 0, 0, w.s, 0,
            is_mx_format(XF) ? x.s[j] : 127);
      }
    }
  };
  // one weight tile's operands ahead of the products, so that reads of shared
  // memory and matrix instructions of one wave overlap
  auto compute = [&](int k, int buf) {
#pragma unroll
    for (int q = 0; q < T::rounds / G::KG; ++q) {
      const int h = G::KG > 1 ? kg : q;
      Tokens x;
      Weights w[2];
      read_tokens(k, h, buf, x);
      read_weights(k, h, buf, 0, w[0]);
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        if (i + 1 < TI) read_weights(k, h, buf, i + 1, w[(i + 1) & 1]);
        multiply_row(i, w[i & 1], x);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  // whole steps, then maybe one that K ends in, loaded as the others are
  const int full = a.K / T::BK;
  const int steps = (a.nb * 32 + T::BK - 1) / T::BK;
#pragma unroll
  for (int k = 0; k < NS - 1; ++k) {
    if (k < steps && k % T::steps_scales == 0) load_scales(k);
    if (k < steps) load_next(k);
  }
  // (newer than those, so that a wait for those is at most longer for these)
  if constexpr (!is_same<AD, NoAdapters> && few) {
    if (!ad.delta) tiles.start(ad, a, r, m0 + wj * WM, n0 + wi * WN);
  }
  constexpr int behind = (NS - 2) * (G::nx + G::nw);
  constexpr int wait_behind = 0x0F70 | (behind & 15) | (behind >> 4) << 14;      // vmcnt alone
  int buf = 0;
  if constexpr (G::tile_waves == 8) {
    // Two waves to a SIMD, half a step apart: while one reads its operands of
    // a step from shared memory, the other one multiplies, and they change
    // places at a barrier.  Waves 0..3 read step k in phase 2k and multiply in
    // 2k + 1, waves 4..7 one phase later.  Step k + NS - 1 goes into the buffer
    // of step k - 1, which was last read in phase 2k - 1.  4096 x 8192 x 8192,
    // 8-bit tokens: 211 us against 220 with all waves in step, bf16 382 against
    // 430.  (A wave's tile as 32 x 32 x 64 instructions: 233.)
    static_assert(T::rounds == 1, "a phase is a step");
    const bool late = wave >= 4;
    auto arrived = [&](int k) {                            // this wave's loads of step k + 1
      if (NS > 2 && k + NS - 1 < steps) __builtin_amdgcn_s_waitcnt(wait_behind);
      else __builtin_amdgcn_s_waitcnt(0x0F70);
    };
    auto change = [&]() {
      __builtin_amdgcn_sched_barrier(0);
      barrier_only();
      __builtin_amdgcn_sched_barrier(0);
    };
    if (full > 0) {
      if (NS > 2 && steps > NS - 2) __builtin_amdgcn_s_waitcnt(wait_behind & ~0x0F00);
      else __builtin_amdgcn_s_waitcnt(0x0070);
      change();
      if (late) change();
    }
    for (int k = 0; k < full; ++k) {
      const int ahead = k + NS - 1;
      if (ahead < steps && ahead % T::steps_scales == 0) load_scales(ahead);
      if (ahead < steps) load_next(buf == 0 ? NS - 1 : buf - 1);
      Tokens x;
      Weights w[TI];
      read_tokens(k, 0, buf, x);
#pragma unroll
      for (int i = 0; i < TI; ++i) read_weights(k, 0, buf, i, w[i]);
      __builtin_amdgcn_s_waitcnt(0xC07F);                  // operands here, own scales written
      if (late) arrived(k);
      change();
#pragma unroll
      for (int i = 0; i < TI; ++i) multiply_row(i, w[i], x);
      if (!late) arrived(k);
      change();
      if (++buf == NS) buf = 0;
    }
    if (full > 0 && !late) change();
  } else {
    for (int k = 0; k < full; ++k) {
      // Step k has arrived when at most the NS - 2 steps after it are still on
      // their way (scales among them only make the wait longer), and this
      // wave's own scales are written.
      if (k + NS - 2 < steps) __builtin_amdgcn_s_waitcnt(wait_behind & ~0x0F00);
      else __builtin_amdgcn_s_waitcnt(0x0070);
      barrier_only();
      // into the buffer of step k - 1, which every wave has left
      const int ahead = k + NS - 1;
      if (ahead < steps && ahead % T::steps_scales == 0) load_scales(ahead);
      if (ahead < steps) load_next(buf == 0 ? NS - 1 : buf - 1);
      compute(k, buf);
      if (++buf == NS) buf = 0;
    }
  }
  if (steps > full) {
    __builtin_amdgcn_s_waitcnt(0x0070);
    barrier_only();
    keep_step(full, buf);
    __syncthreads();
    compute(full, buf);
  }
  if constexpr (G::KG > 1) {
    // the groups' sums, joined in order through shared memory by group 0
    __syncthreads();
    f32x4* part = reinterpret_cast<f32x4*>(smem) + (tw * TI * TJ) * kWave + lane;
    constexpr int group = G::tile_waves * TI * TJ * kWave;
    if (kg > 0) {
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) part[(kg - 1) * group + (i * TJ + j) * kWave] = acc[i][j];
    }
    __syncthreads();
    if (kg > 0) return;
#pragma unroll
    for (int q = 1; q < G::KG; ++q)
#pragma unroll
      for (int i = 0; i < TI; ++i)
#pragma unroll
        for (int j = 0; j < TJ; ++j) acc[i][j] += part[(q - 1) * group + (i * TJ + j) * kWave];
  }
  if constexpr (!is_same<AD, NoAdapters>) {
    if constexpr (XF == AR_E4M3_ROW) {
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const int m = min(m0 + wj * WM + j * 16 + c, a.M - 1);
        const float scale = a.K > 0 ? *reinterpret_cast<const float*>(a.xs + r * a.xs_rank + m * a.xs_stride) : 1.0f;
#pragma unroll
        for (int i = 0; i < TI; ++i) acc[i][j] *= scale;
      }
    }
    const auto sums = [&](int i, int j) -> f32x4& { return acc[i][j]; };
    if constexpr (few) {
      if (ad.delta) add_delta<TI, TJ>(ad, a, r, m0 + wj * WM, n0 + wi * WN, sums);
      else tiles.finish(ad, sums);
    } else {
      add_adapters<G>(ad, a, r, m0, n0, wj * WM, wi * WN, smem, sums);
    }
  }
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    const int m = m0 + wj * WM + j * 16 + c;
    if (m >= a.M) continue;
    float scale = 1.0f;
    if constexpr (XF == AR_E4M3_ROW && is_same<AD, NoAdapters>) {
      if (a.K > 0) scale = *reinterpret_cast<const float*>(a.xs + r * a.xs_rank + m * a.xs_stride);
    }
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int n = n0 + wi * WN + i * 16 + 4 * g;
      f32x4 v = acc[i][j];
      if constexpr (XF == AR_E4M3_ROW && is_same<AD, NoAdapters>) v *= scale;
      if (n < a.N) store_out4<YF>(a.y, r * a.y_rank + m * a.y_stride + n, n, a.N, a.vec != 0, v);
    }
  }
}

// ================================================================ host side

inline int check_linear(const ar_linear_params* p) {
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

// Up to 16 tokens.  Waves of 32 outputs read x half as often as waves of 16,
// and K is split until 2048 waves (two for each SIMD) share the stream of
// weights; where even 8 parts do not give that many, waves take 16 outputs.
// With the weights in the last cache: 16 tokens, 8-bit, 4 x 8192 x 2048: 11.1 us
// with 32 outputs, 14.3 with 16; one token, 4096 x 4096: 3.9 us with 16 outputs and
// 4 parts, 5.4 with 32 and 8; 16 tokens, 8192 x 8192: 11.3 us with 8 parts, 11.9
// with 4, 19 with 2.
constexpr int64_t kRowsWaves = 2048;

template <int XF, int YF, int NT, class AD>
static hipError_t launch_rows(const MxLinArgs& a0, const AD& ad, int nranks, hipStream_t s) {
  MxLinArgs a = a0;
  const int steps = (a.nb + 15) / 16;
  const int64_t tiles = (a.N + 16 * NT - 1) / (16 * NT);
  a.m_groups = (a.M + 15) / 16;
  auto go = [&](auto kernel, int wn, int wk) {
    a.n_groups = (int)((tiles + wn - 1) / wn);
    return launch(kernel, dim3((unsigned)((int64_t)nranks * a.n_groups * a.m_groups)),
                  dim3(kWave * wn * wk), s, a, ad);
  };
  int wk = 1;
  while (wk < 8 && 2 * wk <= steps && tiles * nranks * wk < kRowsWaves) wk *= 2;
  switch (wk) {
    case 1: return go(k_mx_linear_rows<XF, YF, NT, 4, 1, AD>, 4, 1);
    case 2: return go(k_mx_linear_rows<XF, YF, NT, 2, 2, AD>, 2, 2);
    case 4: return go(k_mx_linear_rows<XF, YF, NT, 1, 4, AD>, 1, 4);
    default: return go(k_mx_linear_rows<XF, YF, NT, 1, 8, AD>, 1, 8);
  }
}

template <class G, class AD>
static hipError_t launch_tiles(const MxLinArgs& a0, const AD& ad, int nranks, hipStream_t s) {
  MxLinArgs a = a0;
  a.n_groups = (a.N + G::BN - 1) / G::BN;
  a.m_groups = (a.M + G::BM - 1) / G::BM;
  return launch(k_mx_linear_tiles<G, AD>, dim3((unsigned)((int64_t)nranks * a.n_groups * a.m_groups)),
                dim3(G::threads), s, a, ad);
}

// Which kernel.  Tiles for more than 16 tokens, and for 9 to 16 of 8 or 4 bits
// where the smallest tiles are more than the CUs (256).  Among tiles the largest
// that gives every CU one and is at least half full of tokens; tiles of 32
// tokens with K shared by 4 groups of waves where even those are not more than
// the CUs.  Measured both ways, 8-bit tokens, weights in the last cache but for the
// 131072 outputs (290 MB), in us:
//   32 x 64 tiles against waves on rows: 4 x 16 x 8192 x 2048 9.7 and 11.2, with
//   9 tokens 9.7 and 10.0, 8 9.5 and 9.8, 4 9.3 and 8.8; 16 x 8192 x 8192 (128
//   tiles) 15.9 and 11.5; bf16, 4 x 16 x 8192 x 2048 14.8 and 14.9, 12 14.8 and
//   13.6;
//   256 x 256 against 128 x 128 or less: 4096 to 131072, 16 tokens 107 and 69, 64
//   110 and 95, 128 114 and 91;
//   256 x 256 against 128 x 128 tiles: 2048 x 8192 x 8192 108 and 131, 1024 x
//   8192 x 8192 102 (128 tiles) and 66;
//   128 x 128 against 64 x 64: 4 x 128 x 8192 x 2048 17.5 and 19.4, 256 x 4096 x
//   4096 24.3 (64 tiles) and 11.7;
//   64 x 64 (2 groups) against 32 x 64 (4): 256 x 4096 x 4096 11.7 and 19.9, 64 x
//   4096 x 4096 11.0 (64 tiles) and 10.0, 32 x 8192 x 8192 18.5 (128 tiles) and
//   16.3;
//   32 x 64 (1 group) against 64 x 64 (2): 8 x 32 x 4096 x 512 (bf16) 6.0 and
//   7.9, 4 x 32 x 8192 x 2048 9.9 and 10.5.
// The tile kernels' offsets inside a tile are 31 bits: rows further apart take
// the other kernel at any number of tokens.
inline int64_t linear_tiles(const MxLinArgs& a, int nranks, int bm, int bn) {
  return (int64_t)((a.N + bn - 1) / bn) * ((a.M + bm - 1) / bm) * nranks;
}
// Tiles of 128 x 128 or 256 x 256.
inline bool large_tiles(const MxLinArgs& a, int nranks) {
  return a.x_stride < (1 << 23) && a.w_stride < (1 << 23) &&
         ((a.M > 128 && linear_tiles(a, nranks, 256, 256) >= 256) ||
          (a.M > 64 && linear_tiles(a, nranks, 128, 128) >= 256));
}

template <int XF, int YF, class AD>
static hipError_t launch_linear(const MxLinArgs& a, const AD& ad, int nranks, hipStream_t s) {
  auto tiles = [&](int bm, int bn) { return linear_tiles(a, nranks, bm, bn); };
  const bool many = a.M > 16 || (XF != AR_BF16 && a.M > 8 && tiles(32, 64) > 256);
  if (many && a.x_stride < (1 << 23) && a.w_stride < (1 << 23)) {
    constexpr bool EX = exact8<XF, YF, AD>();
    constexpr int K1 = XF == AR_BF16 ? 64 : 128;           // of a step with all its waves
    constexpr int KI = EX ? 64 : K1;                       // of a round for a group of them
    constexpr bool x4 = XF == AR_E2M1_MX;                  // small enough for steps of 256
    if constexpr (!EX)                                     // whose steps are two rounds
      if (a.M > 128 && tiles(256, 256) >= 256)
        return launch_tiles<Tile<XF, YF, EX, K1, 256, 256, 64, 128, 3>>(a, ad, nranks, s);
    if (a.M > 64 && tiles(128, 128) >= 256)
      return launch_tiles<Tile<XF, YF, EX, x4 ? 256 : K1, 128, 128, 64, 64, x4 ? 2 : 3>>(a, ad, nranks, s);
    if (tiles(32, 64) <= 256) return launch_tiles<Tile<XF, YF, EX, 4 * KI, 32, 64, 32, 16, 3, 4>>(a, ad, nranks, s);
    if (a.M <= 32) return launch_tiles<Tile<XF, YF, EX, K1, 32, 64, 32, 16, 5>>(a, ad, nranks, s);
    return launch_tiles<Tile<XF, YF, EX, 2 * KI, 64, 64, 32, 32, 3, 2>>(a, ad, nranks, s);
  }
  const int64_t steps = (a.nb + 15) / 16, wide = (int64_t)((a.N + 31) / 32) * nranks;
  if (wide * (steps < 8 ? steps : 8) >= kRowsWaves) return launch_rows<XF, YF, 2>(a, ad, nranks, s);
  return launch_rows<XF, YF, 1>(a, ad, nranks, s);
}

template <int XF, class AD>
static hipError_t launch_linear_y(const MxLinArgs& a, const AD& ad, int yf, int nranks, hipStream_t s) {
  return yf == AR_F32 ? launch_linear<XF, AR_F32>(a, ad, nranks, s)
                      : launch_linear<XF, AR_BF16>(a, ad, nranks, s);
}

template <class AD>
static hipError_t launch_linear_x(const MxLinArgs& a, const AD& ad, int xf, int yf, int nranks, hipStream_t s) {
  switch (xf) {
    case AR_BF16: return launch_linear_y<AR_BF16>(a, ad, yf, nranks, s);
    case AR_E4M3_ROW: return launch_linear_y<AR_E4M3_ROW>(a, ad, yf, nranks, s);
    case AR_E4M3_MX: return launch_linear_y<AR_E4M3_MX>(a, ad, yf, nranks, s);
    default: return launch_linear_y<AR_E2M1_MX>(a, ad, yf, nranks, s);
  }
}

// Output the size of more than one launch (no kernel here has more than 512
// threads for 16 x 16 outputs, unless its workgroups are few) goes by ranks, then by
// halves of the longer side, in whole tiles.
template <class AD>
static hipError_t launch_pieces(const MxLinArgs& a, const AD& ad, int xf, int yf, int nranks, hipStream_t s) {
  const int64_t rows = ceil_div64(a.M, 16), outs = ceil_div64(a.N, 16);
  if (rows * outs * nranks <= most_blocks(512)) return launch_linear_x(a, ad, xf, yf, nranks, s);
  const int64_t size = yf == AR_F32 ? 4 : 2;
  auto from = [&](int r, int m, int n) {
    MxLinArgs b = a;
    b.x += r * a.x_rank + m * a.x_stride;
    if (b.xs) b.xs += r * a.xs_rank + m * a.xs_stride;
    b.w += r * a.w_rank + n * a.w_stride;
    b.ws += r * a.ws_rank + n * a.ws_stride;
    b.y = static_cast<uint8_t*>(a.y) + (r * a.y_rank + m * a.y_stride + n) * size;
    b.M -= m;
    b.N -= n;
    return b;
  };
  auto adapters = [&](int r, int m, int n) {
    AD b = ad;
    if constexpr (!is_same<AD, NoAdapters>) {
      b.index += m;
      b.t += r * ad.t_rank + m * ad.t_stride;
      if (b.delta) b.delta += r * ad.delta_rank + m * ad.delta_stride + n;
      b.b += r * ad.b_rank + n * ad.b_stride;
    }
    return b;
  };
  hipError_t e = hipSuccess;
  if (nranks > 1) {
    for (int r = 0; r < nranks && e == hipSuccess; ++r) e = launch_pieces(from(r, 0, 0), adapters(r, 0, 0), xf, yf, 1, s);
    return e;
  }
  const int m = rows >= outs ? (int)ceil_div64(a.M, 512) * 256 : 0;
  const int n = rows >= outs ? 0 : (int)ceil_div64(a.N, 512) * 256;
  MxLinArgs first = a;
  if (m) first.M = m;
  else first.N = n;
  e = launch_pieces(first, ad, xf, yf, 1, s);
  return e == hipSuccess ? launch_pieces(from(0, m, n), adapters(0, m, n), xf, yf, 1, s) : e;
}

inline MxLinArgs linear_args(const ar_linear_params* p) {
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
  return a;
}

}  // namespace ar
