// ar_adapters.hip -- the linear shards on microscaled 4-bit weights with
// low-rank adapters of many requests beside them (gfx950):
//     y_r[m][n] = sum over k of x_r[m][k] w_r[n][k] + sum over j of t_r[m][j] b[n][j],
//     t_r[m][j] = scale * sum over k of x_r[m][k] a[j][k],
// a, b and scale those of token m's adapter.  Two launches: one for t, which is
// small, and the linear layer's own, which adds the second product to its sums
// before their one rounding, so that neither y nor what is added to it makes a
// way through memory.
#include "ar_mxlinear.h"

namespace ar {

// Strides in bytes.
struct TokenArgs {
  const uint8_t* x;
  int64_t x_stride, x_rank;
  const uint8_t* xs;
  int64_t xs_stride, xs_rank;
  const uint8_t* a;
  int64_t a_stride, a_adapter, a_rank;
  const int32_t* index;
  const float* scale;
  uint8_t* t;
  int64_t t_stride, t_rank;
  int32_t M, K, nb;
  int32_t count, rank;
  int32_t slots, r_groups, m_tiles;
};

// A lane's operands of 128 elements of K: group g has 32 of them, from 32g on,
// 8 in each of 4 matrix instructions, so that x's and a's rows are read 16 bytes
// at a time in every format.
template <int XF>
constexpr int row_pieces() { return elem_bits<XF>() / 4; }
template <int XF, int NR>
struct TokenStep {
  u32x4 x[row_pieces<XF>()];
  uint32_t s;
  u32x4 a[NR][4];
};

template <int XF>
__device__ __forceinline__ u32x4 token_operand(const u32x4 (&x)[row_pieces<XF>()], uint32_t scale, int u) {
  if constexpr (XF == AR_BF16) {
    return x[u];
  } else if constexpr (XF == AR_E2M1_MX) {
    return __builtin_bit_cast(u32x4, weights_bf16(x[0][u], __uint_as_float(scale << 23)));
  } else {
    const float s = XF == AR_E4M3_MX ? __uint_as_float(scale << 23) : 1.0f;
    const uint32_t lo = x[u >> 1][2 * (u & 1)], hi = x[u >> 1][2 * (u & 1) + 1];
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, s, true)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, s, true))};
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

constexpr int kTokenWaves = 8;

// t of 16 tokens in 16 * NR of an adapter's dimensions.  Bound by the way of a
// and x to the CU: the waves share K, a step of 128 each in turn, the next one on
// its way while one is multiplied, and join their sums in shared memory.  The
// tokens' adapters go one after the other, `slots` workgroups taking turns.
template <int XF, int NR, int P>
__global__ __launch_bounds__(kWave * kTokenWaves) void k_adapter_tokens(TokenArgs s) {
  __shared__ f32x4 part[kTokenWaves * NR * kWave];
  const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int b = blockIdx.x;
  const int slot = b % s.slots;
  b /= s.slots;
  const int j0 = b % s.r_groups * 16 * NR;
  b /= s.r_groups;
  const int m = b % s.m_tiles * 16 + c, r = b / s.m_tiles;
  const int mine = m < s.M ? s.index[m] : -1;
  const int row = min(m, s.M - 1);
  const uint8_t* x = s.x + r * s.x_rank + row * s.x_stride;
  const uint8_t* xs = s.xs + r * s.xs_rank + row * s.xs_stride;
  uint32_t left = (uint32_t)__ballot((uint32_t)mine < (uint32_t)s.count) & 0xFFFFu;
  for (int turn = 0; left != 0; ++turn) {
    const int which = __builtin_amdgcn_readlane(mine, __builtin_ctz(left));
    const bool take = mine == which;
    left &= ~(uint32_t)__ballot(take);
    if (turn % s.slots != slot) continue;
    const uint8_t* a[NR];
    f32x4 acc[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      a[i] = s.a + r * s.a_rank + which * s.a_adapter + min(j0 + 16 * i + c, s.rank - 1) * s.a_stride;
      acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    auto load = [&](int st, TokenStep<XF, NR>& f) {
      const int at = st * 128 + 32 * g;
      constexpr int per = 128 / elem_bits<XF>();
      const bool whole = st * 128 + 128 <= s.K;
#pragma unroll
      for (int q = 0; q < row_pieces<XF>(); ++q) {
        f.x[q] = u32x4{0u, 0u, 0u, 0u};
        if (whole || at + q * per < s.K) f.x[q] = ldg16(x + (int64_t)(at + q * per) * elem_bits<XF>() / 8);
      }
      f.s = 127;
      if constexpr (is_mx_format(XF)) {
        if (whole || at < s.K) f.s = xs[at / 32];
      }
#pragma unroll
      for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          f.a[i][u] = u32x4{0u, 0u, 0u, 0u};
          if (whole || at + 8 * u < s.K) f.a[i][u] = ldg16(a[i] + (int64_t)(at + 8 * u) * 2);
        }
    };
    auto multiply = [&](int st, TokenStep<XF, NR>& f) {
      const int at = st * 128 + 32 * g;
      if (st * 128 + 128 > s.K) {                          // K ends in this one
        constexpr int per = 128 / elem_bits<XF>();
#pragma unroll
        for (int q = 0; q < row_pieces<XF>(); ++q) f.x[q] = keep_inputs<XF>(f.x[q], at + q * per, s.K);
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
          for (int u = 0; u < 4; ++u) f.a[i][u] = keep_inputs<AR_BF16>(f.a[i][u], at + 8 * u, s.K);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bf16x8 v = __builtin_bit_cast(bf16x8, token_operand<XF>(f.x, f.s, u));
#pragma unroll
        for (int i = 0; i < NR; ++i)
          acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f.a[i][u]), v, acc[i], 0, 0, 0);
      }
    };
    const int steps = (s.K + 127) / 128;
    if (wave < steps) {
      TokenStep<XF, NR> cur;
      int st = wave;
      load(st, cur);
      for (; st + kTokenWaves < steps; st += kTokenWaves) {
        TokenStep<XF, NR> next;
        load(st + kTokenWaves, next);
        multiply(st, cur);
        cur = next;
      }
      multiply(st, cur);
    }
#pragma unroll
    for (int i = 0; i < NR; ++i) part[(wave * NR + i) * kWave + lane] = acc[i];
    __syncthreads();
    if (wave < NR && take) {
      f32x4 v = part[wave * kWave + lane];
#pragma unroll
      for (int w = 1; w < kTokenWaves; ++w) v += part[(w * NR + wave) * kWave + lane];
      if (s.scale) v *= s.scale[which];
      if constexpr (XF == AR_E4M3_ROW) v *= *reinterpret_cast<const float*>(xs);
      const int j = j0 + 16 * wave + 4 * g;
      uint32_t p[4][P];
#pragma unroll
      for (int e = 0; e < 4; ++e) bf16_parts<P>(j + e < s.rank ? v[e] : 0.0f, p[e]);
      uint8_t* t = s.t + r * s.t_rank + m * s.t_stride + j / 8 * (16 * P) + j % 8 * 2;
      if (j0 + 16 * wave < s.rank) {
#pragma unroll
        for (int q = 0; q < P; ++q)
          *reinterpret_cast<u32x2*>(t + 16 * q) = u32x2{pack2(p[0][q], p[1][q]), pack2(p[2][q], p[3][q])};
      }
    }
    __syncthreads();
  }
}

// ================================================================ host side

static int check_adapters(const ar_linear_params* p, const ar_adapter_params* q) {
  if (!p || !q) return AR_EINVAL;
  if (q->reserved != 0 || q->adapters < 0 || q->rank < 0) return AR_EINVAL;
  if (q->rank > AR_ADAPTER_MAX_RANK) return AR_ESIZE;
  return check_linear(p);
}

// Whether an adapter can add anything at all.
static bool adapters_count(const ar_linear_params* p, const ar_adapter_params* q) {
  return q->adapters > 0 && q->rank > 0 && p->rows > 0 && p->outputs > 0 && p->inputs > 0;
}

static int check_adapter_rows(const ar_linear_params* p, const ar_adapter_params* q) {
  if (!q->index) return AR_EINVAL;
  if (!aligned(q->index, 4) || !aligned(q->scale, 4)) return AR_EALIGN;
  int rc = check_format_rows(AR_BF16, q->a, q->a_stride, q->rank, p->inputs);
  if (rc) return rc;
  rc = check_format_rows(AR_BF16, q->b, q->b_stride, p->outputs, q->rank);
  if (rc) return rc;
  const int64_t most = int64_t(1) << 40;
  if (q->a_adapter_stride < 0 || q->a_rank_stride < 0 || q->b_adapter_stride < 0 || q->b_rank_stride < 0)
    return AR_EINVAL;
  if (q->a_adapter_stride >= most || q->a_rank_stride >= most || q->b_adapter_stride >= most ||
      q->b_rank_stride >= most)
    return AR_ESIZE;
  if (q->a_adapter_stride % 8 || q->b_adapter_stride % 8) return AR_EALIGN;
  if (p->nranks > 1 && (q->a_rank_stride % 8 || q->b_rank_stride % 8)) return AR_EALIGN;
  return AR_OK;
}

// Ranks that share tokens and a also share t.
static int t_ranks(const ar_linear_params* p, const ar_adapter_params* q) {
  return p->x_rank_stride == 0 && (p->x_format == AR_BF16 || p->x_scale_rank_stride == 0) && q->a_rank_stride == 0
             ? 1
             : p->nranks;
}

static int64_t t_row_bytes(const ar_linear_params* p, const ar_adapter_params* q) {
  return ceil_div64(q->rank, 16) * 16 * 2 * t_parts(p->y_format);
}

static int64_t adapter_work(const ar_linear_params* p, const ar_adapter_params* q) {
  if (!adapters_count(p, q)) return 0;
  return (t_ranks(p, q) * p->rows * t_row_bytes(p, q) + 255) / 256 * 256;
}

template <int XF, int NR, int P>
static hipError_t launch_tokens(const TokenArgs& a0, int ranks, hipStream_t s) {
  TokenArgs a = a0;
  a.r_groups = (a.rank + 16 * NR - 1) / (16 * NR);
  // as many workgroups at once for the adapters of 16 tokens as fill the chip
  const int64_t groups = ceil_div64(a0.M, 16) * ranks * a.r_groups;
  a.slots = 1;
  while (a.slots < 16 && a.slots < a.M && a.slots < a.count && groups * a.slots < 512) a.slots *= 2;
  const int64_t most = most_blocks(kWave * kTokenWaves) / ((int64_t)ranks * a.r_groups * a.slots) * 16;
  for (int64_t m = 0; m < a0.M; m += most) {
    a.M = (int32_t)(a0.M - m < most ? a0.M - m : most);
    a.m_tiles = (a.M + 15) / 16;
    a.x = a0.x + m * a0.x_stride;
    if (a0.xs) a.xs = a0.xs + m * a0.xs_stride;
    a.index = a0.index + m;
    a.t = a0.t + m * a0.t_stride;
    const int64_t blocks = (int64_t)ranks * a.m_tiles * a.r_groups * a.slots;
    const hipError_t e = launch(k_adapter_tokens<XF, NR, P>, dim3((unsigned)blocks), dim3(kWave * kTokenWaves), s, a);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int XF, int P>
static hipError_t launch_tokens_rank(const TokenArgs& a, int ranks, hipStream_t s) {
  if (a.rank <= 16 || a.M <= 16) return launch_tokens<XF, 1, P>(a, ranks, s);
  if (a.rank <= 32) return launch_tokens<XF, 2, P>(a, ranks, s);
  return launch_tokens<XF, 4, P>(a, ranks, s);
}

template <int P>
static hipError_t launch_tokens_x(const TokenArgs& a, int xf, int ranks, hipStream_t s) {
  switch (xf) {
    case AR_BF16: return launch_tokens_rank<AR_BF16, P>(a, ranks, s);
    case AR_E4M3_ROW: return launch_tokens_rank<AR_E4M3_ROW, P>(a, ranks, s);
    case AR_E4M3_MX: return launch_tokens_rank<AR_E4M3_MX, P>(a, ranks, s);
    default: return launch_tokens_rank<AR_E2M1_MX, P>(a, ranks, s);
  }
}

}  // namespace ar

using namespace ar;

extern "C" {

int64_t ar_adapter_work_bytes(const ar_linear_params* p, const ar_adapter_params* q) {
  const int rc = check_adapters(p, q);
  return rc ? rc : adapter_work(p, q);
}

int ar_mx4_linear_adapters(const ar_linear_params* p, const ar_adapter_params* q, void* work, int64_t work_bytes,
                           void* stream) {
  int rc = check_adapters(p, q);
  if (rc) return rc;
  if (!adapters_count(p, q)) return ar_mx4_linear(p, stream);
  rc = check_adapter_rows(p, q);
  if (rc) return rc;
  if (ceil_div64(p->outputs, 16) * ceil_div64(p->rows, 16) * p->nranks > INT32_MAX) return AR_ESIZE;
  if (!work) return AR_EINVAL;
  if (!aligned(work, 256)) return AR_EALIGN;
  if (work_bytes < adapter_work(p, q)) return AR_ESIZE;
  const MxLinArgs a = linear_args(p);
  const int ranks = t_ranks(p, q);
  TokenArgs t{};
  t.x = a.x;
  t.x_stride = a.x_stride;
  t.x_rank = a.x_rank;
  t.xs = a.xs;
  t.xs_stride = a.xs_stride;
  t.xs_rank = a.xs_rank;
  t.a = static_cast<const uint8_t*>(q->a);
  t.a_stride = q->a_stride * 2;
  t.a_adapter = q->a_adapter_stride * 2;
  t.a_rank = q->a_rank_stride * 2;
  t.index = q->index;
  t.scale = q->scale;
  t.t = static_cast<uint8_t*>(work);
  t.t_stride = t_row_bytes(p, q);
  t.t_rank = ranks > 1 ? p->rows * t.t_stride : 0;
  t.M = a.M;
  t.K = a.K;
  t.nb = a.nb;
  t.count = q->adapters;
  t.rank = q->rank;
  Adapters ad{};
  ad.index = q->index;
  ad.t = t.t;
  ad.t_stride = t.t_stride;
  ad.t_rank = t.t_rank;
  ad.b = static_cast<const uint8_t*>(q->b);
  ad.b_stride = q->b_stride * 2;
  ad.b_adapter = q->b_adapter_stride * 2;
  ad.b_rank = q->b_rank_stride * 2;
  ad.count = q->adapters;
  ad.rank = q->rank;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const hipError_t e = t_parts(p->y_format) == 2 ? launch_tokens_x<2>(t, p->x_format, ranks, s)
                                                 : launch_tokens_x<3>(t, p->x_format, ranks, s);
  if (e != hipSuccess) return map_hip(e);
  return map_hip(launch_pieces(a, ad, p->x_format, p->y_format, p->nranks, s));
}

}  // extern "C"
