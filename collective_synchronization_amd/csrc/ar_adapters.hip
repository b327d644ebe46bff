// ar_adapters.hip -- the linear shards on microscaled 4-bit weights with
// low-rank adapters of many requests beside them (gfx950):
//     y_r[m][n] = sum over k of x_r[m][k] w_r[n][k] + sum over j of t_r[m][j] b[n][j],
//     t_r[m][j] = scale * sum over k of x_r[m][k] a[j][k],
// a, b and scale those of token m's adapter.  t is small and has a launch of its
// own: k_adapter_few_tokens reads every token's rows of a for it alone, and
// k_adapter_tokens (with k_adapter_sum) those of an adapter for all its tokens.  The
// second product joins the layer's sums before their one rounding, so that y does
// not make a way through memory for it: in the largest tiles through shared memory
// (add_adapters), for 16 tokens and dimensions in the layer's waves (AdapterLanes),
// else made ready in binary32 first (k_adapter_delta).
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
  int64_t t_stride, t_part, t_rank;  // part p of rank r's row m: t + p * t_part + r * t_rank + m * t_stride
  int32_t M, K, nb;
  int32_t count, rank;
  int32_t splits, slots, r_groups, m_groups;
};

// A lane's part of 128 elements of K: group g has 32 of them, from 32g on, 8 in
// each of 4 matrix instructions, so that rows of x are read 16 bytes at a time in
// every format.
template <int XF>
constexpr int row_pieces() { return elem_bits<XF>() / 4; }

template <int XF>
__device__ __forceinline__ u32x4 token_operand(const u32x4 (&x)[row_pieces<XF>()], uint32_t scale, int u) {
  if constexpr (XF == AR_BF16) {
    return x[u];
  } else if constexpr (XF == AR_E2M1_MX) {
    return __builtin_bit_cast(u32x4, weights_bf16(x[0][u], __uint_as_float(scale << 23)));
  } else {
    const float s = XF == AR_E4M3_MX ? __uint_as_float(scale << 23) : 1.0f;
    return __builtin_bit_cast(u32x4, tokens_bf16(x[u >> 1][2 * (u & 1)], x[u >> 1][2 * (u & 1) + 1], s));
  }
}

// 8 elements of a token's row from `at` on, as it lies in memory, and their values.
template <int XF>
struct Token8 {
  u32x4 d;
  uint32_t s;
};
template <int XF>
__device__ __forceinline__ Token8<XF> load_token8(const uint8_t* x, const uint8_t* xs, int at) {
  Token8<XF> t{};
  const uint8_t* p = x + (int64_t)at * elem_bits<XF>() / 8;
  if constexpr (XF == AR_BF16) {
    t.d = ldg16(p);
  } else if constexpr (XF == AR_E2M1_MX) {
    t.d.x = *reinterpret_cast<const uint32_t*>(p);
  } else {
    const u32x2 v = *reinterpret_cast<const u32x2*>(p);
    t.d.x = v.x;
    t.d.y = v.y;
  }
  if constexpr (is_mx_format(XF)) t.s = xs[at / 32];
  return t;
}
template <int XF>
__device__ __forceinline__ void token8(const Token8<XF>& t, float (&v)[8]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const float s = XF == AR_E4M3_ROW ? 1.0f : __uint_as_float(t.s << 23);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    f32x2 p;
    if constexpr (XF == AR_BF16) {
      p = f32x2{bf_lo(t.d[k]), bf_hi(t.d[k])};
    } else if constexpr (XF == AR_E2M1_MX) {
      if (k == 0) p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(t.d.x, s, 0);
      if (k == 1) p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(t.d.x, s, 1);
      if (k == 2) p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(t.d.x, s, 2);
      if (k == 3) p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(t.d.x, s, 3);
    } else {
      p = k % 2 == 0 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(t.d[k / 2], s, false)
                     : __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(t.d[k / 2], s, true);
    }
    v[2 * k] = p.x;
    v[2 * k + 1] = p.y;
  }
}

// t of one token, 4 dimensions a wave, for few tokens: each has rows of a to
// itself, so they are read as they are multiplied, in binary32, 512 elements of K
// at a time.  WK waves share K; without, a workgroup has 16 dimensions.  Bound by the
// loads' latency: index, then x and a, then the join (1 to 2 us beside the launch for
// 4 ranks of 16 tokens of 2048; in matrix instructions for 16 tokens at a time, with
// 15 of them empty where each has its own adapter, 6).  Up to kFewTokens, and as
// long as a is read no more than 64 MB in all.
constexpr int kFewTokens = 32;
constexpr int64_t kFewProducts = int64_t(1) << 25;
template <int XF, int WK>
__global__ __launch_bounds__(kBlock) void k_adapter_few_tokens(TokenArgs s) {
  static_assert(WK == 1 || WK == kWavesPerBlock, "");
  __shared__ f32x4 part[kWavesPerBlock];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int per = WK == 1 ? 16 : 4;                    // dimensions of a workgroup
  int b = blockIdx.x;
  const int j0 = b % s.r_groups * per + (WK == 1 ? 4 * wave : 0);
  b /= s.r_groups;
  const int m = b % s.M, r = b / s.M;
  const int which = s.index[m];
  if ((uint32_t)which >= (uint32_t)s.count) return;
  const uint8_t* x = s.x + r * s.x_rank + m * s.x_stride;
  const uint8_t* xs = s.xs + r * s.xs_rank + m * s.xs_stride;
  const uint8_t* a[4];
  f32x4 sum = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    a[e] = s.a + r * s.a_rank + which * s.a_adapter + min(j0 + e, s.rank - 1) * s.a_stride;
  const float scale = s.scale ? s.scale[which] : 1.0f;
  for (int k0 = (WK == 1 ? 0 : wave) * 512; k0 < s.K; k0 += WK * 512) {
    const int at = k0 + lane * 8;
    if (at >= s.K) continue;
    const Token8<XF> t = load_token8<XF>(x, xs, at);
    u32x4 w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = ldg16(a[e] + (int64_t)at * 2);
    float v[8];
    token8<XF>(t, v);
    const bool cut = at + 8 > s.K;                         // K ends in these
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (cut && at + u >= s.K) v[u] = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (cut) w[e] = keep_inputs<AR_BF16>(w[e], at, s.K);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        sum[e] = __builtin_fmaf(v[2 * u], bf_lo(w[e][u]), sum[e]);
        sum[e] = __builtin_fmaf(v[2 * u + 1], bf_hi(w[e][u]), sum[e]);
      }
    }
  }
#pragma unroll
  for (int d = 32; d > 0; d /= 2)
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[e] += __shfl_xor(sum[e], d);
  if constexpr (WK > 1) {
    if (lane == 0) part[wave] = sum;
    __syncthreads();
    if (wave > 0) return;
    sum = part[0];
#pragma unroll
    for (int w = 1; w < WK; ++w) sum += part[w];
  }
  if (lane > 0 || j0 >= (s.rank + 15) / 16 * 16) return;
  sum *= scale;
  if constexpr (XF == AR_E4M3_ROW) sum *= *reinterpret_cast<const float*>(xs);
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[e] = j0 + e < s.rank ? sum[e] : 0.0f;
  *reinterpret_cast<f32x4*>(s.t + r * s.t_rank + m * s.t_stride + j0 * 4) = sum;
}

constexpr int kTokenGroup = 256;
constexpr int kTokenParts = 16;                            // most workgroups that share K
constexpr int kTurn = 64;                                  // tokens of a workgroup's turn

// Parts of t for up to 64 tokens of one adapter, in 16 * NR of its dimensions, over
// a share of K.  Bound by the way of a and x to the CUs.  A group is 256 tokens:
// its workgroups find the group's adapters, each with the list of its tokens, and
// take turns with them, so that tokens in any order read an adapter's rows once
// for all of them.  `splits` workgroups share K for each; their sums are joined by
// k_adapter_sum.  A wave has 16 of the tokens.  Steps of 128 elements pass
// through shared memory, loaded straight into it, the ones after a step on their
// way while it is multiplied; rows lie there with their 16-byte pieces permuted
// so that lanes which read at once meet different banks.  (Groups go round the
// XCDs, so that each reads all of K: with a share of K each, rows 8 and 16 KiB
// apart meet a quarter of an L2's channels.)
template <int XF, int NR>
struct TokenTile {
  static constexpr int XB = 16 * elem_bits<XF>(), XC = XB / 16, AC = 16;   // bytes and pieces of a row's step
  static constexpr int nx = kTurn * XC / kBlock, na = NR * 16 * AC / kBlock;
  static constexpr int scales = is_mx_format(XF) ? kWavesPerBlock * 256 : 0;
  static constexpr int stage = kTurn * XB + NR * 16 * AC * 16 + scales;
  static constexpr int NS = 3 * stage <= 80 * 1024 ? 3 : 2;   // two workgroups to a CU, or more
  static constexpr int loads = nx + na + (is_mx_format(XF) ? 1 : 0);
  static_assert(kWavesPerBlock * 16 == kTurn, "a wave has 16 tokens");
};
template <int XF, int NR>
__global__ __launch_bounds__(kBlock) void k_adapter_tokens(TokenArgs s) {
  using T = TokenTile<XF, NR>;
  constexpr int NS = T::NS;
  __shared__ __align__(256) uint8_t smem[NS * T::stage];
  __shared__ int list[kTokenGroup];
  const int tid = threadIdx.x, lane = tid & 63, c = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int b = blockIdx.x;
  const int m0 = b % s.m_groups * kTokenGroup;
  b /= s.m_groups;
  const int slot = b % s.slots;
  b /= s.slots;
  const int split = b % s.splits;
  b /= s.splits;
  const int j0 = b % s.r_groups * 16 * NR, r = b / s.r_groups;
  const int steps = (s.K + 127) / 128, each = (steps + s.splits - 1) / s.splits;
  const int st0 = split * each, n = max(min(steps, st0 + each) - st0, 0);
  int mine[4];
  uint64_t left[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int m = m0 + 64 * k + lane;
    mine[k] = m < s.M ? s.index[m] : -1;
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) left[k] = __ballot((uint32_t)mine[k] < (uint32_t)s.count);
  int turn = 0;
  while ((left[0] | left[1] | left[2] | left[3]) != 0) {
    int which = 0;
    bool found = false;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (!found && left[k] != 0) {
        which = __builtin_amdgcn_readlane(mine[k], __builtin_ctzll(left[k]));
        found = true;
      }
    int tokens = 0, before = 0;
    uint64_t has[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      has[k] = __ballot(mine[k] == which) & left[k];
      left[k] &= ~has[k];
      tokens += __builtin_popcountll(has[k]);
    }
    const int first = turn;
    turn += (tokens + kTurn - 1) / kTurn;
    // this workgroup's turns among them
    if (first + (slot - first % s.slots + s.slots) % s.slots >= turn) continue;
    __syncthreads();                                       // the list was read
    if (wave == 0) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint64_t below = has[k] & ((uint64_t(1) << lane) - 1);
        if (has[k] >> lane & 1) list[before + __builtin_popcountll(below)] = 64 * k + lane;
        before += __builtin_popcountll(has[k]);
      }
    }
    __syncthreads();
    const float scale = s.scale ? s.scale[which] : 1.0f;
    for (int t0 = 0, it = first; t0 < tokens; t0 += kTurn, ++it) {
      if (it % s.slots != slot) continue;
      // this thread's pieces: rows, and bytes in a step
      const uint8_t *xp[T::nx], *ap[T::na];
      int xo[T::nx], ao[T::na];
#pragma unroll
      for (int i = 0; i < T::nx; ++i) {
        const int at = i * kBlock + tid, row = at / T::XC;
        xp[i] = s.x + r * s.x_rank + (m0 + list[min(t0 + row, tokens - 1)]) * s.x_stride;
        xo[i] = place<T::XC>(row, at % T::XC) * 16;
      }
#pragma unroll
      for (int i = 0; i < T::na; ++i) {
        const int at = i * kBlock + tid, row = at / T::AC;
        ap[i] = s.a + r * s.a_rank + which * s.a_adapter + min(j0 + row, s.rank - 1) * s.a_stride;
        ao[i] = place<T::AC>(row, at % T::AC) * 16;
      }
      const int m = m0 + list[min(t0 + 16 * wave + c, tokens - 1)];
      const uint8_t* xs = s.xs + r * s.xs_rank + m * s.xs_stride;
      // rows' last pieces, which are read again in the place of those past them
      // (offsets in a row pass 31 bits)
      const uint32_t x_last = (uint32_t)(((int64_t)s.K * elem_bits<XF>() + 127) / 128 * 16 - 16);
      const uint32_t a_last = (uint32_t)(((int64_t)s.K + 7) / 8 * 16 - 16);
      auto load = [&](int k, int buf) {
        uint8_t* at = smem + buf * T::stage;
        const int st = st0 + k;
#pragma unroll
        for (int i = 0; i < T::nx; ++i)
          load_to_lds(xp[i] + min((uint32_t)st * T::XB + xo[i], x_last), at + (i * kBlock + wave * kWave) * 16);
#pragma unroll
        for (int i = 0; i < T::na; ++i)
          load_to_lds(ap[i] + min((uint32_t)st * 256 + ao[i], a_last), at + kTurn * T::XB + (i * kBlock + wave * kWave) * 16);
        if constexpr (is_mx_format(XF)) {                  // 4 scales of each of the wave's tokens
          typedef __attribute__((address_space(3))) void lds_void;
          typedef const __attribute__((address_space(1))) void global_void;
          uint8_t* to = at + kTurn * T::XB + NR * 16 * T::AC * 16 + wave * 256;
          __builtin_amdgcn_global_load_lds((global_void*)(xs + min(4 * st, (s.nb - 1) / 4 * 4)), (lds_void*)to, 4, 0, 0);
        }
      };
      f32x4 acc[NR];
#pragma unroll
      for (int i = 0; i < NR; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      const bool idle = t0 + 16 * wave >= tokens;
      auto compute = [&](int k, int buf) {
        const uint8_t* at = smem + buf * T::stage;
        const int st = st0 + k, first = st * 128 + 32 * g, row = 16 * wave + c;
        const bool cut = st * 128 + 128 > s.K;             // K ends in this step: zeros behind it
        u32x4 x[row_pieces<XF>()];
#pragma unroll
        for (int q = 0; q < row_pieces<XF>(); ++q) {
          x[q] = *reinterpret_cast<const u32x4*>(at + row * T::XB + place<T::XC>(row, row_pieces<XF>() * g + q) * 16);
          if (cut) x[q] = keep_inputs<XF>(x[q], first + q * (128 / elem_bits<XF>()), s.K);
        }
        uint32_t sc = 127;
        if constexpr (is_mx_format(XF)) {
          sc = at[kTurn * T::XB + NR * 16 * T::AC * 16 + wave * 256 + c * 4 + g];
          if (cut && first >= s.K) sc = 127;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const bf16x8 v = __builtin_bit_cast(bf16x8, token_operand<XF>(x, sc, u));
#pragma unroll
          for (int i = 0; i < NR; ++i) {
            u32x4 w = *reinterpret_cast<const u32x4*>(at + kTurn * T::XB + (16 * i + c) * 256 +
                                                      place<T::AC>(16 * i + c, 4 * g + u) * 16);
            if (cut) w = keep_inputs<AR_BF16>(w, first + 8 * u, s.K);
            acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), v, acc[i], 0, 0, 0);
          }
        }
      };
      constexpr int behind = (NS - 2) * T::loads;
      constexpr int wait_behind = 0x0070 | (behind & 15) | (behind >> 4) << 14;
      static_assert(behind < 64, "loads on their way that a wait can name");
#pragma unroll
      for (int k = 0; k < NS - 1; ++k)
        if (k < n) load(k, k);
      for (int k = 0, buf = 0; k < n; ++k) {
        // step k has arrived when at most the steps after it are on their way
        if (NS > 2 && k + NS - 2 < n) __builtin_amdgcn_s_waitcnt(wait_behind);
        else __builtin_amdgcn_s_waitcnt(0x0070);
        barrier_only();                                    // and the buffer of step k - 1 is left
        if (k + NS - 1 < n) load(k + NS - 1, buf == 0 ? NS - 1 : buf - 1);
        if (!idle) compute(k, buf);
        if (++buf == NS) buf = 0;
      }
      const int token = t0 + 16 * wave + c;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        if (token >= tokens || j0 + 16 * i >= s.rank) continue;
        f32x4 v = acc[i] * scale;
        if constexpr (XF == AR_E4M3_ROW) v *= *reinterpret_cast<const float*>(xs);
        const int d = j0 + 16 * i + 4 * g;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = d + e < s.rank ? v[e] : 0.0f;
        *reinterpret_cast<f32x4*>(s.t + split * s.t_part + r * s.t_rank + m * s.t_stride + d * 4) = v;
      }
      __syncthreads();                                     // the next turn's first loads
    }
  }
}

// The parts of t added up, in order, into the first.
struct TokenSum {
  uint8_t* t;
  int64_t part, pieces;              // bytes of a part, 16-byte pieces of it
  int32_t parts;
};
__global__ __launch_bounds__(kBlock) void k_adapter_sum(TokenSum s) {
  const int64_t at = (int64_t)blockIdx.x * kBlock + threadIdx.x;
  if (at >= s.pieces) return;
  uint8_t* p = s.t + at * 16;
  f32x4 v[kTokenParts];
#pragma unroll
  for (int k = 0; k < kTokenParts; ++k) {
    v[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (k < s.parts) v[k] = *reinterpret_cast<const f32x4*>(p + k * s.part);
  }
#pragma unroll
  for (int k = 1; k < kTokenParts; ++k)
    if (k < s.parts) v[0] += v[k];
  *reinterpret_cast<f32x4*>(p) = v[0];
}

// What the adapters add, ready in binary32, for tokens that are too few for the
// layer's largest tiles: every thread has an output, and its row of b for one
// adapter in registers, which it uses for all ranks that share b and for as many
// of its tokens as have that adapter next to each other.  So rows of b are read
// as they lie, once, where the layer's own waves would each gather them again
// for 16 tokens (64 tokens with an adapter each, rank 64, 4 shards of 8192 x 2048: 173
// us).  Bound by the stream of b.  t is the same for all threads: scalars.
struct DeltaArgs {
  const int32_t* index;
  const float* t;                    // strides in floats
  int64_t t_stride, t_rank;
  const uint8_t* b;
  int64_t b_stride, b_adapter, b_rank;
  float* delta;
  int64_t delta_stride, delta_rank;
  int32_t M, N, count, rank;
  int32_t ranks, n_blocks, m_blocks, tokens;   // ranks of one workgroup, its tokens
};
template <int R16>
__global__ __launch_bounds__(kBlock) void k_adapter_delta(DeltaArgs s) {
  int b = blockIdx.x;
  const int n = b % s.n_blocks * kBlock + threadIdx.x;
  b /= s.n_blocks;
  const int m0 = b % s.m_blocks * s.tokens, r0 = b / s.m_blocks * s.ranks;
  const uint8_t* row = s.b + r0 * s.b_rank + min(n, s.N - 1) * s.b_stride;
  u32x4 w[2 * R16];
  int have = -1;
  for (int m = m0; m < min(s.M, m0 + s.tokens); ++m) {
    const int which = ld_const(s.index, m);
    if ((uint32_t)which >= (uint32_t)s.count) continue;
    if (which != have) {
      have = which;
#pragma unroll
      for (int k = 0; k < 2 * R16; ++k) w[k] = load_b8(row + which * s.b_adapter, 8 * k, s.rank);
#pragma unroll
      for (int k = 0; k < 2 * R16; ++k) w[k] = keep_b8(w[k], 8 * k, s.rank);
    }
    for (int r = r0; r < r0 + s.ranks; ++r) {
      const float* t = s.t + r * s.t_rank + m * s.t_stride;
      float sum = 0.0f;
#pragma unroll
      for (int k = 0; k < R16; ++k) {                      // (t's row ends with a multiple of 16)
        if (16 * k >= s.rank) continue;
        float part = 0.0f;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint32_t d = w[2 * k + u / 4][u % 4];
          part = __builtin_fmaf(ld_const(t, 16 * k + 2 * u), bf_lo(d), part);
          part = __builtin_fmaf(ld_const(t, 16 * k + 2 * u + 1), bf_hi(d), part);
        }
        sum += part;
      }
      if (n < s.N) s.delta[r * s.delta_rank + m * s.delta_stride + n] = sum;
    }
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
  const int64_t each = (int64_t(1) << 60) / q->adapters;
  if (q->a_adapter_stride > each || q->b_adapter_stride > each) return AR_ESIZE;
  if (q->b_stride >= 1 << 23) return AR_ESIZE;             // 128 rows' offsets stay 32-bit
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

static int64_t t_row_bytes(const ar_adapter_params* q) { return ceil_div64(q->rank, 16) * 16 * 4; }

// Workgroups that share K (up to 128 in all), and those that share a group's
// adapters, for about 1024 in all, of which many may have no turn: 4096 x 8192,
// rank 64, one adapter for 512 tokens 21 us, rank 16 with 16 adapters in any order 23;
// 512 tokens 4, 6.5 with half as many shares of K.
constexpr int kTokenBlocks = 1024;

// Outputs of all ranks up to which up to 16 dimensions of 16 tokens' adapters are
// left to the layer's own waves, against sums made ready, K 2048, with an adapter for
// each token (and one for all): 4 x 16 x 4096 12.6 and 15.8 us (12.6 and 15.8),
// 4 x 16 x 8192 18.6 and 18.8 (14.9 and 18.4), 1 x 16 x 65536 29.7 and 29.5 (23.7 and
// 27.1), 8 x 16 x 8192 30.4 and 28.7 (23.7 and 27.5).
constexpr int64_t kLaneOutputs = 1 << 19;

struct TokenPlan {
  int32_t nr, splits, slots;         // nr 0: few tokens
};
static TokenPlan plan_tokens(const ar_linear_params* p, const ar_adapter_params* q) {
  TokenPlan t{0, 1, 1};
  if (p->rows <= kFewTokens ||
      (p->rows <= 1024 && p->rows * t_ranks(p, q) * p->inputs * q->rank <= kFewProducts))
    return t;
  t.nr = q->rank <= 16 ? 1 : (q->rank <= 32 ? 2 : 4);
  const int64_t blocks = t_ranks(p, q) * ceil_div64(p->rows, kTokenGroup) * ceil_div64(q->rank, 16 * t.nr);
  const int64_t steps = ceil_div64(p->inputs, 256);        // two steps each at least
  while (t.splits < kTokenParts && 2 * t.splits <= steps && blocks * t.splits < 128) t.splits *= 2;
  const int64_t group = p->rows < kTokenGroup ? p->rows : kTokenGroup;
  const int64_t turns = group < q->adapters + 4 ? group : q->adapters + 4;
  while (t.slots < turns && blocks * t.splits * t.slots < kTokenBlocks) t.slots *= 2;
  return t;
}

// Bytes of t, and of the sums that are made ready for the layer (0: none are).
static int64_t t_bytes(const ar_linear_params* p, const ar_adapter_params* q) {
  return (plan_tokens(p, q).splits * t_ranks(p, q) * p->rows * t_row_bytes(q) + 255) / 256 * 256;
}
static int64_t delta_row(const ar_linear_params* p) { return (p->outputs + 3) / 4 * 4; }
static int64_t delta_bytes(const ar_linear_params* p, const ar_adapter_params* q) {
  const MxLinArgs a = linear_args(p);
  if (large_tiles(a, p->nranks)) return 0;
  if (p->rows <= 16 && q->rank <= 16 && p->nranks * p->rows * p->outputs <= kLaneOutputs) return 0;
  return (p->nranks * p->rows * delta_row(p) * 4 + 255) / 256 * 256;
}

// A work buffer that does for these tokens and for any fewer: both forms of t, and
// sums made ready, need less again from some number of tokens on.  Of t, shares of K
// are kTokenParts at most, and fewer than 256 for each group of kTokenGroup tokens
// together; sums are made ready up to where the largest tiles begin.
static int64_t adapter_work(const ar_linear_params* p, const ar_adapter_params* q) {
  if (!adapters_count(p, q)) return 0;
  int64_t t = t_ranks(p, q) * p->rows;
  if (p->rows > kFewTokens) {
    const int64_t groups = ceil_div64(q->rank, 64), shares = 256 * kTokenGroup / groups;
    const int64_t most = kTokenParts * t < shares ? kTokenParts * t : shares;
    if (t < most) t = most;
  }
  ar_linear_params few = *p;
  MxLinArgs a = linear_args(p);
  if (large_tiles(a, p->nranks)) {
    int64_t small = 1, large = p->rows;                    // the first number of tokens with the largest tiles
    while (small + 1 < large) {
      a.M = (int32_t)((small + large) / 2);
      if (large_tiles(a, p->nranks)) large = a.M;
      else small = a.M;
    }
    few.rows = small;
  }
  return (t * t_row_bytes(q) + 255) / 256 * 256 + delta_bytes(&few, q);
}

static hipError_t launch_delta(const Adapters& ad, const MxLinArgs& a, int nranks, hipStream_t s) {
  DeltaArgs d{};
  d.index = ad.index;
  d.t = reinterpret_cast<const float*>(ad.t);
  d.t_stride = ad.t_stride / 4;
  d.t_rank = ad.t_rank / 4;
  d.b = ad.b;
  d.b_stride = ad.b_stride;
  d.b_adapter = ad.b_adapter;
  d.b_rank = ad.b_rank;
  d.delta = const_cast<float*>(ad.delta);
  d.delta_stride = ad.delta_stride;
  d.delta_rank = ad.delta_rank;
  d.N = a.N;
  d.count = ad.count;
  d.rank = ad.rank;
  d.ranks = ad.b_rank == 0 ? nranks : 1;
  d.n_blocks = (a.N + kBlock - 1) / kBlock;
  // (at most 2^22 of them, so a launch takes 4 ranks' at least)
  const int groups = nranks / d.ranks;
  const int64_t at_once = most_blocks(kBlock) / d.n_blocks;
  const int each = (int)(at_once < groups ? at_once : groups);
  // tokens of a workgroup: as many as leave 1024 workgroups, at most 16
  const int64_t all = (int64_t)each * d.n_blocks;
  int64_t tokens = all * a.M / 1024;
  tokens = tokens < 1 ? 1 : (tokens > 16 ? 16 : tokens);
  d.tokens = (int32_t)tokens;
  const int64_t most = most_blocks(kBlock) / all * tokens;
  for (int r = 0; r < groups; r += each) {
    const int ranks = groups - r < each ? groups - r : each;
    for (int64_t m = 0; m < a.M; m += most) {
      d.M = (int32_t)(a.M - m < most ? a.M - m : most);
      d.m_blocks = (int32_t)ceil_div64(d.M, tokens);
      d.index = ad.index + m;
      d.t = reinterpret_cast<const float*>(ad.t + r * ad.t_rank + m * ad.t_stride);
      d.b = ad.b + r * ad.b_rank;
      d.delta = const_cast<float*>(ad.delta) + r * ad.delta_rank + m * ad.delta_stride;
      const dim3 grid((unsigned)((int64_t)ranks * d.n_blocks * d.m_blocks)), block(kBlock);
      const hipError_t e = ad.rank <= 16   ? launch(k_adapter_delta<1>, grid, block, s, d)
                           : ad.rank <= 32 ? launch(k_adapter_delta<2>, grid, block, s, d)
                           : ad.rank <= 64 ? launch(k_adapter_delta<4>, grid, block, s, d)
                                           : launch(k_adapter_delta<8>, grid, block, s, d);
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

template <int XF, int NR>
static hipError_t launch_tokens(const TokenArgs& a0, int ranks, hipStream_t s) {
  TokenArgs a = a0;
  a.r_groups = (a.rank + 16 * NR - 1) / (16 * NR);
  const int64_t each = (int64_t)ranks * a.r_groups * a.slots * a.splits;
  const int64_t most = most_blocks(kBlock) / each * kTokenGroup;
  for (int64_t m = 0; m < a0.M; m += most) {
    a.M = (int32_t)(a0.M - m < most ? a0.M - m : most);
    a.m_groups = (a.M + kTokenGroup - 1) / kTokenGroup;
    a.x = a0.x + m * a0.x_stride;
    if (a0.xs) a.xs = a0.xs + m * a0.xs_stride;
    a.index = a0.index + m;
    a.t = a0.t + m * a0.t_stride;
    const hipError_t e = launch(k_adapter_tokens<XF, NR>, dim3((unsigned)(each * a.m_groups)),
                                dim3(kBlock), s, a);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int XF>
static hipError_t launch_few_tokens(const TokenArgs& a0, int ranks, hipStream_t s) {
  TokenArgs a = a0;
  const bool share = a.K > 512;                            // K is long enough for 4 waves
  a.r_groups = (a.rank + 15) / 16 * (share ? 4 : 1);
  const dim3 grid((unsigned)(ranks * a.M * a.r_groups)), block(kBlock);
  return share ? launch(k_adapter_few_tokens<XF, kWavesPerBlock>, grid, block, s, a)
               : launch(k_adapter_few_tokens<XF, 1>, grid, block, s, a);
}

template <int XF>
static hipError_t launch_tokens_x(const TokenArgs& a, const TokenPlan& t, int ranks, hipStream_t s) {
  if (t.nr == 0) return launch_few_tokens<XF>(a, ranks, s);
  if (t.nr == 1) return launch_tokens<XF, 1>(a, ranks, s);
  if (t.nr == 2) return launch_tokens<XF, 2>(a, ranks, s);
  return launch_tokens<XF, 4>(a, ranks, s);
}

static hipError_t launch_tokens_any(const TokenArgs& a, const TokenPlan& t, int xf, int ranks, hipStream_t s) {
  switch (xf) {
    case AR_BF16: return launch_tokens_x<AR_BF16>(a, t, ranks, s);
    case AR_E4M3_ROW: return launch_tokens_x<AR_E4M3_ROW>(a, t, ranks, s);
    case AR_E4M3_MX: return launch_tokens_x<AR_E4M3_MX>(a, t, ranks, s);
    default: return launch_tokens_x<AR_E2M1_MX>(a, t, ranks, s);
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
  const TokenPlan plan = plan_tokens(p, q);
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
  t.t_stride = t_row_bytes(q);
  t.t_rank = ranks > 1 ? p->rows * t.t_stride : 0;
  t.t_part = ranks * p->rows * t.t_stride;
  t.M = a.M;
  t.K = a.K;
  t.nb = a.nb;
  t.splits = plan.splits;
  t.slots = plan.slots;
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
  hipError_t e = launch_tokens_any(t, plan, p->x_format, ranks, s);
  if (e == hipSuccess && plan.splits > 1) {
    const TokenSum sum{t.t, t.t_part, t.t_part / 16, plan.splits};
    // (shares of K are for 2^15 tokens at most)
    e = launch(k_adapter_sum, dim3((unsigned)ceil_div64(sum.pieces, kBlock)), dim3(kBlock), s, sum);
  }
  if (delta_bytes(p, q) > 0) {
    ad.delta = reinterpret_cast<const float*>(t.t + t_bytes(p, q));
    ad.delta_stride = delta_row(p);
    ad.delta_rank = p->rows * ad.delta_stride;
    if (e == hipSuccess) e = launch_delta(ad, a, p->nranks, s);
  }
  if (e != hipSuccess) return map_hip(e);
  return map_hip(launch_pieces(a, ad, p->x_format, p->y_format, p->nranks, s));
}

}  // extern "C"
