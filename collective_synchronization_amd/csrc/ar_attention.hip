// ar_attention.hip -- decode attention over a shared prefix and every sequence's
// own tokens, both in one paged cache (gfx950):
//     out = softmax(scale * q K^T) V
// The sequences of a batch that share a prefix are, for each head of the cache,
// many rows of one product with the same keys: those keys are read once, for
// all of them.  A sequence's own tokens meet the heads of its group alone.
//
// Two kernels.  The first one takes ranges of keys, prefix and own ones in one
// launch, and leaves for each row and range the sum of its values under the
// weights 2^(s - r), the sum l of those weights and the reference r; the second
// joins a row's ranges.
// Scores are kept in units of log2: s = q.k * scale * log2(e).
//
// The products take keys as their first operand, so a lane holds scores of one
// row (its column), and those registers are the second operand of the product
// with the values as they are: keys may be summed in any order, and the values
// are read from shared memory, transposed on the way, in the order that the
// scores came in.  Sums, maxima and the joined outputs are binary32; the weights
// are rounded to 16 bits for the matrix cores, which is what their operands
// are: each by at most half a step, and their sum l is of the unrounded ones.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "../../include/ar.h"
#include "ar_cache.h"
#include "ar_host.h"
#include "ar_rows.h"

namespace ar {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kAttnThreads = 256;
constexpr int kAttnWaves = kAttnThreads / kWave;
constexpr int kTileRows = 32 * kAttnWaves;   // rows of a workgroup in the tile form
constexpr int kFewRows = 16;                 // up to these, the other form

// Strides in bytes for the cache, in elements for q, out and lse.
struct AttnArgs {
  CacheView kv;
  const uint8_t* q;
  int64_t q_stride, q_head;
  void* out;
  int64_t out_stride, out_head;
  float* lse;
  int64_t lse_stride;
  const int32_t* prefix_pages;
  const int32_t* lengths;
  const int32_t* tables;
  int64_t table_stride;
  float* part_o;                     // [parts][rows][dim]
  float* part_m;                     // [parts][rows][2]: r, l
  float c;                           // scale * log2(e)
  int32_t prefix, capacity;          // tokens shared, and most own ones
  int32_t sequences, queries, heads, group;
  int32_t rows;                      // sequences * queries * heads
  int32_t prefix_splits, prefix_chunk, prefix_tiles, prefix_blocks;
  int32_t own_splits, own_tiles, own_blocks;
};

// ------------------------------------------------------- 16-bit operands ---

template <int F>
__device__ __forceinline__ f32x16 mma32(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (F == AR_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
template <int F>
__device__ __forceinline__ f32x4 mma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (F == AR_BF16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Two values of a 16-bit type, nearest even.
template <int F>
__device__ __forceinline__ uint32_t pair16(float lo, float hi) {
  if constexpr (F == AR_BF16) return bf16_pair(lo, hi);
  else return __builtin_bit_cast(uint32_t, f16x2{(_Float16)lo, (_Float16)hi});
}

// Two binary32 weights as two bf16 parts each, off by 2^-16 together: the first
// is cut, not rounded, and the rest, which has 2^-23 of the weight added, is therefore
// above zero wherever the weight is: times an infinite value both are the same
// infinity.  SCALED: weights times scales, which may be infinities; these are in the rest
// (64 x 2 tokens behind 8192, fp16 on an 8-bit cache: 84 us, 77 with rounded parts, which
// make NaNs of infinities).
struct Parts16 {
  uint32_t top, rest;
};
template <bool SCALED>
__device__ __forceinline__ Parts16 parts16(float lo, float hi) {
  constexpr float most = 0x1.fffffep127f, more = 0x1.000002p0f;
  const float a = SCALED ? __builtin_amdgcn_fmed3f(lo, -most, most) : lo;
  const float b = SCALED ? __builtin_amdgcn_fmed3f(hi, -most, most) : hi;
  const uint32_t u = __float_as_uint(a), v = __float_as_uint(b);
  return Parts16{__builtin_amdgcn_perm(v, u, 0x07060302u),
                 bf16_pair(__builtin_fmaf(lo, more, -bf_hi(u)), __builtin_fmaf(hi, more, -bf_hi(v)))};
}

// 8 e4m3 codes in a 16-bit type, without loss.
template <int F>
__device__ __forceinline__ u32x4 wide8(uint32_t lo, uint32_t hi) {
  if constexpr (F == AR_BF16)
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true))};
  else
    return u32x4{__builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false)),
                 __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true))};
}

// 4 consecutive rows' elements of one column: lane i of 16 names row i / 4,
// columns 4 * (i % 4) on, and receives column i.
__device__ __forceinline__ u32x2 read_transposed(const uint8_t* p) {
  typedef __attribute__((address_space(3))) s16x4 lds_t;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)p));
}

__device__ __forceinline__ float other_half_max(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float other_half_sum(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float other_row_max(float v) {     // lanes l and l ^ 16
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float other_row_sum(float v) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Where the maximum of a row has grown by less than 2^kSlack since the weights'
// reference was taken, the reference stays: no sum has to be scaled, and the
// weights stay below 2^kSlack.  In fp16 they are 2^kF16Up times as large, so that
// those down to 2^-20 of the largest keep their bits; smaller ones are subnormal there,
// each off by up to 2^-31 of the largest.
constexpr float kSlack = 8.0f;
constexpr float kF16Up = 6.0f;
template <int F> constexpr float weights_up() { return F == AR_F16 ? kF16Up : 0.0f; }

constexpr int pow2_up(int n) { int p = 1; while (p < n) p *= 2; return p; }

// What a workgroup works on: `rows` rows that meet the same keys [k0, k1).
struct Piece {
  const int32_t* table;
  int32_t kh;                        // head of the cache
  int32_t k0, k1;
  int32_t rows, row0;                // and the first one of this workgroup
  int32_t token0;                    // token of row 0
  int32_t limit0;                    // keys that the first token sees, one more with each next ...
  bool causal;                       // ... or all of them the same
  int32_t part;
};

// ---------------------------------------------------------------- forms ---

// 16 bytes a lane straight into shared memory, at `lds` (the wave's own address)
// + 16 * lane.
__device__ __forceinline__ void load_to_lds(rsrc_t r, uint8_t* lds, uint32_t off) {
  typedef __attribute__((address_space(3))) void lds_void;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, off, 0, 0, 0);
}
constexpr uint32_t kNowhere = 0x80000000u;   // past every range: reads as zeros

// Masks, in integer arithmetic: a condition for each of many values would take more
// scalar registers than there are, and cost the loops around it theirs.
// Which halves of a pair of 16-bit values are infinities or NaNs: all ones there.
template <int F>
__device__ __forceinline__ uint32_t odd_halves(uint32_t v) {
  constexpr uint32_t exponent = F == AR_BF16 ? 0x7F807F80u : 0x7C007C00u, one = F == AR_BF16 ? 0x00800080u : 0x04000400u;
  const uint32_t top = ((v & exponent) + one) & 0x80008000u;
  return top | (top - (top >> 15));
}
// All ones for an infinity or a NaN.
__device__ __forceinline__ uint32_t odd_mask(float v) {
  return (uint32_t)((int32_t)((__float_as_uint(v) & kInfBits) + 0x00800000u) >> 31);
}
__device__ __forceinline__ uint32_t nonzero_mask(uint32_t v) {       // below 2^31
  return (uint32_t)(-(int32_t)v >> 31);
}
__device__ __forceinline__ uint32_t choose(uint32_t mask, uint32_t one, uint32_t zero) {
  return (one & mask) | (zero & ~mask);
}
// What an infinity or a NaN counts for, as a 16-bit value: powers of two (2^14 for a
// NaN, 2^7 and 1), so that a sum over up to 64 keys says how many there are of each.
template <int F>
__device__ __forceinline__ uint32_t count_of(uint32_t nan, uint32_t negative) {
  constexpr bool b = F == AR_BF16;
  return choose(nan, b ? 0x4680u : 0x7400u, choose(negative, b ? 0x4300u : 0x5800u, b ? 0x3F80u : 0x3C00u));
}
__device__ __forceinline__ float add_counted(float sum, float count) {
  const uint32_t n = (uint32_t)count;
  float v = (n & 127) != 0 ? __builtin_inff() : 0.0f;
  if ((n >> 7 & 127) != 0) v = v == 0.0f ? -__builtin_inff() : __builtin_nanf("");
  return n == 0 ? sum : sum + (n >> 14 != 0 ? __builtin_nanf("") : v);
}

template <int I> struct Index { static constexpr int value = I; };
template <int N, int I = 0, class F>
__device__ __forceinline__ void for_each(F f) {
  if constexpr (I < N) {
    f(Index<I>{});
    for_each<N, I + 1>(f);
  }
}

// LATER: there may be tokens that other tokens of their step do not see (two and
// more queries of a sequence).
template <int QF, bool C8, int DT, bool LATER>
struct Attn {
  static constexpr int VF = C8 ? AR_BF16 : QF;             // type of weights and values
  // Weights times the scales of 8-bit values can have any exponent, so they are
  // bf16; for fp16 outputs in two parts, since one alone has 3 bits too few.
  static constexpr bool two = C8 && QF == AR_F16;
  // (few rows take bf16 ones always so: they wait for memory, and their times do not change)
  static constexpr bool few_two = VF == AR_BF16;
  static constexpr int KT = DT > 128 ? 32 : 64;            // keys of a tile
  static constexpr int CB = C8 ? 16 : 8;                   // elements of 16 bytes of the cache
  static constexpr int CH = pow2_up(DT / CB);              // lanes to a row
  static constexpr int wave_keys = kWave / CH;             // rows that a wave loads at once: at most 16, on one page
  static constexpr int passes = KT * CH / kAttnThreads;
  // Rows in shared memory: C16 pieces of 8 elements.  16 rows' reads of one piece
  // (keys), and 4 rows' of four (values), meet different banks, since pieces are
  // permuted by the row; loads straight into shared memory have the permutation in
  // their addresses.
  static constexpr int C16 = pow2_up(DT / 8), RS = C16 * 16;
  static constexpr int tile = 2 * KT * RS + (C8 ? KT * 8 : 0);
  static constexpr int few_step = 32 * RS + (C8 ? 32 * 8 : 0);
  static constexpr int few_wave = (C8 ? 1 : 2) * few_step; // (8-bit values wait in registers)
  static constexpr int few_join = kAttnWaves * (16 * DT * 4 + 16 * 8);
  static constexpr int few = kAttnWaves * few_wave > few_join ? kAttnWaves * few_wave : few_join;
  static constexpr int lds = 2 * tile > few ? 2 * tile : few;
  static_assert(wave_keys <= 16 && KT * CH % kAttnThreads == 0, "");

  static __device__ __forceinline__ int swap_k(int row) { return C16 == 8 ? row >> 1 & 7 : row & 15; }
  static __device__ __forceinline__ int swap_v(int row) { return C16 == 8 ? (row >> 1 & 1) << 2 : (row & 3) << 2; }

  // Pages of the N 16-key runs from `key` on; -1 for those that are none, or past the end.
  template <int N>
  struct Pages {
    int at[N];
    // Run B + sub, sub < S.
    template <int B, int S>
    __device__ __forceinline__ int of(int sub) const {
      int page = at[B];
      if constexpr (S > 1) page = sub == 1 ? at[B + 1] : page;
      if constexpr (S > 2) page = sub == 2 ? at[B + 2] : page;
      if constexpr (S > 3) page = sub == 3 ? at[B + 3] : page;
      return page;
    }
  };
  template <int N>
  static __device__ __forceinline__ Pages<N> find_pages(const AttnArgs& a, const Piece& p, int key) {
    Pages<N> r;
#pragma unroll
    for (int i = 0; i < N; ++i) r.at[i] = ld_const(p.table, min(key + 16 * i, p.k1 - 1) >> a.kv.page_shift);
    return r;
  }
  template <int N>
  static __device__ __forceinline__ void check_pages(const AttnArgs& a, const Piece& p, int key, Pages<N>& r) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (key + 16 * i >= p.k1 || (uint32_t)r.at[i] >= (uint32_t)a.kv.pages) r.at[i] = -1;
  }
  // Of checked ones, those that are none (past the end they are, too).
  template <int N>
  static __device__ __forceinline__ uint32_t missing(const Pages<N>& r) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) m |= r.at[i] < 0 ? 1u << i : 0u;
    return m;
  }
  // The rows of a run of 16 tokens from `key` on, as far as they go: where the first
  // one's keys and values are, and bytes up to the last one's end.
  struct Run {
    int64_t at;
    uint32_t range;
  };
  static __device__ __forceinline__ Run run_of(const AttnArgs& a, const Piece& p, int page, int key) {
    const int count = min(16, p.k1 - key);
    if (page < 0 || count <= 0) return Run{0, 0};
    return Run{page * a.kv.page_stride + (key & (a.kv.page - 1)) * a.kv.token_stride + p.kh * a.kv.head_stride,
               (uint32_t)(count - 1) * (uint32_t)a.kv.token_stride + (uint32_t)(a.kv.dim * (C8 ? 1 : 2))};
  }
  static __device__ __forceinline__ rsrc_t rows(const uint8_t* base, const Run& r) {
    // (the same for all lanes, which the compiler does not always see)
    const uint64_t from = (uint64_t)(base + r.at);
    const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)from);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((int)(uint32_t)(from >> 32));
    return make_rsrc(reinterpret_cast<const void*>((uint64_t)hi << 32 | lo),
                     __builtin_amdgcn_readfirstlane((int)r.range));
  }
  // Scales: each lane has its own key, whose page it has read before.
  static __device__ __forceinline__ int scale_page(const AttnArgs& a, const Piece& p, int key) {
    return C8 ? p.table[min(key, p.k1 - 1) >> a.kv.page_shift] : -1;
  }
  static __device__ __forceinline__ float load_scale(const AttnArgs& a, const Piece& p, const float* base, int page,
                                                     int key) {
    if ((uint32_t)page >= (uint32_t)a.kv.pages || key >= p.k1) return 0.0f;
    return base[page * a.kv.scale_page_stride + (key & (a.kv.page - 1)) * a.kv.scale_token_stride +
                p.kh * a.kv.scale_head_stride];
  }
  // 16 bytes of the cache as 16-bit values of row `row` in shared memory.
  template <int F>
  static __device__ __forceinline__ void store8(uint8_t* rows, int row, int swap, int c, u32x4 v) {
    static_assert(C8, "");
    if (c * 16 >= DT) return;
    *reinterpret_cast<u32x4*>(rows + row * RS + ((2 * c) ^ swap) * 16) = wide8<F>(v.x, v.y);
    *reinterpret_cast<u32x4*>(rows + row * RS + ((2 * c + 1) ^ swap) * 16) = wide8<F>(v.z, v.w);
  }

  static __device__ __forceinline__ const uint8_t* query(const AttnArgs& a, const Piece& p, int row) {
    row = min(row, p.rows - 1);
    const int token = p.token0 + row / a.group, head = p.kh * a.group + row % a.group;
    return a.q + (token * a.q_stride + head * a.q_head) * 2;
  }
  static __device__ __forceinline__ u32x4 query8(const AttnArgs& a, const uint8_t* row, int d) {
    return d < a.kv.dim ? ldg16(row + d * 2) : u32x4{0u, 0u, 0u, 0u};
  }
  // What a token of the step does not see may not touch it, be it an infinity or a
  // NaN, which its weight 0 would make NaN.  So where keys that some of the rows do
  // not see have such values, or scales (values_odd), these are taken out, and for
  // each output those of the keys that it sees are counted by a product, for what
  // they make of it.
  static __device__ __forceinline__ bool values_odd(const uint8_t* values, const float* scales, int n, int lane) {
    uint32_t odd = 0;
    for (int i = lane; i < n * C16; i += kWave) {
      // (what lies behind a row of 8-bit codes is not written)
      if (C8 && C16 > DT / 8 && ((i % C16) ^ swap_v(i / C16)) >= DT / 8) continue;
      const u32x4 v = *reinterpret_cast<const u32x4*>(values + i * 16);
      odd |= odd_halves<VF>(v.x) | odd_halves<VF>(v.y) | odd_halves<VF>(v.z) | odd_halves<VF>(v.w);
    }
    if constexpr (C8) {
      if (lane < n && abs_bits(scales[lane]) >= kInfBits) odd = 1;
    }
    return __any(odd != 0);
  }
  // Halves of two keys' values that are odd, or whose scales are.
  static __device__ __forceinline__ uint32_t odd_pair(uint32_t v, const float* scale) {
    uint32_t odd = odd_halves<VF>(v);
    if constexpr (C8) odd |= (odd_mask(scale[0]) & 0xFFFFu) | (odd_mask(scale[1]) & 0xFFFF0000u);
    return odd;
  }
  // 8 keys' weights of a row, and a column's values without odd ones.  `sum`: the
  // weights are added to it one by one, as they are where nothing is odd, so that bits
  // do not depend on the values' way.
  struct Apart {
    u32x4 w, w2, v;
  };
  template <bool TWO>
  static __device__ __forceinline__ Apart apart(const float (&score)[8], float c, float ref, const float (&scale)[8],
                                                u32x4 v, float& sum) {
    Apart x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float e[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        e[u] = __builtin_amdgcn_exp2f(__builtin_fmaf(score[2 * j + u], c, -ref));
        sum += e[u];
        if constexpr (C8) {
          const float by = scale[2 * j + u];
          e[u] *= __uint_as_float(__float_as_uint(by) & ~odd_mask(by));
        }
      }
      if constexpr (TWO) {
        const Parts16 p = parts16<C8>(e[0], e[1]);
        x.w[j] = p.top;
        x.w2[j] = p.rest;
      } else {
        x.w[j] = pair16<VF>(e[0], e[1]);
        x.w2[j] = 0;
      }
      x.v[j] = v[j] & ~odd_pair(v[j], scale + 2 * j);
    }
    return x;
  }
  // 1 for those of 8 keys that are seen, and what a column's odd values count for.
  struct Counted {
    u32x4 seen, odd;
  };
  static __device__ __forceinline__ Counted counted(const float (&score)[8], const float (&scale)[8], u32x4 v) {
    Counted x;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t odd = odd_pair(v[j], scale + 2 * j);
      float s[2];
      x.odd[j] = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        s[u] = score[2 * j + u] == -__builtin_inff() ? 0.0f : 1.0f;
        const uint32_t mine = v[j] >> 16 * u & 0xFFFFu;
        uint32_t nan = nonzero_mask(mine & (VF == AR_BF16 ? 0x7Fu : 0x3FFu)), negative = nonzero_mask(mine & 0x8000u);
        if constexpr (C8) {                                // codes are NaNs alone, scales infinities, too
          const uint32_t by = __float_as_uint(scale[2 * j + u]);
          nan = odd_halves<VF>(mine) | nonzero_mask(by & 0x7FFFFFu) | ~nonzero_mask(mine & 0x7FFFu);
          negative ^= (uint32_t)((int32_t)by >> 31);
        }
        x.odd[j] |= count_of<VF>(nan, negative) << 16 * u;
      }
      x.odd[j] &= odd;
      x.seen[j] = pair16<VF>(s[0], s[1]);
    }
    return x;
  }
  // Row of the parts' arrays.
  static __device__ __forceinline__ int64_t out_row(const AttnArgs& a, const Piece& p, int row) {
    return (int64_t)p.part * a.rows + (int64_t)(p.token0 + row / a.group) * a.heads + p.kh * a.group + row % a.group;
  }

  // Many rows: bound by the matrix cores and the exponentials beside them.  Each
  // wave has 32 rows, and tiles of KT keys pass through shared memory, the next
  // one on its way while one is multiplied (8-bit ones in registers, since they
  // are converted), and the pages of the one after that.  Two waves to a SIMD take
  // turns with matrix cores and vector units.  128 x 64 heads over 32768: bf16 168 us
  // (0.82 PFLOP/s), 8-bit 194; the matrix cores are busy 42% and 33% of the cycles.
  // With the scores of the next tile formed beside the weights of this one 222 and 295,
  // where this form took 190 and 222: registers and shared memory for it cost more
  // than it hides.  With LATER, heads of 128 and 8-bit rows 44 to 58 vector registers
  // are spilled (64 x 2 tokens behind 8192 73 us, 62 in bf16).
  static __device__ void many_rows(const AttnArgs& a, const Piece& p, uint8_t* smem) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    const int first = p.row0 + wave * 32, row = first + col;
    const bool idle = first >= p.rows;
    constexpr int runs = KT / 16, pass_keys = kAttnThreads / CH;
    auto pages = find_pages<runs>(a, p, p.k0);
    int of_scale = scale_page(a, p, p.k0 + tid % KT);
    u32x4 q[DT / 16];
    {
      const uint8_t* at = query(a, p, row);
#pragma unroll
      for (int s = 0; s < DT / 16; ++s) q[s] = query8(a, at, 16 * s + 8 * half);
    }
    const int limit = p.causal ? min(p.k1, p.limit0 + min(row, p.rows - 1) / a.group) : p.k1;
    const int least = p.causal ? min(p.k1, p.limit0 + p.row0 / a.group) : p.k1;
    f32x16 o[DT / 32];
#pragma unroll
    for (int i = 0; i < DT / 32; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[i][r] = 0.0f;
    float top = -__builtin_inff(), ref = 0.0f, l = 0.0f;

    // this lane's piece of a row: as loaded, and straight into its place
    uint32_t k_off[passes], v_off[passes];
    const int piece = lane % CH, key_in = lane / CH;
#pragma unroll
    for (int i = 0; i < passes; ++i) {
      const int k = i * pass_keys + wave * wave_keys + key_in;
      const int kc = C8 ? piece : piece ^ swap_k(k), vc = C8 ? piece : piece ^ swap_v(k);
      k_off[i] = kc * CB < a.kv.dim ? (uint32_t)(k & 15) * (uint32_t)a.kv.token_stride + kc * 16 : kNowhere;
      v_off[i] = vc * CB < a.kv.dim ? (uint32_t)(k & 15) * (uint32_t)a.kv.token_stride + vc * 16 : kNowhere;
    }
    u32x4 kr[C8 ? passes : 1], vr[C8 ? passes : 1];
    float scale = 0.0f;
    auto load_tile = [&](int key, int buf) {
      uint8_t* at = smem + buf * tile;
      for_each<passes>([&](auto pass) {
        constexpr int i = pass.value;
        const int k = i * pass_keys + wave * wave_keys;    // of the tile; on one page with the wave's others
        constexpr int each = pass_keys > 16 ? pass_keys / 16 : 1;
        const int page = pages.template of<i * pass_keys / 16, each>(wave * wave_keys / 16);
        const Run run = run_of(a, p, page, key + (k & ~15));
        const rsrc_t kp = rows(a.kv.k, run), vp = rows(a.kv.v, run);
        if constexpr (C8) {
          kr[i] = __builtin_amdgcn_raw_buffer_load_b128(kp, k_off[i], 0, 0);
          vr[i] = __builtin_amdgcn_raw_buffer_load_b128(vp, v_off[i], 0, 0);
        } else {
          load_to_lds(kp, at + k * RS, k_off[i]);
          load_to_lds(vp, at + KT * RS + k * RS, v_off[i]);
        }
      });
      if constexpr (C8) {
        if (tid < 2 * KT)
          scale = load_scale(a, p, tid < KT ? a.kv.k_scales : a.kv.v_scales, of_scale, key + tid % KT);
      }
    };
    auto store_tile = [&](int buf) {
      uint8_t* at = smem + buf * tile;
      if constexpr (C8) {
#pragma unroll
        for (int i = 0; i < passes; ++i) {
          const int k = i * pass_keys + wave * wave_keys + key_in;
          store8<QF>(at, k, swap_k(k), piece, kr[i]);
          store8<VF>(at + KT * RS, k, swap_v(k), piece, vr[i]);
        }
        if (tid < 2 * KT) reinterpret_cast<float*>(at + 2 * KT * RS)[tid] = scale;
      }
    };
    // every wave's pieces of the tile are there
    auto arrived = [&]() {
      if constexpr (C8) {
        __syncthreads();
      } else {
        compiler_barrier();
        __builtin_amdgcn_s_waitcnt(0x0070);                // vmcnt and lgkmcnt
        __builtin_amdgcn_s_barrier();
        compiler_barrier();
      }
    };

    check_pages(a, p, p.k0, pages);
    load_tile(p.k0, 0);
    uint32_t gone = missing(pages);
    pages = find_pages<runs>(a, p, p.k0 + KT);
    of_scale = scale_page(a, p, p.k0 + KT + tid % KT);
    store_tile(0);
    arrived();
    // group of 16 lanes: columns 16 * (group % 2) on, keys 4 * half on and 8 after them
    const int vk = 4 * half + (lane & 15) / 4, vc = 2 * (lane >> 4 & 1) + (lane & 3) / 2;
    const int k_base = col * RS, k_swap = half ^ swap_k(col);
    const int v_base = KT * RS + vk * RS + (lane & 1) * 8, v_swap = vc ^ swap_v(vk);
    int buf = 0;
    auto step = [&](auto all_see, int key) {
      const bool more = key + KT < p.k1;
      uint32_t next_gone = 0;
      if (more) {
        check_pages(a, p, key + KT, pages);
        load_tile(key + KT, buf ^ 1);
        next_gone = missing(pages);
        pages = find_pages<runs>(a, p, key + 2 * KT);
        of_scale = scale_page(a, p, key + 2 * KT + tid % KT);
      }
      if (!idle) {
        const uint8_t* ks = smem + buf * tile;
        const float* sc = reinterpret_cast<const float*>(ks + 2 * KT * RS);
        f32x16 s[KT / 32];
#pragma unroll
        for (int t = 0; t < KT / 32; ++t)
#pragma unroll
          for (int r = 0; r < 16; ++r) s[t][r] = 0.0f;
        // these come first among the waves of a SIMD, with 8 reads ahead of the products
        // (up to 3% less time; heads above 128, alone on their SIMD, do not gain)
        if constexpr (DT <= 128) __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < DT / 16; ++i)
#pragma unroll
          for (int t = 0; t < KT / 32; ++t)
            s[t] = mma32<QF>(*reinterpret_cast<const u32x4*>(ks + k_base + 32 * t * RS + ((2 * i) ^ k_swap) * 16), q[i], s[t]);
        __builtin_amdgcn_sched_group_barrier(0x100, 8, 0);           // reads of shared memory
#pragma unroll
        for (int i = 0; i < DT / 16 - 4; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x8, KT / 32, 0);     // products
          __builtin_amdgcn_sched_group_barrier(0x100, KT / 32, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x8, 4 * KT / 32, 0);
        if constexpr (DT <= 128) __builtin_amdgcn_s_setprio(0);
        if constexpr (C8) {
#pragma unroll
          for (int t = 0; t < KT / 32; ++t)
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
              const f32x4 m = *reinterpret_cast<const f32x4*>(sc + 32 * t + 2 * r + 4 * half);
#pragma unroll
              for (int j = 0; j < 4; ++j) s[t][r + j] *= m[j];
            }
        }
        if (gone != 0 || !all_see.value) {
#pragma unroll
          for (int t = 0; t < KT / 32; ++t)
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const int at = 32 * t + 8 * (r >> 2) + 4 * half + (r & 3);
              if (key + at >= limit || (gone >> (at >> 4) & 1)) s[t][r] = -__builtin_inff();
            }
        }
        float m = s[0][0];
#pragma unroll
        for (int t = 0; t < KT / 32; ++t)
#pragma unroll
          for (int r = 0; r < 16; ++r) m = fmaxf(m, s[t][r]);
        m = other_half_max(m) * a.c;
        if (__any(m > top + kSlack)) {
          const bool up = m > top;
          const float next = up ? m - weights_up<VF>() : ref;
          const float f = top == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(ref - next);
          if (up) top = m;
          ref = next;
          l *= f;
#pragma unroll
          for (int i = 0; i < DT / 32; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) o[i][r] *= f;
        }
        if (LATER && !all_see.value && values_odd(ks + KT * RS, sc + KT, KT, lane)) {
          for_each<DT / 32>([&](auto index) {
            constexpr int i = index.value;
            // one piece at a time, and its weights formed anew for each i: registers are short
            auto with_piece = [&](auto index, auto f) {
              constexpr int t = index.value;
              __builtin_amdgcn_sched_barrier(0);
              int first = 4 * half;
              __asm__ volatile("" : "+v"(first));
              float score[8], scale[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                score[j] = s[t / 2][8 * (t % 2) + j];
                __asm__ volatile("" : "+v"(score[j]));
                scale[j] = C8 ? sc[KT + 16 * t + (j < 4 ? 0 : 4) + first + j] : 1.0f;
              }
              const uint8_t* at = ks + v_base + ((4 * i) ^ v_swap) * 16 + 16 * t * RS;
              const u32x2 lo = read_transposed(at), hi = read_transposed(at + 8 * RS);
              f(score, scale, u32x4{lo.x, lo.y, hi.x, hi.y});
            };
            for_each<KT / 16>([&](auto index) {
              with_piece(index, [&](const float (&score)[8], const float (&scale)[8], u32x4 v) {
                float aside = 0.0f;                        // the sum has them once
                const Apart x = apart<two>(score, a.c, ref, scale, v, i == 0 ? l : aside);
                o[i] = mma32<VF>(x.v, x.w, o[i]);
                if constexpr (two) o[i] = mma32<VF>(x.v, x.w2, o[i]);
              });
            });
            f32x16 count;
#pragma unroll
            for (int r = 0; r < 16; ++r) count[r] = 0.0f;
            for_each<KT / 16>([&](auto index) {
              with_piece(index, [&](const float (&score)[8], const float (&scale)[8], u32x4 v) {
                const Counted x = counted(score, scale, v);
                count = mma32<VF>(x.odd, x.seen, count);
              });
            });
#pragma unroll
            for (int r = 0; r < 16; ++r) o[i][r] = add_counted(o[i][r], count[r]);
          });
        } else {
        u32x4 w[KT / 16], w2[two ? KT / 16 : 1];
#pragma unroll
        for (int t = 0; t < KT / 32; ++t) {
          float e[16];
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            e[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][r], a.c, -ref));
            l += e[r];
          }
          if constexpr (C8) {
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
              const f32x4 v = *reinterpret_cast<const f32x4*>(sc + KT + 32 * t + 2 * r + 4 * half);
#pragma unroll
              for (int j = 0; j < 4; ++j) e[r + j] *= v[j];
            }
          }
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float a0 = e[8 * u + 2 * j], a1 = e[8 * u + 2 * j + 1];
              if constexpr (two) {
                const Parts16 p = parts16<C8>(a0, a1);
                w[2 * t + u][j] = p.top;
                w2[2 * t + u][j] = p.rest;
              } else {
                w[2 * t + u][j] = pair16<VF>(a0, a1);
              }
            }
        }
#pragma unroll
        for (int t = 0; t < KT / 16; ++t)
#pragma unroll
          for (int i = 0; i < DT / 32; ++i) {
            const uint8_t* at = ks + v_base + ((4 * i) ^ v_swap) * 16 + 16 * t * RS;
            const u32x2 lo = read_transposed(at), hi = read_transposed(at + 8 * RS);
            o[i] = mma32<VF>(u32x4{lo.x, lo.y, hi.x, hi.y}, w[t], o[i]);
            if constexpr (two) o[i] = mma32<VF>(u32x4{lo.x, lo.y, hi.x, hi.y}, w2[t], o[i]);
          }
        }
      }
      if (more) {
        store_tile(buf ^ 1);
        gone = next_gone;
      }
      arrived();
      buf ^= 1;
    };
    // tiles that all tokens see whole, and those in which some stop, or all
    int key = p.k0;
    for (; key + KT <= least; key += KT) step(Index<1>{}, key);
    for (; key < p.k1; key += KT) step(Index<0>{}, key);
    l = other_half_sum(l);
    if (row < p.rows) {
      const int64_t at = out_row(a, p, row);
      if (half == 0) *reinterpret_cast<f32x2*>(a.part_m + 2 * at) = f32x2{ref, l};
      float* dst = a.part_o + at * a.kv.dim;
#pragma unroll
      for (int i = 0; i < DT / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; r += 4) {
          const int d = 32 * i + 2 * r + 4 * half;
          if (d < a.kv.dim)
            *reinterpret_cast<f32x4*>(dst + d) = f32x4{o[i][r], o[i][r + 1], o[i][r + 2], o[i][r + 3]};
        }
    }
  }

  // Up to 16 rows: bound by the stream of the cache.  The waves take 32 keys in
  // turn, each on its own: keys straight into registers as the operand that they
  // are, values through the wave's own part of shared memory, to be transposed.
  // The next 32 are on their way meanwhile, and the pages of those after them.  8
  // sequences of up to 32768, 64 heads: 160 us, 4.4 TB/s (a copy 5.0 read and
  // written); one workgroup to a CU does as well as two, so it is memory that they
  // wait for.  8-bit 106 us, 3.4 TB/s.
  static __device__ void few_rows(const AttnArgs& a, const Piece& p, uint8_t* smem) {
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, g = lane >> 4;
    constexpr int stride = 32 * kAttnWaves;
    constexpr int steps = DT / 32;                         // of 32 elements of a row
    constexpr int vloads = 32 / wave_keys;
    // which elements group g has in step i: 8 of each 32, of 8-bit rows 16 of each 64
    constexpr bool wide = C8 && DT % 64 == 0;
    constexpr int kloads = wide ? steps / 2 : steps;
    auto elem = [&](int i) { return wide ? 64 * (i / 2) + 16 * g + 8 * (i & 1) : 32 * i + 8 * g; };
    int key = p.k0 + 32 * wave;
    auto pages = find_pages<2>(a, p, key);
    int of_scale = scale_page(a, p, key + (lane & 31));
    u32x4 q[steps];
    {
      const uint8_t* at = query(a, p, col);
#pragma unroll
      for (int i = 0; i < steps; ++i) q[i] = query8(a, at, elem(i));
    }
    const int limit = p.causal ? min(p.k1, p.limit0 + min(col, p.rows - 1) / a.group) : p.k1;
    const int least = p.causal ? min(p.k1, p.limit0) : p.k1;
    f32x4 o[DT / 16];
#pragma unroll
    for (int i = 0; i < DT / 16; ++i) o[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    float top = -__builtin_inff(), ref = 0.0f, l = 0.0f;
    uint8_t* mine = smem + wave * few_wave;

    const int piece = lane % CH, key_in = lane / CH;
    uint32_t k_off[kloads], v_off[vloads];
#pragma unroll
    for (int i = 0; i < kloads; ++i) {
      const int d = elem(wide ? 2 * i : i);
      k_off[i] = d < a.kv.dim ? (uint32_t)col * (uint32_t)a.kv.token_stride + d * (C8 ? 1 : 2) : kNowhere;
    }
#pragma unroll
    for (int i = 0; i < vloads; ++i) {
      const int c = C8 ? piece : piece ^ swap_v(i * wave_keys + key_in);
      v_off[i] = c * CB < a.kv.dim
                     ? (uint32_t)((i * wave_keys + key_in) & 15) * (uint32_t)a.kv.token_stride + c * 16 : kNowhere;
    }
    struct Keys {
      u32x4 k[2][kloads];
      u32x4 v[C8 ? vloads : 1];
      float scale;
      uint32_t gone;
    };
    constexpr int loads = 2 * kloads + vloads;             // of a step, without scales
    auto load_keys = [&](int at, int buf, Keys& f) {       // values first: keys that are there say that they are, too
      const Run run[2] = {run_of(a, p, pages.at[0], at), run_of(a, p, pages.at[1], at + 16)};
#pragma unroll
      for (int i = 0; i < vloads; ++i) {
        const rsrc_t r = rows(a.kv.v, run[i * wave_keys / 16]);
        if constexpr (C8) f.v[i] = __builtin_amdgcn_raw_buffer_load_b128(r, v_off[i], 0, 0);
        else load_to_lds(r, mine + buf * few_step + i * wave_keys * RS, v_off[i]);
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const rsrc_t r = rows(a.kv.k, run[t]);
#pragma unroll
        for (int i = 0; i < kloads; ++i) {
          if constexpr (C8 && !wide) {
            const u32x2 d = __builtin_amdgcn_raw_buffer_load_b64(r, k_off[i], 0, 0);
            f.k[t][i] = u32x4{d.x, d.y, 0u, 0u};
          } else {
            f.k[t][i] = __builtin_amdgcn_raw_buffer_load_b128(r, k_off[i], 0, 0);
          }
        }
      }
      if constexpr (C8)
        f.scale = load_scale(a, p, lane < 32 ? a.kv.k_scales : a.kv.v_scales, of_scale, at + (lane & 31));
      f.gone = missing(pages);
    };

    Keys cur;
    if (key < p.k1) {
      check_pages(a, p, key, pages);
      load_keys(key, 0, cur);
      pages = find_pages<2>(a, p, key + stride);
      of_scale = scale_page(a, p, key + stride + (lane & 31));
    }
    for (int buf = 0; key < p.k1; key += stride, buf ^= C8 ? 0 : 1) {
      const uint32_t gone = cur.gone;
      uint8_t* vs = mine + buf * few_step;
      float* sc = reinterpret_cast<float*>(vs + 32 * RS);
      u32x4 k[2][steps];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < steps; ++i) {
          if constexpr (wide) {
            const u32x4 d = cur.k[t][i / 2];
            k[t][i] = i % 2 == 0 ? wide8<QF>(d.x, d.y) : wide8<QF>(d.z, d.w);
          } else if constexpr (C8) {
            k[t][i] = wide8<QF>(cur.k[t][i].x, cur.k[t][i].y);
          } else {
            k[t][i] = cur.k[t][i];
          }
        }
      if constexpr (C8) {
#pragma unroll
        for (int i = 0; i < vloads; ++i) {
          const int r = i * wave_keys + key_in;
          store8<VF>(vs, r, swap_v(r), piece, cur.v[i]);
        }
        sc[lane] = cur.scale;
      }
      const bool more = key + stride < p.k1;
      if (more) {
        check_pages(a, p, key + stride, pages);
        load_keys(key + stride, buf ^ 1, cur);
        pages = find_pages<2>(a, p, key + 2 * stride);
        of_scale = scale_page(a, p, key + 2 * stride + (lane & 31));
      }
      f32x4 s[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) s[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < steps; ++i)
#pragma unroll
        for (int t = 0; t < 2; ++t) s[t] = mma16<QF>(k[t][i], q[i], s[t]);
      compiler_barrier();
      if constexpr (!C8) {                                 // this step's values
        constexpr int wait_next = 0x0F70 | (loads & 15) | (loads >> 4) << 14;
        static_assert(loads < 64, "loads on their way that a wait can name");
        if (more) __builtin_amdgcn_s_waitcnt(wait_next);
        else __builtin_amdgcn_s_waitcnt(0x0F70);
        compiler_barrier();
      }
      if constexpr (C8) {
#pragma unroll
        for (int t = 0; t < 2; ++t) s[t] *= *reinterpret_cast<const f32x4*>(sc + 16 * t + 4 * g);
      }
      if (gone != 0 || key + 32 > least) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (key + 16 * t + 4 * g + r >= limit || (gone >> t & 1)) s[t][r] = -__builtin_inff();
      }
      float m = fmaxf(fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[0][2], s[0][3])),
                      fmaxf(fmaxf(s[1][0], s[1][1]), fmaxf(s[1][2], s[1][3])));
      m = other_half_max(other_row_max(m)) * a.c;
      if (__any(m > top + kSlack)) {
        const bool up = m > top;
        const float next = up ? m - weights_up<VF>() : ref;
        const float f = top == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(ref - next);
        if (up) top = m;
        ref = next;
        l *= f;
#pragma unroll
        for (int i = 0; i < DT / 16; ++i) o[i] *= f;
      }
      // rows 4g on and 16 after them, columns 4 * (lane % 4) on of each 16
      const int vk = 4 * g + col / 4, swap = ((lane & 3) / 2) ^ swap_v(vk);
      const uint8_t* at = vs + vk * RS + (lane & 1) * 8;
      if (LATER && p.causal && key + 32 > least && values_odd(vs, sc + 32, 32, lane)) {
        float score[8], scale[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          score[j] = s[j / 4][j % 4];
          scale[j] = C8 ? sc[32 + 16 * (j / 4) + 4 * g + j % 4] : 1.0f;
        }
#pragma unroll
        for (int i = 0; i < DT / 16; ++i) {
          __builtin_amdgcn_sched_barrier(0);
          float again = ref;
          __asm__ volatile("" : "+v"(again));
          const u32x2 lo = read_transposed(at + ((2 * i) ^ swap) * 16), hi = read_transposed(at + 16 * RS + ((2 * i) ^ swap) * 16);
          float aside = 0.0f;                              // the sum has them once
          const Apart x = apart<few_two>(score, a.c, again, scale, u32x4{lo.x, lo.y, hi.x, hi.y}, i == 0 ? l : aside);
          o[i] = mma16<VF>(x.v, x.w, o[i]);
          if constexpr (few_two) o[i] = mma16<VF>(x.v, x.w2, o[i]);
          const Counted y = counted(score, scale, u32x4{lo.x, lo.y, hi.x, hi.y});
          const f32x4 count = mma16<VF>(y.odd, y.seen, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
          for (int r = 0; r < 4; ++r) o[i][r] = add_counted(o[i][r], count[r]);
        }
      } else {
      f32x4 e[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          e[t][r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][r], a.c, -ref));
          l += e[t][r];
        }
        if constexpr (C8) e[t] *= *reinterpret_cast<const f32x4*>(sc + 32 + 16 * t + 4 * g);
      }
      u32x4 w, w2;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a0 = e[j / 2][j % 2 * 2], a1 = e[j / 2][j % 2 * 2 + 1];
        if constexpr (few_two) {
          const Parts16 p = parts16<C8>(a0, a1);
          w[j] = p.top;
          w2[j] = p.rest;
        } else {
          w[j] = pair16<VF>(a0, a1);
        }
      }
#pragma unroll
      for (int i = 0; i < DT / 16; ++i) {
        const u32x2 lo = read_transposed(at + ((2 * i) ^ swap) * 16), hi = read_transposed(at + 16 * RS + ((2 * i) ^ swap) * 16);
        o[i] = mma16<VF>(u32x4{lo.x, lo.y, hi.x, hi.y}, w, o[i]);
        if constexpr (few_two) o[i] = mma16<VF>(u32x4{lo.x, lo.y, hi.x, hi.y}, w2, o[i]);
      }
      }
      compiler_barrier();                                  // before the buffer is filled again
      if constexpr (!C8) __builtin_amdgcn_s_waitcnt(0xC07F);   // (lgkmcnt: loads to it keep no order with reads)
    }
    l = other_half_sum(other_row_sum(l));
    // the waves' sums, joined in shared memory
    __syncthreads();
    float* po = reinterpret_cast<float*>(smem);            // [wave][row][DT]
    float* pm = po + kAttnWaves * 16 * DT;                 // [wave][row][2]
#pragma unroll
    for (int i = 0; i < DT / 16; ++i)
      *reinterpret_cast<f32x4*>(po + (wave * 16 + col) * DT + 16 * i + 4 * g) = o[i];
    if (g == 0) *reinterpret_cast<f32x2*>(pm + 2 * (wave * 16 + col)) = f32x2{ref, l};
    __syncthreads();
    for (int i = tid; i < p.rows * (DT / 4); i += kAttnThreads) {
      const int row = i / (DT / 4), d = i % (DT / 4) * 4;
      f32x2 m[kAttnWaves];
      float most = -__builtin_inff();
#pragma unroll
      for (int w = 0; w < kAttnWaves; ++w) {
        m[w] = *reinterpret_cast<const f32x2*>(pm + 2 * (w * 16 + row));
        if (m[w].y != 0.0f) most = fmaxf(most, m[w].x);
      }
      f32x4 v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kAttnWaves; ++w) {
        if (m[w].y == 0.0f) continue;
        const float f = __builtin_amdgcn_exp2f(m[w].x - most);
        sum += f * m[w].y;
        v += f * *reinterpret_cast<const f32x4*>(po + (w * 16 + row) * DT + d);
      }
      const int64_t at = out_row(a, p, row);
      if (d == 0) *reinterpret_cast<f32x2*>(a.part_m + 2 * at) = f32x2{most == -__builtin_inff() ? 0.0f : most, sum};
      if (d < a.kv.dim) *reinterpret_cast<f32x4*>(a.part_o + at * a.kv.dim + d) = v;
    }
  }
};

// One range of keys of one head of the cache: of the prefix for a tile of all
// sequences' rows, or of one sequence's own tokens.  Workgroups go round the 8
// XCDs one by one; each XCD takes a run of pieces, those with the same keys
// next to each other, in its own L2.
template <int QF, bool C8, int DT, bool LATER>
__global__ __launch_bounds__(kAttnThreads, DT > 128 ? 1 : 2) void k_attention(AttnArgs a) {
  using G = Attn<QF, C8, DT, LATER>;
  __shared__ __align__(256) uint8_t smem[G::lds];
  Piece p;
  int b = blockIdx.x;
  const bool shared = b < a.prefix_blocks;
  const int total = shared ? a.prefix_blocks : a.own_blocks;
  if (!shared) b -= a.prefix_blocks;
  {
    const int per = total / 8, extra = total % 8, xcd = b % 8;
    b = xcd * per + min(xcd, extra) + b / 8;
  }
  const int kv = a.kv.kv_heads;
  if (shared) {
    const int tile = b % a.prefix_tiles;
    b /= a.prefix_tiles;
    p.part = b % a.prefix_splits;
    p.kh = b / a.prefix_splits;
    p.table = a.prefix_pages;
    p.k0 = p.part * a.prefix_chunk;
    p.k1 = min(a.prefix, p.k0 + a.prefix_chunk);
    p.rows = a.sequences * a.queries * a.group;
    p.row0 = tile * kTileRows;
    p.token0 = 0;
    p.limit0 = 0;
    p.causal = false;
  } else {
    const int tile = a.own_tiles - 1 - b % a.own_tiles;    // those that see most first
    b /= a.own_tiles;
    p.kh = b % kv;
    b /= kv;
    const int split = b % a.own_splits, seq = b / a.own_splits;
    const int length = ld_const(a.lengths, seq);
    const int most = max(min(length, a.capacity), 0);
    const int chunk = ((most + a.own_splits - 1) / a.own_splits + 127) / 128 * 128;
    p.part = a.prefix_splits + split;
    p.table = a.tables + seq * a.table_stride;
    p.k0 = min(most, split * chunk);
    p.k1 = min(most, p.k0 + chunk);
    p.rows = a.queries * a.group;
    p.row0 = tile * kTileRows;
    p.token0 = seq * a.queries;
    p.limit0 = length - a.queries + 1;
    p.causal = true;
    // what the tile's last token does not see, none of its tokens does (2 x 2048
    // tokens by themselves 554 us without this, 320 with it, 303 in this order of tiles)
    p.k1 = min(p.k1, p.limit0 + (min(p.row0 + kTileRows, p.rows) - 1) / a.group);
    if (p.k0 >= p.k1) {
      for (int i = p.row0 + threadIdx.x; i < min(p.rows, p.row0 + kTileRows); i += kAttnThreads)
        *reinterpret_cast<f32x2*>(a.part_m + 2 * G::out_row(a, p, i)) = f32x2{0.0f, 0.0f};
      return;
    }
  }
  if (p.rows <= kFewRows) G::few_rows(a, p, smem);
  else G::many_rows(a, p, smem);
}

// A row's ranges joined: a wave for each row, 4 elements a lane, so that
// kWave / LR ranges are read at once, and those of up to 4 rounds are on their
// way together.  Ranges that nothing was seen in are passed over.
template <int QF, int LR>
__global__ __launch_bounds__(kBlock) void k_attention_join(AttnArgs a) {
  constexpr int at_once = kWave / LR;
  const int lane = threadIdx.x & 63;
  const int row = blockIdx.x * kWavesPerBlock + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (row >= a.rows) return;
  const int token = row / a.heads, head = row % a.heads;
  const int parts = a.prefix_splits + a.own_splits;
  const f32x2* ml = reinterpret_cast<const f32x2*>(a.part_m) + row;
  const int d = lane % LR * 4, turn = lane / LR;
  const float* po = a.part_o + (int64_t)row * a.kv.dim + d;
  const int64_t part_stride = (int64_t)a.rows * a.kv.dim;
  const bool mine = d < a.kv.dim;
  f32x4 o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  float most = -__builtin_inff(), l = 0.0f;
  for (int s0 = 0; s0 < parts; s0 += kWave) {              // 64 ranges, one a lane
    f32x2 m = f32x2{0.0f, 0.0f};
    if (s0 + lane < parts) m = ml[(int64_t)(s0 + lane) * a.rows];
    float next = m.y != 0.0f ? m.x : -__builtin_inff();
#pragma unroll
    for (int i = 32; i > 0; i /= 2) next = fmaxf(next, __shfl_xor(next, i));
    next = fmaxf(next, most);
    if (next > most) {
      const float f = most == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(most - next);
      l *= f;
      o *= f;
      most = next;
    }
    const float w = m.y != 0.0f ? __builtin_amdgcn_exp2f(m.x - most) : 0.0f;
    float sum = m.y != 0.0f ? w * m.y : 0.0f;
#pragma unroll
    for (int i = 32; i > 0; i /= 2) sum += __shfl_xor(sum, i);
    l += sum;
    const uint64_t seen = __ballot(m.y != 0.0f);
    const int count = min(kWave, parts - s0);
    for (int s = 0; s < count; s += 4 * at_once) {
      f32x4 v[4];
      float f[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = min(s + u * at_once + turn, kWave - 1);
        f[u] = __shfl(w, k);
        v[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (s + u * at_once + turn < count && (seen >> k & 1) && mine)
          v[u] = *reinterpret_cast<const f32x4*>(po + (s0 + k) * part_stride);
        else f[u] = 0.0f;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) o += f[u] * v[u];
    }
  }
#pragma unroll
  for (int i = LR; i < kWave; i *= 2)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] += __shfl_xor(o[e], i);
  if (ld_const(a.lengths, token / a.queries) < 0) return;
  if (lane < LR && mine) {
    o *= l == 0.0f ? 0.0f : 1.0f / l;
    uint16_t* dst = static_cast<uint16_t*>(a.out) + token * a.out_stride + head * a.out_head + d;
    *reinterpret_cast<u32x2*>(dst) = u32x2{pair16<QF>(o[0], o[1]), pair16<QF>(o[2], o[3])};
  }
  // the logarithm of the sum, whose reference `most` is
  if (a.lse && lane == 0)
    a.lse[token * a.lse_stride + head] =
        l == 0.0f ? -__builtin_inff() : (most + __builtin_log2f(l)) * 0.69314718055994531f;
}

// ================================================================ host side

static int check_attention(const ar_attention_params* p) {
  if (!p) return AR_EINVAL;
  if (p->reserved != 0 || p->sequences < 0 || p->queries < 1 || p->heads < 1 || p->prefix < 0 || p->max_pages < 0)
    return AR_EINVAL;
  if (p->format != AR_BF16 && p->format != AR_F16) return AR_EINVAL;
  if (!(p->scale > 0.0f) || p->scale > 0x1p127f) return AR_EINVAL;   // times log2(e), finite
  int rc = check_cache(&p->cache);
  if (rc) return rc;
  if (p->heads % p->cache.kv_heads != 0) return AR_EINVAL;
  if (p->cache.format != AR_E4M3_ROW && p->cache.format != p->format) return AR_EINVAL;
  const int64_t most = int64_t(1) << 30;
  if (p->sequences > most || p->prefix > most || p->max_pages > most) return AR_ESIZE;
  if (p->max_pages * p->cache.page > most) return AR_ESIZE;
  // rows of all parts stay within 31 bits
  if ((double)p->sequences * p->queries * p->heads >= (double)(1 << 26)) return AR_ESIZE;
  return AR_OK;
}

static int check_attention_rows(const ar_attention_params* p) {
  const int64_t most = int64_t(1) << 36;                   // times 2^26 rows within 2^62
  const int64_t tokens = p->sequences * p->queries;
  if (!p->q || !p->out || !p->lengths) return AR_EINVAL;
  if (p->max_pages > 0 && (!p->pages || (p->sequences > 1 && p->pages_stride < p->max_pages))) return AR_EINVAL;
  if (p->prefix > 0 && !p->prefix_pages) return AR_EINVAL;
  if (p->q_stride < 0 || p->q_head_stride < 0 || p->out_stride < 0 || p->out_head_stride < 0 || p->lse_stride < 0)
    return AR_EINVAL;
  if (p->q_stride >= most || p->q_head_stride >= most || p->out_stride >= most || p->out_head_stride >= most ||
      p->lse_stride >= most || p->pages_stride >= (int64_t(1) << 30))
    return AR_ESIZE;
  // outputs may not overlap each other
  const int64_t dim = p->cache.dim, heads = p->heads;
  auto apart = [&](int64_t ts, int64_t hs, int64_t width) {
    if (heads > 1 && hs < width) return false;
    if (tokens <= 1) return true;
    return ts >= (heads - 1) * hs + width || (ts >= width && hs >= (tokens - 1) * ts + width);
  };
  if (!apart(p->out_stride, p->out_head_stride, dim)) return AR_EINVAL;
  if (p->lse && tokens > 1 && p->lse_stride < heads) return AR_EINVAL;
  if (!aligned(p->q, 16) || p->q_stride % 8 || p->q_head_stride % 8 || !aligned(p->out, 16) || p->out_stride % 8 ||
      p->out_head_stride % 8 || !aligned(p->lengths, 4) || !aligned(p->pages, 4) || !aligned(p->prefix_pages, 4) ||
      !aligned(p->lse, 4))
    return AR_EALIGN;
  return AR_OK;
}

// How the keys are split.
struct AttnPlan {
  int32_t prefix_splits, prefix_chunk, prefix_tiles, own_splits, own_tiles;
};

static int64_t row_tiles(int64_t rows) { return rows <= kFewRows ? 1 : ceil_div64(rows, kTileRows); }
static int64_t step_keys(int64_t rows) { return rows <= kFewRows ? 128 : 64; }
static int64_t most_places(const ar_attention_params* p) {
  return p->cache.dim <= 64 ? 1024 : (p->cache.dim <= 128 ? 512 : 256);
}

// Pieces of keys.  A piece costs a step for each 64 keys of a tile of many rows,
// or for each 128 that the waves of few rows take together; all are made as
// long as fills the chip's places for workgroups once: four to a CU where heads are of
// up to 64, two up to 128, else one, by registers and shared memory.  Short pieces
// are made twice as long: their rows' way through memory to the join counts more.
// 128 x 64 heads over 32768, bf16: 168 us with 512 pieces, 179 with 1024; heads of 64
// 101 to 105 and 103; of 256 241 and, with 256 pieces, 226; 16 x 64 heads over 8192 27 with
// 512, 23 with 256.  Where no sequence's own tokens are split, the prefix has the
// places that they leave, if its pieces grow by a third at most for it: 37 x 2 tokens,
// prefix 4999, own 777, heads of 96, 28.4 us so, 33.0 with 536 pieces; own 400 26.9 and
// 27.8.  (Up to 256 pieces there are places for all: 20 x 2 tokens, own 777, 25.3 with
// 288 pieces in 512 places, 28.6 with 256.  Pieces of split ones vary with the lengths:
// 8 sequences of up to 32768, 161 with 520, 169 with 512.)  Own tokens count with all
// that the table has room for, which may be far more than there are: the prefix's
// pieces are therefore at most twice as long as by itself, or 8 steps.  16 x 64 heads,
// prefix 8192, own 500, a table for 512 tokens 26 us, for 32768 27, 98 without that
// limit; 128 x 64 heads, prefix 32768, 8-bit, own 200, a table for 32768 245 and 910.
// Own pieces are as many for every sequence: one of 32768 tokens among 127 of 200 is
// 335 us, 31 by itself.
static AttnPlan plan_attention(const ar_attention_params* p) {
  AttnPlan s{};
  const int64_t kv = p->cache.kv_heads, group = p->heads / kv;
  const int64_t rows = p->sequences * p->queries * group, own_rows = p->queries * group;
  const int64_t capacity = p->max_pages * p->cache.page;
  s.prefix_tiles = (int32_t)row_tiles(rows);
  s.own_tiles = (int32_t)row_tiles(own_rows);
  const int64_t shared = kv * s.prefix_tiles * ceil_div64(p->prefix, step_keys(rows));
  const int64_t own = p->sequences * kv * s.own_tiles * ceil_div64(capacity, step_keys(own_rows));
  const int64_t places = most_places(p);
  auto piece = [&](int64_t all) {
    const int64_t n = ceil_div64(all, places);
    return n < 6 ? ceil_div64(all, 256) : n;
  };
  const int64_t steps = piece(shared + own);
  if (capacity > 0) s.own_splits = (int32_t)ceil_div64(capacity, steps * step_keys(own_rows));
  if (p->prefix > 0) {
    const int64_t alone = piece(shared) < 4 ? 8 : 2 * piece(shared);
    int64_t n = ceil_div64(p->prefix, (steps < alone ? steps : alone) * step_keys(rows));
    const int64_t room = (places - p->sequences * kv * s.own_tiles * s.own_splits) / (kv * s.prefix_tiles);
    if (s.own_splits <= 1 && room < n && 4 * room >= 3 * n) n = room;
    s.prefix_chunk = (int32_t)(ceil_div64(ceil_div64(p->prefix, n), 64) * 64);
    s.prefix_splits = (int32_t)ceil_div64(p->prefix, s.prefix_chunk);
  }
  return s;
}

// A work buffer that does for the plan, and for that of every batch with fewer
// sequences, a shorter prefix or fewer pages.  A plan's steps go into `places` times
// what a workgroup takes, so that
//     sequences * kv_heads * own_tiles * own_splits < places + sequences * kv_heads * own_tiles,
// and the prefix's splits in the same way; times the rows of a tile neither bound falls
// as a size grows.  Few keys have no more pieces than steps.
static int64_t attention_bytes(const ar_attention_params* p) {
  const int64_t kv = p->cache.kv_heads, own_rows = p->queries * (p->heads / kv);
  const int64_t rows = p->sequences * p->queries * p->heads, shared_rows = p->sequences * own_rows;
  const int64_t capacity = p->max_pages * p->cache.page, places = most_places(p);
  const int64_t own_step = ceil_div64(capacity, step_keys(own_rows)), prefix_step = ceil_div64(p->prefix, step_keys(kTileRows));
  const int64_t tile = shared_rows < kTileRows ? shared_rows : kTileRows;
  auto least = [](int64_t a, int64_t b) { return a < b ? a : b; };
  int64_t n = 0;                                           // rows of all parts
  if (capacity > 0) n += least(own_step * rows, ceil_div64(places * own_rows, row_tiles(own_rows)) + rows);
  if (p->prefix > 0) n += least(prefix_step * rows, places * tile + rows);
  return (n * (p->cache.dim + 2) * 4 + 255) / 256 * 256;
}

template <int QF, bool C8, int DT>
static hipError_t launch_parts(const AttnArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)(a.prefix_blocks + a.own_blocks)), block(kAttnThreads);
  return a.queries > 1 ? launch(k_attention<QF, C8, DT, true>, grid, block, s, a)
                       : launch(k_attention<QF, C8, DT, false>, grid, block, s, a);
}
template <int QF, bool C8>
static hipError_t launch_parts_dim(const AttnArgs& a, hipStream_t s) {
  if (a.kv.dim <= 64) return launch_parts<QF, C8, 64>(a, s);
  if (a.kv.dim <= 96) return launch_parts<QF, C8, 96>(a, s);
  if (a.kv.dim <= 128) return launch_parts<QF, C8, 128>(a, s);
  if (a.kv.dim <= 192) return launch_parts<QF, C8, 192>(a, s);
  return launch_parts<QF, C8, 256>(a, s);
}
template <int QF>
static hipError_t launch_join(const AttnArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)ceil_div64(a.rows, kWavesPerBlock)), block(kBlock);
  if (a.kv.dim <= 64) return launch(k_attention_join<QF, 16>, grid, block, s, a);
  if (a.kv.dim <= 128) return launch(k_attention_join<QF, 32>, grid, block, s, a);
  return launch(k_attention_join<QF, 64>, grid, block, s, a);
}
template <int QF>
static hipError_t launch_attention(const AttnArgs& a, bool c8, hipStream_t s) {
  hipError_t e = hipSuccess;
  if (a.prefix_blocks + a.own_blocks > 0)
    e = c8 ? launch_parts_dim<QF, true>(a, s) : launch_parts_dim<QF, false>(a, s);
  return e == hipSuccess ? launch_join<QF>(a, s) : e;
}

}  // namespace ar

using namespace ar;

extern "C" {

int64_t ar_prefix_attention_work_bytes(const ar_attention_params* p) {
  const int rc = check_attention(p);
  if (rc) return rc;
  if (p->sequences == 0) return 0;
  return attention_bytes(p);
}

int ar_prefix_attention(const ar_attention_params* p, void* work, int64_t work_bytes, void* stream) {
  int rc = check_attention(p);
  if (rc) return rc;
  if (p->sequences == 0) return AR_OK;
  rc = check_attention_rows(p);
  if (rc) return rc;
  if (p->prefix > 0 || p->max_pages > 0) {
    rc = check_cache_rows(&p->cache);
    if (rc) return rc;
  }
  const AttnPlan plan = plan_attention(p);
  const int64_t bytes = attention_bytes(p);
  if (bytes > 0) {
    if (!work) return AR_EINVAL;
    if (!aligned(work, 256)) return AR_EALIGN;
    if (work_bytes < bytes) return AR_ESIZE;
  }
  AttnArgs a{};
  const int64_t kv = p->cache.kv_heads;
  a.kv = cache_view(&p->cache);
  a.q = static_cast<const uint8_t*>(p->q);
  a.q_stride = p->q_stride;
  a.q_head = p->q_head_stride;
  a.out = p->out;
  a.out_stride = p->out_stride;
  a.out_head = p->out_head_stride;
  a.lse = p->lse;
  a.lse_stride = p->lse_stride;
  a.prefix_pages = p->prefix_pages;
  a.lengths = p->lengths;
  a.tables = p->pages;
  a.table_stride = p->pages_stride;
  a.c = (float)((double)p->scale * 1.4426950408889634);
  a.prefix = (int32_t)p->prefix;
  a.capacity = (int32_t)(p->max_pages * p->cache.page);
  a.sequences = (int32_t)p->sequences;
  a.queries = p->queries;
  a.heads = p->heads;
  a.group = (int32_t)(p->heads / kv);
  a.rows = (int32_t)(p->sequences * p->queries * p->heads);
  a.prefix_splits = plan.prefix_splits;
  a.prefix_chunk = plan.prefix_chunk;
  a.prefix_tiles = plan.prefix_tiles;
  a.own_splits = plan.own_splits;
  a.own_tiles = plan.own_tiles;
  const int64_t pb = kv * plan.prefix_tiles * plan.prefix_splits;
  const int64_t ob = p->sequences * kv * plan.own_tiles * plan.own_splits;
  if (pb + ob > most_blocks(kAttnThreads)) return AR_ESIZE;
  a.prefix_blocks = (int32_t)pb;
  a.own_blocks = (int32_t)ob;
  const int64_t parts = plan.prefix_splits + plan.own_splits;
  a.part_o = static_cast<float*>(work);
  a.part_m = a.part_o + parts * a.rows * p->cache.dim;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool c8 = p->cache.format == AR_E4M3_ROW;
  return map_hip(p->format == AR_BF16 ? launch_attention<AR_BF16>(a, c8, s) : launch_attention<AR_F16>(a, c8, s));
}

}  // extern "C"
