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

// ---------------------------------------------------------- many tokens ---
//
// Bound by the matrix cores.  A workgroup holds BN outputs by BM tokens; K
// goes by in steps of 128 elements (64 for bf16 inputs), three steps' codes in
// shared memory: while one is multiplied the next has arrived and the one
// after is on its way, loaded straight into shared memory, and one barrier a
// step is enough.  Rows lie there as they come, 16-byte pieces permuted by the
// row so that the lanes that read at once meet different banks; the loads
// apply the permutation to their addresses.  Scales come 512 elements at a
// time, one row a thread.

// 16 bytes a lane from the buffer straight into shared memory, at `lds` (the
// wave's own address) + 16 * lane.
__device__ __forceinline__ void load_to_lds(rsrc_t r, uint8_t* lds, uint32_t lane_off, uint32_t off) {
  typedef __attribute__((address_space(3))) void lds_void;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void*)lds, 16, lane_off, off, 0, 0);
}

template <int XF>
struct TileShape {
  static constexpr int BK = XF == AR_BF16 ? 64 : 128;      // elements of K a step
  static constexpr int XB = XF == AR_E2M1_MX ? 64 : 128;   // bytes of an x row a step
  static constexpr int WB = BK / 2;                        // bytes of a weight row
  static constexpr int XC = XB / 16, WC = WB / 16;         // 16-byte pieces
  static constexpr int steps_scales = 512 / BK;            // steps that share 16 scales a row
};

// Where piece `c` of row `r` lies among the row's C pieces: 8 rows that are
// read together cover every 16-byte column of 128 bytes.
template <int C>
__device__ __forceinline__ int place(int r, int c) {
  if constexpr (C == 8) return c ^ (r & 7);
  else if constexpr (C == 4) return c ^ ((r >> 1) & 3);
  else return c ^ ((r >> 2) & 1);
}

__device__ __forceinline__ void barrier_only() {
  compiler_barrier();
  __builtin_amdgcn_s_barrier();
  compiler_barrier();
}

template <int XF_, int YF_, int BM_, int BN_, int WM_, int WN_>
struct Tile {
  static constexpr int XF = XF_, YF = YF_, BM = BM_, BN = BN_, WM = WM_, WN = WN_;
  using T = TileShape<XF>;
  static constexpr int waves = (BM / WM) * (BN / WN);
  static constexpr int threads = waves * kWave;
  static constexpr int xbytes = BM * T::XB, wbytes = BN * T::WB;
  static constexpr int stage = xbytes + wbytes;
  static constexpr int nx = xbytes / 16 / threads, nw = wbytes / 16 / threads;   // loads a thread
  static constexpr int scales = (BM + BN) * 16;
  static constexpr int lds = 3 * stage + 2 * scales;
  static_assert(nx >= 1 && nw >= 1 && BM + BN == threads, "one row of scales a thread");
};

template <class G>
__global__ __launch_bounds__(G::threads) void k_mx_linear_tiles(MxLinArgs a) {
  using T = typename G::T;
  constexpr int XF = G::XF, YF = G::YF, BM = G::BM, BN = G::BN, WM = G::WM, WN = G::WN;
  constexpr int TI = WN / 16, TJ = WM / 16;                // matrix tiles of a wave
  __shared__ __align__(256) uint8_t smem[G::lds];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int wi = wave % (BN / WN), wj = wave / (BN / WN);

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
  const rsrc_t xr = make_rsrc(xbase, 0x7FFFFFFFu), wr = make_rsrc(wbase, 0x7FFFFFFFu);
  const int mlast = a.M - 1 - m0, nlast = a.N - 1 - n0;    // rows past the end read the last one

  // this thread's pieces of a step: source offsets at step 0
  uint32_t xo[G::nx], wo[G::nw];
#pragma unroll
  for (int i = 0; i < G::nx; ++i) {
    const int at = i * G::threads + tid, row = at / T::XC;
    xo[i] = (uint32_t)min(row, mlast) * (uint32_t)a.x_stride + place<T::XC>(row, at % T::XC) * 16;
  }
#pragma unroll
  for (int i = 0; i < G::nw; ++i) {
    const int at = i * G::threads + tid, row = at / T::WC;
    wo[i] = (uint32_t)min(row, nlast) * (uint32_t)a.w_stride + place<T::WC>(row, at % T::WC) * 16;
  }
  auto load_step = [&](int k, int buf) {
    uint8_t* at = smem + buf * G::stage + wave * 1024;
#pragma unroll
    for (int i = 0; i < G::nx; ++i)
      load_to_lds(xr, at + i * G::threads * 16, xo[i], (uint32_t)k * T::XB);
#pragma unroll
    for (int i = 0; i < G::nw; ++i)
      load_to_lds(wr, at + G::xbytes + i * G::threads * 16, wo[i], (uint32_t)k * T::WB);
  };
  // a step that K ends in: zeros past it
  auto load_tail = [&](int k, int buf) {
    uint8_t* at = smem + buf * G::stage + tid * 16;
#pragma unroll
    for (int i = 0; i < G::nx; ++i) {
      const int slot = i * G::threads + tid, row = slot / T::XC;
      const int first = k * T::XB + place<T::XC>(row, slot % T::XC) * 16;       // byte of the row
      const int end = XF == AR_BF16 ? 2 * a.K : (XF == AR_E4M3_ROW ? a.K : a.nb * (XF == AR_E2M1_MX ? 16 : 32));
      u32x4 v = u32x4{0u, 0u, 0u, 0u};
      if (first < end) v = keep_bytes(ldg16(xbase + xo[i] + k * T::XB), end - first);
      *reinterpret_cast<u32x4*>(at + i * G::threads * 16) = v;
    }
#pragma unroll
    for (int i = 0; i < G::nw; ++i) {
      const int slot = i * G::threads + tid, row = slot / T::WC;
      const int first = k * T::WB + place<T::WC>(row, slot % T::WC) * 16;
      u32x4 v = u32x4{0u, 0u, 0u, 0u};
      if (first < a.nb * 16) v = ldg16(wbase + wo[i] + k * T::WB);
      *reinterpret_cast<u32x4*>(at + G::xbytes + i * G::threads * 16) = v;
    }
  };
  // scales: thread t holds weight row t, or token t - BN
  const bool mine_w = tid < BN;
  const bool no_scale = !mine_w && !is_mx_format(XF);
  const uint8_t* wsafe = a.ws + r * a.ws_rank + n0 * a.ws_stride;
  const uint8_t* srow = mine_w ? a.ws + r * a.ws_rank + (n0 + min(tid, nlast)) * a.ws_stride
                               : a.xs + r * a.xs_rank + (m0 + min(tid - BN, mlast)) * a.xs_stride;
  // 16 scales from step k on, raw; the last dword again where the row has ended
  const int slast = (a.nb - 1) & ~3;
  auto load_scales = [&](int k) -> u32x4 {
    const int blk = k * (T::BK / 32);
    u32x4 v;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      v[q] = *reinterpret_cast<const uint32_t*>((no_scale ? wsafe : srow) + min(blk + 4 * q, slast));
    return v;
  };
  // into shared memory, with 1 for every block past the end
  auto put_scales = [&](int k, u32x4 v) {
    const int left = a.nb - k * (T::BK / 32);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int n = no_scale ? 0 : left - 4 * q;
      const uint32_t keep = n >= 4 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << (8 * n)) - 1u);
      v[q] = (v[q] & keep) | (0x7F7F7F7Fu & ~keep);
    }
    *reinterpret_cast<u32x4*>(smem + 3 * G::stage + (k / T::steps_scales & 1) * G::scales + tid * 16) = v;
  };

  f32x4 acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  auto compute = [&](int k, int buf) {
    const uint8_t* xs = smem + buf * G::stage;
    const uint8_t* ws = xs + G::xbytes;
    const int ss = k / T::steps_scales;
    const uint8_t* sc = smem + 3 * G::stage + (ss & 1) * G::scales + (k % T::steps_scales) * (T::BK / 32);
    if constexpr (XF == AR_BF16) {
      // group g takes elements 16g .. 16g + 15, 8 in each of two instructions
      u32x4 x[TJ][2];
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const int row = wj * WM + j * 16 + c;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          x[j][h] = *reinterpret_cast<const u32x4*>(xs + row * T::XB + place<T::XC>(row, 2 * g + h) * 16);
      }
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        const int row = wi * WN + i * 16 + c;
        const u32x2 w = *reinterpret_cast<const u32x2*>(ws + row * T::WB + place<T::WC>(row, g >> 1) * 16 +
                                                        (g & 1) * 8);
        const float scale = __uint_as_float((uint32_t)sc[row * 16 + (g >> 1)] << 23);
        const bf16x8 w0 = weights_bf16(w.x, scale), w1 = weights_bf16(w.y, scale);
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w0, __builtin_bit_cast(bf16x8, x[j][0]),
                                                              acc[i][j], 0, 0, 0);
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w1, __builtin_bit_cast(bf16x8, x[j][1]),
                                                              acc[i][j], 0, 0, 0);
        }
      }
    } else {
      constexpr u32x4 none = u32x4{0u, 0u, 0u, 0u};
      constexpr int xcode = XF == AR_E2M1_MX ? 4 : 0;
      i32x8 x[TJ];
      int xsc[TJ];
#pragma unroll
      for (int j = 0; j < TJ; ++j) {
        const int row = wj * WM + j * 16 + c;
        if constexpr (XF == AR_E2M1_MX) {
          x[j] = operand(*reinterpret_cast<const u32x4*>(xs + row * T::XB + place<T::XC>(row, g) * 16), none);
        } else {
          x[j] = operand(*reinterpret_cast<const u32x4*>(xs + row * T::XB + place<T::XC>(row, g) * 16),
                         *reinterpret_cast<const u32x4*>(xs + row * T::XB + place<T::XC>(row, 4 + g) * 16));
        }
        xsc[j] = XF == AR_E4M3_ROW ? 127 : (int)sc[(BN + row) * 16 + g];
      }
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        const int row = wi * WN + i * 16 + c;
        const i32x8 w =
            operand(*reinterpret_cast<const u32x4*>(ws + row * T::WB + place<T::WC>(row, g) * 16), none);
        const int wsc = (int)sc[row * 16 + g];
#pragma unroll
        for (int j = 0; j < TJ; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x[j], acc[i][j], 4, xcode, 0, wsc,
                                                                       0, xsc[j]);
      }
    }
  };

  // whole steps, then maybe one that K ends in
  const int full = (is_mx_format(XF) ? a.nb * 32 : a.K) / T::BK;
  const int steps = (a.nb * 32 + T::BK - 1) / T::BK;
  if (full > 0) load_step(0, 0);
  if (full > 1) load_step(1, 1);
  if (steps > 0) put_scales(0, load_scales(0));
  u32x4 next = u32x4{0u, 0u, 0u, 0u};
  int buf = 0;
  for (int k = 0; k < full; ++k) {
    // step k has arrived when at most one step's loads are still on their way
    // (the scales' loads, where there are some, only make the wait longer), and
    // this wave's own scales are written
    if (k + 1 < full) __builtin_amdgcn_s_waitcnt(0x0070 | (G::nx + G::nw));
    else __builtin_amdgcn_s_waitcnt(0x0070);
    barrier_only();
    int into = buf + 2;
    if (into >= 3) into -= 3;
    if (k + 2 < full) load_step(k + 2, into);
    const int ks = k % T::steps_scales;
    if (ks == 0 && k + T::steps_scales < steps) next = load_scales(k + T::steps_scales);
    compute(k, buf);
    if (ks == T::steps_scales - 1 && k + 1 < steps) put_scales(k + 1, next);
    if (++buf == 3) buf = 0;
  }
  if (steps > full) {
    __syncthreads();
    load_tail(full, buf);
    __syncthreads();
    compute(full, buf);
  }
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    const int m = m0 + wj * WM + j * 16 + c;
    if (m >= a.M) continue;
    float scale = 1.0f;
    if constexpr (XF == AR_E4M3_ROW) {
      if (a.K > 0) scale = *reinterpret_cast<const float*>(a.xs + r * a.xs_rank + m * a.xs_stride);
    }
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int n = n0 + wi * WN + i * 16 + 4 * g;
      f32x4 v = acc[i][j];
      if constexpr (XF == AR_E4M3_ROW) v *= scale;
      if (n < a.N) store_out4<YF>(a.y, r * a.y_rank + m * a.y_stride + n, n, a.N, a.vec != 0, v);
    }
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

template <int XF, int YF, int BM, int BN, int WM, int WN>
static hipError_t launch_tiles(const MxLinArgs& a0, int nranks, hipStream_t s) {
  MxLinArgs a = a0;
  a.n_groups = (a.N + BN - 1) / BN;
  a.m_groups = (a.M + BM - 1) / BM;
  using G = Tile<XF, YF, BM, BN, WM, WN>;
  return launch(k_mx_linear_tiles<G>, dim3((unsigned)((int64_t)nranks * a.n_groups * a.m_groups)),
                dim3(G::threads), s, a);
}

template <int XF, int YF>
static hipError_t launch_linear(const MxLinArgs& a, int nranks, hipStream_t s) {
  // the tile kernels' offsets inside a tile are 31 bits
  if (a.M > 64 && a.x_stride < (1 << 23) && a.w_stride < (1 << 23)) {
    const int64_t big = (int64_t)((a.N + 255) / 256) * ((a.M + 255) / 256) * nranks;
    if (big >= 256) return launch_tiles<XF, YF, 256, 256, 64, 128>(a, nranks, s);
    return launch_tiles<XF, YF, 128, 128, 64, 64>(a, nranks, s);
  }
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
