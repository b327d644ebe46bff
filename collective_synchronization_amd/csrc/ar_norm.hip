// ar_norm.hip -- residual addition and root-mean-square norm of rows, alone
// and in the receive side of the one-shot all-reduce (gfx950).
//
//     h = residual + x,  r = 1 / sqrt(sum(h^2) / hidden + eps),
//     v = (h * r) * gamma;  residual_out = round(h);  y = v in y's format.
//
// h is binary32 and not rounded before the norm, the sum and r are binary64; how
// v is rounded goes by the format (products8 below).
//
// What bounds it: for many rows the memory system (x and the residual read
// once, both outputs written once; a row stays in registers between the sum
// and the scaling): 16384 x 8192, bf16, to 8-bit blocks 164 us, 5.8 TB/s, to
// bf16 180 us, 6.0 TB/s, where a plain copy reaches 5.1.  For few rows the launch
// and one trip to memory: one row of 4096 2.9 us.  One
// workgroup a row: 8 consecutive elements a thread and step, so a wave reads
// 1 KiB of a 16-bit row in one instruction, and the 4 lanes of an aligned
// group hold one 32-element block of the MX formats.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include <type_traits>

#include "../../include/ar.h"
#include "ar_host.h"
#include "ar_rows.h"
#include "../../include/ar_protocols.h"

namespace ar {

// Threads a row at most: 16384 rows of 8192, bf16 to 8-bit blocks, took 164 us
// with 512 threads and 2 chunks each, 179 with 1024 and 1, 173 with 256 and 4.
constexpr int kNormThreads = 512;
constexpr int kNormChunks = 8;       // chunks a thread at most
static_assert(kNormThreads * kNormChunks * 8 == AR_NORM_MAX_HIDDEN, "the longest row");

struct NormArgs {
  const void* x;
  int64_t x_stride;
  const void* gamma;                 // null: ones
  const void* res;                   // null: no residual
  int64_t res_stride;
  void* h;                           // null: not written
  int64_t h_stride;
  void* y;
  int64_t y_stride;
  void* scales;
  int64_t scale_stride;
  int64_t hidden;
  float eps;
  double inv_hidden;
};

// The waves' partial sums or maxima; a second array so that the maximum's
// writes need not wait for the sum's readers.
struct NormShared {
  double sum[kNormThreads / kWave];
  uint32_t max[kNormThreads / kWave];
};

__device__ __forceinline__ int64_t chunk_first(int i) {
  return ((int64_t)i * blockDim.x + threadIdx.x) * 8;
}

// Gamma is loaded beside the rows, before the sum: one trip to memory for all
// inputs, which is what bounds a single row.  Beyond two chunks a thread the
// registers are better spent on more rows in flight; gamma then comes, from
// the L2, when it is used.
constexpr bool gamma_first(int ni) { return ni <= 2; }

template <int FX, int NI>
struct Gamma {
  Raw<FX> raw[gamma_first(NI) ? NI : 1];
  rsrc_t row;
  __device__ __forceinline__ Gamma(const NormArgs& a) : row(raw_row(a.gamma, a.hidden, sizeof(typename Elem<FX>::type))) {
    if constexpr (gamma_first(NI)) {
#pragma unroll
      for (int i = 0; i < NI; ++i) raw[i] = load_raw<FX>(row, chunk_first(i));
    }
  }
  __device__ __forceinline__ void get(const NormArgs& a, int i, float (&g)[8]) const {
    if (!a.gamma) {
#pragma unroll
      for (int k = 0; k < 8; ++k) g[k] = 1.0f;
    } else if constexpr (gamma_first(NI)) {
      values<FX>(raw[i], a.hidden, chunk_first(i), g);
    } else {
      values<FX>(load_raw<FX>(row, chunk_first(i)), a.hidden, chunk_first(i), g);
    }
  }
};

// 1 / sqrt(x) for x >= 0, right to 2^-50 over all of binary64: the root
// instruction on x times an even power of two, in [1/2, 2), then one step of
// the third order.  0, infinities and NaN give inf, 0 and NaN.
__device__ __forceinline__ double reciprocal_root(double x) {
  const int e = __builtin_amdgcn_frexp_exp(x) & ~1;
  const double xs = __builtin_ldexp(x, -e);
  const double r = (double)__builtin_amdgcn_rsqf((float)xs);
  const double t = __builtin_fma(-xs * r, r, 1.0);
  const double better = __builtin_fma(r * t, __builtin_fma(0.375, t, 0.5), r);
  return __builtin_ldexp(x > 0.0 && x < __builtin_inf() ? better : r, -(e >> 1));
}

// The row's factor, in scalar registers: r, and r in two binary32 parts with room
// for a product's rounding error, unless the row is not an ordinary one (values
// below 2^-100 with eps 0, or above 2^100).
struct Root {
  double r;
  float hi, lo;
  bool ordinary;
  __device__ __forceinline__ explicit Root(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);    // the same in all lanes
    const uint32_t low = __builtin_amdgcn_readfirstlane((uint32_t)u);
    const uint32_t high = __builtin_amdgcn_readfirstlane((uint32_t)(u >> 32));
    r = __builtin_bit_cast(double, (uint64_t)high << 32 | low);
    hi = (float)r;
    lo = (float)(r - (double)hi);
    ordinary = (high >> 20) - (1023u - 100u) < 200u;       // 2^-100 <= r < 2^100
  }
};

// a * r * b = q + c, for products above 2^-100, below which an error may be less
// than binary32 holds.
struct Product {
  float p, q, c;
  __device__ __forceinline__ Product(float a, const Root& r, float b) : p(a * r.hi), q(p * b) {
    const float e = __builtin_fmaf(a, r.lo, __builtin_fmaf(a, r.hi, -p));
    c = __builtin_fmaf(e, b, __builtin_fmaf(p, b, -q));
  }
  // Right to binary32's last bit; an infinite q, whose c is as infinite the other
  // way, stays.
  __device__ __forceinline__ float nearest() const {
    return q + __builtin_amdgcn_fmed3f(c, -0x1.fffffep127f, 0x1.fffffep127f);
  }
  // Towards zero with the last bit set where that is not exact.
  __device__ __forceinline__ float odd() const {
    const float t = q + c, d = c - (t - q);                // what t lacks
    const bool above = (int)(__float_as_uint(d) ^ __float_as_uint(t)) < 0;
    return d == 0.0f ? t : __uint_as_float((__float_as_uint(t) - (above ? 1u : 0u)) | 1u);
  }
};

// a * r * b in binary64, to binary32: to nearest, or as odd() does.
template <bool ODD>
__device__ __forceinline__ float product64(float a, double r, float b) {
  __asm__("" : "+v"(a));                                   // the sum's conversions are not held for it
  const double d = (double)a * r * (double)b;
  const float f = (float)d;
  if constexpr (!ODD) return f;
  const double back = (double)f;
  if (!(back < d || back > d) || abs_bits(f) >= kInfBits) return f;
  return __uint_as_float((__float_as_uint(f) - (__builtin_fabs(back) > __builtin_fabs(d) ? 1u : 0u)) | 1u);
}

// h = (h * r) * g.  For a 16-bit type, whose own rounding is 2^13 times as large or
// more, two plain products, off by at most 3 * 2^-24 (r.hi's error among them); the
// exact ones cost 1000 x 4100 fp16 8.1 us instead of 7.6.  Otherwise right to
// binary32's last bit, unless h * r or the result is below 2^-100.  All in binary64,
// 16384 x 8192 to 8 bits takes 188 us instead of 165: about 45 instructions an
// element are what the vector units do in the memory's time.
template <int FY>
__device__ __forceinline__ void products8(float (&h)[8], const Root& r, const float (&g)[8]) {
  if (__builtin_expect(r.ordinary, 1)) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      h[k] = FY == AR_BF16 || FY == AR_F16 ? (h[k] * r.hi) * g[k] : Product(h[k], r, g[k]).nearest();
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = product64<false>(h[k], r.r, g[k]);
  }
}

// The same for an MX format.  A value that lies just beside a border between two
// codes must not come out on its other side.  Borders, and powers of two, those of
// the scales, have 19 trailing zeros in binary32: two plain products do for a
// chunk without a value within kNear steps of such a place, which cover their
// error and that of r.hi, 3 * 2^-24.  The others (0.8% of the waves' chunks of
// random rows, and those with zeros) are rounded to odd, in binary64 where a
// product that is not a zero of its own is small.
constexpr uint32_t kNear = 4;
__device__ __forceinline__ void products8_mx(float (&h)[8], const Root& r, const float (&g)[8]) {
  float v[8], least_p = r.ordinary ? __builtin_inff() : 0.0f, least_q = __builtin_inff();
  uint32_t near = 0xFFFFFFFFu;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float p = h[k] * r.hi;
    v[k] = p * g[k];
    least_p = fminf(least_p, fabsf(p));
    least_q = fminf(least_q, fabsf(v[k]));
    near = min(near, (__float_as_uint(v[k]) + kNear) & 0x7FFFFu);
  }
  if (__builtin_expect(least_p < 0x1p-100f || least_q < 0x1p-100f || near <= 2 * kNear, 0)) {
    bool wide = !r.ordinary;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const Product x(h[k], r, g[k]);
      v[k] = x.odd();
      const bool small = fminf(fabsf(x.p), fabsf(x.q)) < 0x1p-100f && h[k] != 0.0f && g[k] != 0.0f;
      wide = wide || small || !(fabsf(x.q) < __builtin_inff());
      __builtin_amdgcn_sched_barrier(0);                   // one at a time: few registers
    }
    if (__builtin_expect(wide, 0)) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[k] = product64<true>(h[k], r.r, g[k]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) h[k] = v[k];
}

// From the row's h in registers (chunk i of thread t: elements
// [8 * (i * threads + t), ...)) to both outputs.
// Order of the sum, fixed by hidden and the thread count: a thread's own
// elements in order, lanes by a butterfly, waves in order.
template <int FX, int FR, int FY, int NI>
__device__ __forceinline__ void norm_finish(const NormArgs& a, int64_t row, float (&h)[NI][8],
                                            const Gamma<FX, NI>& gamma, NormShared& sm) {
  const int t = threadIdx.x, threads = blockDim.x;
  const int waves = threads >> 6, wave = t >> 6;
  const int chunks = (int)((a.hidden + 7) >> 3);
  const int64_t H = a.hidden;

  if (a.h) {
    typename Elem<FR>::type* hr = static_cast<typename Elem<FR>::type*>(a.h) + row * a.h_stride;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int c = i * threads + t;
      if (c < chunks) store8<FR>(hr, H, (int64_t)c * 8, h[i]);
    }
  }
  // The sum and r are binary64: with binary32 steps throughout, a few of 4 million
  // 8-bit codes came out a step off.
  double s = 0.0;
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) s = __builtin_fma((double)h[i][k], (double)h[i][k], s);
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) s += __shfl_xor(s, m, kWave);
  if (waves > 1) {
    if ((t & 63) == 0) sm.sum[wave] = s;
    __syncthreads();
    s = sm.sum[0];
    for (int w = 1; w < waves; ++w) s += sm.sum[w];
  }
  const Root r(reciprocal_root(s * a.inv_hidden + (double)a.eps));

#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int c = i * threads + t;
    const int left = (int)H - c * 8;                       // elements of the row from here on
    float g[8];
    gamma.get(a, i, g);
    if constexpr (is_mx_format(FY)) {
      if (left < 8) {                                      // zeros would be taken for small products
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          h[i][k] = k < left ? h[i][k] : 1.0f;
          g[k] = k < left ? g[k] : 1.0f;
        }
      }
      products8_mx(h[i], r, g);
    } else {
      products8<FY>(h[i], r, g);
    }
    // back to zeros; a row whose r is not finite makes NaN of zeros too
    if (left < 8) {
#pragma unroll
      for (int k = 0; k < 8; ++k) h[i][k] = k < left ? h[i][k] : 0.0f;
    }
  }

  if constexpr (is_float_format(FY)) {
    typename Elem<FY>::type* yr = static_cast<typename Elem<FY>::type*>(a.y) + row * a.y_stride;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int c = i * threads + t;
      if (c < chunks) store8<FY>(yr, H, (int64_t)c * 8, h[i]);
    }
  } else if constexpr (is_mx_format(FY)) {
    uint8_t* yr = static_cast<uint8_t*>(a.y) + row * a.y_stride;
    uint8_t* sr = static_cast<uint8_t*>(a.scales) + row * a.scale_stride;
    const int padded = (int)((H + kMxBlock - 1) / kMxBlock) * 4;   // chunks of whole blocks
#pragma unroll
    for (int i = 0; i < NI; ++i) store8_mx<FY>(yr, sr, i * threads + t, padded, h[i]);
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) m = max(m, max8_bits(h[i]));
#pragma unroll
    for (int k = 1; k < kWave; k <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, k, kWave));
    if (waves > 1) {
      if ((t & 63) == 0) sm.max[wave] = m;
      __syncthreads();
      m = sm.max[0];
      for (int w = 1; w < waves; ++w) m = max(m, sm.max[w]);
    }
    const bool nan = m >= kInfBits;
    const float scale = nan ? __uint_as_float(0x7FC00000u)
                            : fmaxf(__uint_as_float(m) / kE4m3Max, 0x1p-126f);
    const float mul = nan ? 1.0f : 1.0f / scale;
    if (t == 0) static_cast<float*>(a.scales)[row] = scale;
    uint8_t* yr = static_cast<uint8_t*>(a.y) + row * a.y_stride;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int c = i * threads + t;
      if (c >= chunks) continue;
      const u32x2 d = e4m3_codes(h[i], mul, nan);
      if ((int64_t)c * 8 + 8 <= H) {
        *reinterpret_cast<u32x2*>(yr + (int64_t)c * 8) = d;
      } else {
        for (int k = 0; (int64_t)c * 8 + k < H; ++k)
          yr[(int64_t)c * 8 + k] = (uint8_t)((k < 4 ? d.x : d.y) >> (8 * (k & 3)));
      }
    }
  }
}

template <int FX, int FR, int FY, int NI>
__global__ __launch_bounds__(kNormThreads) void k_residual_norm(NormArgs a) {
  __shared__ NormShared sm;
  const int64_t row = blockIdx.x;
  const int64_t H = a.hidden;
  constexpr int sx = sizeof(typename Elem<FX>::type), sr = sizeof(typename Elem<FR>::type);
  const rsrc_t xr = raw_row(static_cast<const uint8_t*>(a.x) + row * a.x_stride * sx, H, sx);
  const rsrc_t rr =
      raw_row(a.res ? static_cast<const uint8_t*>(a.res) + row * a.res_stride * sr : nullptr, H, sr);
  const Gamma<FX, NI> gamma(a);
  float h[NI][8];
  Raw<FX> xw[NI];
  Raw<FR> rw[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) xw[i] = load_raw<FX>(xr, chunk_first(i));
#pragma unroll
  for (int i = 0; i < NI; ++i) rw[i] = load_raw<FR>(rr, chunk_first(i));
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    values<FX>(xw[i], H, chunk_first(i), h[i]);
    if (a.res) {
      float q[8];
      values<FR>(rw[i], H, chunk_first(i), q);
#pragma unroll
      for (int k = 0; k < 8; ++k) h[i][k] = q[k] + h[i][k];
    }
  }
  norm_finish<FX, FR, FY, NI>(a, row, h, gamma, sm);
}

// ------------------------------------------------- in the receive side ---

struct ReduceNormArgs {
  NormArgs n;
  const uint8_t* scratch;
  uint32_t scratch_bytes, slot_bytes;
  int32_t nranks, rows;
  uint32_t seq, parity;
  int* ctrl;
  uint64_t timeout_ticks;
  int32_t rearm;
  int32_t res_format, y_format;
};

// 8 elements [e, e + 8) (e a multiple of 8) of one rank's payload as they lie
// in its slot: 32 bytes of LL words, 16 of the others.
template <int P> struct Raw8 { u32x4 a; };
template <> struct Raw8<kLL> { u32x4 a, b; };

template <int P>
__device__ __forceinline__ Raw8<P> recv8(rsrc_t rs, uint32_t slot, uint32_t e) {
  if constexpr (P == kLL) {
    return {ld16(rs, slot + e * 4u), ld16(rs, slot + e * 4u + 16u)};
  } else if constexpr (P == kLL128) {
    // the two halves of the chunk lie in one line each (60 = 15 * 4), maybe
    // in different ones; their flags have been seen before this load
    const uint32_t l0 = e / 60u, l1 = (e + 4u) / 60u;
    const u32x2 a = ld8(rs, slot + l0 * 128u + (e - 60u * l0) * 2u);
    const u32x2 b = ld8(rs, slot + l1 * 128u + (e + 4u - 60u * l1) * 2u);
    return {u32x4{a.x, a.y, b.x, b.y}};
  } else {
    return {ld16(rs, slot + e * 2u)};
  }
}

// Evidence that the chunk has arrived (LL128: the flags', elsewhere).
template <int P>
__device__ __forceinline__ void check8(const Raw8<P>& v, uint32_t seq, uint32_t stale, bool& ok, bool& bad) {
  if constexpr (P == kLL) {
    bool o, b;
    classify<P>(v.a, seq, stale, o, b);
    ok = ok && o;
    bad = bad || b;
    classify<P>(v.b, seq, stale, o, b);
    ok = ok && o;
    bad = bad || b;
  } else if constexpr (P != kLL128) {
    bool o, b;
    classify<P>(v.a, seq, stale, o, b);
    ok = ok && o;
    bad = bad || b;
  }
}

template <int P>
__device__ __forceinline__ void words8(const Raw8<P>& v, uint32_t (&w)[4]) {
  if constexpr (P == kLL) {
    w[0] = v.a.x; w[1] = v.a.z; w[2] = v.b.x; w[3] = v.b.z;
  } else {
    w[0] = v.a.x; w[1] = v.a.y; w[2] = v.a.z; w[3] = v.a.w;
  }
}

// The norm of a reduced row.  The formats are chosen at run time here: one
// kernel for each protocol and shape instead of eight.
template <int FR, int NI>
__device__ __forceinline__ void reduce_finish(const ReduceNormArgs& a, int64_t row, float (&h)[NI][8],
                                              const Gamma<AR_BF16, NI>& gamma, NormShared& sm) {
  switch (a.y_format) {
    case AR_E4M3_ROW: norm_finish<AR_BF16, FR, AR_E4M3_ROW, NI>(a.n, row, h, gamma, sm); break;
    case AR_E4M3_MX: norm_finish<AR_BF16, FR, AR_E4M3_MX, NI>(a.n, row, h, gamma, sm); break;
    case AR_E2M1_MX: norm_finish<AR_BF16, FR, AR_E2M1_MX, NI>(a.n, row, h, gamma, sm); break;
    default: norm_finish<AR_BF16, FR, AR_BF16, NI>(a.n, row, h, gamma, sm); break;
  }
}

// One workgroup per (consumer, row): every thread polls its own 8 elements
// of every rank until they carry their evidence (in whatever order the
// blocks arrive), adds them in rank order in binary32 and goes on with the
// norm; the sum is never rounded or written.
// 8 ranks, [1,4096], to 8-bit blocks: LL 7.6 us, LL128 6.8, sentinel 5.8, plain
// 4.2 (and 2.4 to 2.8 for the pack); 16 ranks, [8,4096], to 8 bits a row: 12.5, 11.8,
// 9.5, 6.5.  Plain slots are as long as the sentinel's, so in the 16-rank case 3 us
// are checks and re-arming; LL reads twice as much.  The rest is one CU's read of
// its row from every rank, past the L2, and the norm.  A row stays in one
// workgroup all the same: sharing it would put an exchange of sums between
// workgroups, which then must all be resident, into every row.
template <int P, int NMAX, int NI>
__global__ __launch_bounds__(kNormThreads) void k_reduce_norm(ReduceNormArgs a) {
  __shared__ NormShared sm;
  __shared__ int status[kNormThreads / kWave];
  const int t = threadIdx.x, threads = blockDim.x, lane = t & 63;
  const int c = blockIdx.x / a.rows;                       // consumer
  const int row = blockIdx.x - c * a.rows;
  const int64_t H = a.n.hidden;
  const rsrc_t rs = make_rsrc(a.scratch, a.scratch_bytes);
  const uint32_t src0 = ((uint32_t)c * 2u + a.parity) * (uint32_t)a.nranks * a.slot_bytes;
  const uint32_t stale = seq_prev(seq_prev(a.seq));
  // gamma and the residual need no waiting: on their way before the polls
  const int64_t orow = (int64_t)c * a.rows + row;
  const Gamma<AR_BF16, NI> gamma(a.n);
  const bool res32 = a.res_format == AR_F32;
  const int sr = res32 ? 4 : 2;
  const rsrc_t rr = raw_row(
      a.n.res ? static_cast<const uint8_t*>(a.n.res) + orow * a.n.res_stride * sr : nullptr, H, sr);
  Raw<AR_F32> rw[NI];                                      // a bf16 residual takes the first half
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const uint32_t off = (uint32_t)chunk_first(i) * (uint32_t)sr;
    rw[i].a = __builtin_amdgcn_raw_buffer_load_b128(rr, off, 0, 0);
    rw[i].b = __builtin_amdgcn_raw_buffer_load_b128(rr, res32 ? off + 16u : 0xFFFFFFF0u, 0, 0);
  }
  float h[NI][8];
  int st = 0;
  Waiter wt(a.timeout_ticks, a.ctrl);                      // one deadline for all of the wave's chunks
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int64_t first = ((int64_t)i * threads + t) * 8;
    const bool active = first < H;
    const uint32_t e = (uint32_t)row * (uint32_t)H + (uint32_t)first;
    Raw8<P> raw[NMAX];
    if (P == kLL128 && st == 0) {
      // the line flags first, the data only after they have been seen
      while (true) {
        bool ok = true, bad = false;
        if (active) {
          const uint32_t l0 = e / 60u, l1 = (e + 4u) / 60u;
          u32x2 f[NMAX][2];
#pragma unroll
          for (int r = 0; r < NMAX; ++r)
            if (r < a.nranks) {
              const uint32_t slot = src0 + (uint32_t)r * a.slot_bytes;
              f[r][0] = ld8(rs, slot + l0 * 128u + 120u);
              f[r][1] = ld8(rs, slot + l1 * 128u + 120u);
            }
#pragma unroll
          for (int r = 0; r < NMAX; ++r)
            if (r < a.nranks)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const u32x2 v = f[r][k];
                const bool o = v.x == a.seq && v.y == 0u;
                ok = ok && o;
                bad = bad || (!o && !(v.y == 0u && (v.x == 0u || v.x == stale)));
              }
        }
        if (__ballot(bad) != 0ull) {
          if (lane == 0) report_error(a.ctrl, kEcorrupt);
          st = kEcorrupt;
          break;
        }
        if (__ballot(!ok) == 0ull) break;
        if (!wt.again(lane)) {
          st = kEtimeout;
          break;
        }
      }
      fence_acquire();
    }
    while (st == 0) {
      bool ok = true, bad = false;
      if (active) {
        // every rank's loads first, then the checks: one trip for all
#pragma unroll
        for (int r = 0; r < NMAX; ++r)
          if (r < a.nranks) raw[r] = recv8<P>(rs, src0 + (uint32_t)r * a.slot_bytes, e);
#pragma unroll
        for (int r = 0; r < NMAX; ++r)
          if (r < a.nranks) check8<P>(raw[r], a.seq, stale, ok, bad);
      }
      if (__ballot(bad) != 0ull) {
        if (lane == 0) report_error(a.ctrl, kEcorrupt);
        st = kEcorrupt;
        break;
      }
      if (__ballot(!ok) == 0ull) break;
      if (!wt.again(lane)) {
        st = kEtimeout;
        break;
      }
    }
    if (P == kSentinel && st == 0 && a.rearm && active) {
#pragma unroll
      for (int r = 0; r < NMAX; ++r)
        if (r < a.nranks)
          st16(rs, src0 + (uint32_t)r * a.slot_bytes + e * 2u,
               u32x4{0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu, 0xFFFFFFFFu});
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) h[i][k] = 0.0f;
    if (st == 0 && active) {
#pragma unroll
      for (int r = 0; r < NMAX; ++r) {
        if (r >= a.nranks) continue;
        uint32_t w[4];
        words8<P>(raw[r], w);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // rank 0 starts the sum: an addition to zero would lose a -0
          h[i][2 * k] = r == 0 ? bf_lo(w[k]) : h[i][2 * k] + bf_lo(w[k]);
          h[i][2 * k + 1] = r == 0 ? bf_hi(w[k]) : h[i][2 * k + 1] + bf_hi(w[k]);
        }
      }
    }
  }
  if (lane == 0) status[t >> 6] = st;
  __syncthreads();
  for (int w = 0; w < threads >> 6; ++w) st |= status[w];
  if (st != 0) return;                                     // whole workgroup
  if (a.n.res) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float q[8];
      if (res32) values<AR_F32>(rw[i], H, chunk_first(i), q);
      else values<AR_BF16>(Raw<AR_BF16>{rw[i].a}, H, chunk_first(i), q);
#pragma unroll
      for (int k = 0; k < 8; ++k) h[i][k] = q[k] + h[i][k];
    }
  }
  if (res32) reduce_finish<AR_F32, NI>(a, orow, h, gamma, sm);
  else reduce_finish<AR_BF16, NI>(a, orow, h, gamma, sm);
}

// ================================================================ host side

// Threads a row and 8-element steps a thread.  MX rows take whole blocks.
struct NormShape {
  int threads, ni;
};

static NormShape norm_shape(int64_t hidden) {
  const int64_t chunks = (hidden + 31) / 32 * 4;
  int ni = 1;
  while (chunks > (int64_t)ni * kNormThreads) ni <<= 1;
  int64_t threads = (ceil_div64(chunks, ni) + 63) / 64 * 64;
  return {(int)threads, ni};
}

static int check_norm(const ar_norm_params* p, int64_t out_rows) {
  if (!p) return AR_EINVAL;
  if (p->rows < 0 || p->hidden < 0 || p->reserved != 0) return AR_EINVAL;
  if (!is_float_format(p->format)) return AR_EINVAL;
  if (p->res_format != p->format && p->res_format != AR_F32) return AR_EINVAL;
  if (p->y_format != p->format && (p->y_format < AR_E4M3_ROW || p->y_format > AR_E2M1_MX))
    return AR_EINVAL;
  if (!(p->eps >= 0.0f) || p->eps > 3.0e38f) return AR_EINVAL;
  if (p->rows == 0 || p->hidden == 0) return AR_OK;
  if (p->hidden > AR_NORM_MAX_HIDDEN) return AR_ESIZE;
  if (p->rows > INT32_MAX || out_rows > INT32_MAX) return AR_ESIZE;
  if (p->gamma && !aligned(p->gamma, 16)) return AR_EALIGN;
  int rc = AR_OK;
  if (p->residual) rc = check_format_rows(p->res_format, p->residual, p->residual_stride, out_rows, p->hidden);
  if (rc) return rc;
  if (p->residual_out)
    rc = check_format_rows(p->res_format, p->residual_out, p->residual_out_stride, out_rows, p->hidden);
  if (rc) return rc;
  rc = check_format_rows(p->y_format, p->y, p->y_stride, out_rows, p->hidden);
  if (rc) return rc;
  return check_scales(p->y_format, p->scales, p->scale_stride, out_rows, p->hidden);
}

static NormArgs norm_args(const ar_norm_params* p) {
  NormArgs a{};
  a.gamma = p->gamma;
  a.res = p->residual;
  a.res_stride = p->residual_stride;
  a.h = p->residual_out;
  a.h_stride = p->residual_out_stride;
  a.y = p->y;
  a.y_stride = p->y_stride;
  a.scales = p->scales;
  a.scale_stride = p->scale_stride;
  a.hidden = p->hidden;
  a.eps = p->eps;
  a.inv_hidden = 1.0 / (double)p->hidden;
  return a;
}

// A workgroup a row: one launch, or several where the rows are more than it takes.
template <int FX, int FR, int FY>
static hipError_t launch_norm_ni(NormArgs a, int64_t rows, NormShape g, hipStream_t s) {
  auto later = [](auto*& p, int64_t bytes) {
    if (p) p = static_cast<std::remove_reference_t<decltype(p)>>((void*)((uintptr_t)p + bytes));
  };
  auto go = [&](void (*kernel)(NormArgs)) {
    const int64_t most = most_blocks(g.threads);
    for (;; rows -= most) {
      const hipError_t e = launch(kernel, dim3((unsigned)(rows < most ? rows : most)), dim3(g.threads), s, a);
      if (e != hipSuccess || rows <= most) return e;
      later(a.x, most * format_bytes(FX, a.x_stride));
      later(a.res, most * format_bytes(FR, a.res_stride));
      later(a.h, most * format_bytes(FR, a.h_stride));
      later(a.y, most * format_bytes(FY, a.y_stride));
      later(a.scales, most * (FY == AR_E4M3_ROW ? 4 : a.scale_stride));
    }
  };
  switch (g.ni) {
    case 1: return go(k_residual_norm<FX, FR, FY, 1>);
    case 2: return go(k_residual_norm<FX, FR, FY, 2>);
    case 4: return go(k_residual_norm<FX, FR, FY, 4>);
    default: return go(k_residual_norm<FX, FR, FY, 8>);
  }
}

template <int FX, int FR>
static hipError_t launch_norm_y(const NormArgs& a, int64_t rows, int fy, NormShape g, hipStream_t s) {
  switch (fy) {
    case AR_E4M3_ROW: return launch_norm_ni<FX, FR, AR_E4M3_ROW>(a, rows, g, s);
    case AR_E4M3_MX: return launch_norm_ni<FX, FR, AR_E4M3_MX>(a, rows, g, s);
    case AR_E2M1_MX: return launch_norm_ni<FX, FR, AR_E2M1_MX>(a, rows, g, s);
    default: return launch_norm_ni<FX, FR, FX>(a, rows, g, s);
  }
}

template <int P, int NMAX>
static hipError_t launch_rnorm_ni(const ReduceNormArgs& a, unsigned blocks, NormShape g, hipStream_t s) {
  const dim3 grid(blocks), block(g.threads);
  switch (g.ni) {
    case 1: return launch(k_reduce_norm<P, NMAX, 1>, grid, block, s, a);
    case 2: return launch(k_reduce_norm<P, NMAX, 2>, grid, block, s, a);
    default: return launch(k_reduce_norm<P, NMAX, 4>, grid, block, s, a);
  }
}

template <int P>
static hipError_t launch_rnorm(const ReduceNormArgs& a, unsigned blocks, NormShape g, hipStream_t s) {
  if (a.nranks <= 4) return launch_rnorm_ni<P, 4>(a, blocks, g, s);
  if (a.nranks <= 8) return launch_rnorm_ni<P, 8>(a, blocks, g, s);
  return launch_rnorm_ni<P, 16>(a, blocks, g, s);
}

}  // namespace ar

using namespace ar;

extern "C" {

int ar_residual_norm(const ar_norm_params* p, const void* x, int64_t x_stride, void* stream) {
  int rc = check_norm(p, p ? p->rows : 0);
  if (rc) return rc;
  rc = check_format_rows(p->format, x, x_stride, p->rows, p->hidden);
  if (rc) return rc;
  if (p->rows == 0 || p->hidden == 0) return AR_OK;
  NormArgs a = norm_args(p);
  a.x = x;
  a.x_stride = x_stride;
  const NormShape g = norm_shape(p->hidden);
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t e;
  if (p->format == AR_F32) {
    e = launch_norm_y<AR_F32, AR_F32>(a, p->rows, p->y_format, g, s);
  } else if (p->format == AR_BF16) {
    e = p->res_format == AR_F32 ? launch_norm_y<AR_BF16, AR_F32>(a, p->rows, p->y_format, g, s)
                                : launch_norm_y<AR_BF16, AR_BF16>(a, p->rows, p->y_format, g, s);
  } else {
    e = p->res_format == AR_F32 ? launch_norm_y<AR_F16, AR_F32>(a, p->rows, p->y_format, g, s)
                                : launch_norm_y<AR_F16, AR_F16>(a, p->rows, p->y_format, g, s);
  }
  return map_hip(e);
}

int ar_reduce_norm(const ar_desc* d, void* scratch, const ar_norm_params* p, ar_epoch e, void* ctrl,
                   uint64_t timeout_ns, int32_t flags, void* stream) {
  int rc = check_desc(d);
  if (rc) return rc;
  if (d->collective != AR_ALLREDUCE) return AR_EINVAL;
  if (e.parity > 1u || e.seq == 0u) return AR_EINVAL;
  if (flags & ~AR_FLAG_REARM) return AR_EINVAL;
  if (!timeout_ok(timeout_ns)) return AR_EINVAL;
  if (!p || p->rows < 0 || p->hidden < 0) return AR_EINVAL;
  if (p->rows > INT32_MAX || p->hidden > INT32_MAX) return AR_ESIZE;
  rc = check_norm(p, p->rows * d->nconsumers);
  if (rc) return rc;
  if (p->format != AR_BF16) return AR_EINVAL;
  if (p->rows * p->hidden != d->count) return AR_EINVAL;
  if (d->count == 0) return AR_OK;
  if (p->hidden % 8 != 0) return AR_EALIGN;
  if (p->hidden > AR_REDUCE_NORM_MAX_HIDDEN) return AR_ESIZE;
  const NormShape g = norm_shape(p->hidden);
  if (p->rows * d->nconsumers > most_blocks(g.threads)) return AR_ESIZE;
  if (!scratch || !ctrl) return AR_EINVAL;
  if (!aligned(scratch, 256) || !aligned(ctrl, 256)) return AR_EALIGN;
  DeviceInfo di;
  rc = device_info(&di);
  if (rc) return rc;
  ReduceNormArgs a{};
  a.n = norm_args(p);
  a.scratch = static_cast<const uint8_t*>(scratch);
  a.slot_bytes = (uint32_t)desc_slot_bytes(d);
  a.scratch_bytes = (uint32_t)desc_scratch_bytes(d);
  a.nranks = d->nranks;
  a.rows = (int32_t)p->rows;
  a.seq = e.seq;
  a.parity = e.parity;
  a.ctrl = static_cast<int*>(ctrl);
  a.timeout_ticks = ns_to_ticks(timeout_ns, di.wallclock_hz);
  a.rearm = (flags & AR_FLAG_REARM) && d->proto == kSentinel;
  a.res_format = p->res_format;
  a.y_format = p->y_format;
  const unsigned blocks = (unsigned)(p->rows * d->nconsumers);
  hipStream_t s = static_cast<hipStream_t>(stream);
  hipError_t err;
  switch (d->proto) {
    case kLL: err = launch_rnorm<kLL>(a, blocks, g, s); break;
    case kLL128: err = launch_rnorm<kLL128>(a, blocks, g, s); break;
    case kSentinel: err = launch_rnorm<kSentinel>(a, blocks, g, s); break;
    default: err = launch_rnorm<kBarrier>(a, blocks, g, s); break;
  }
  return map_hip(err);
}

}  // extern "C"
