// ar_norm.hip -- residual addition and root-mean-square norm of rows, alone
// and in the receive side of the one-shot all-reduce (gfx950).
//
//     h = residual + x,  r = 1 / sqrt(sum(h^2) / hidden + eps),
//     v = (h * r) * gamma;  residual_out = round(h);  y = v in y's format.
//
// Everything between the inputs and the two outputs is binary32: h is not
// rounded before the norm, and each output is rounded once.
//
// What bounds it: for many rows the memory system (x and the residual read
// once, both outputs written once; a row stays in registers between the sum
// and the scaling), for few rows the launch and one trip to memory.  One
// workgroup a row: 8 consecutive elements a thread and step, so a wave reads
// 1 KiB of a 16-bit row in one instruction, and the 4 lanes of an aligned
// group hold one 32-element block of the MX formats.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "../../include/ar.h"
#include "ar_host.h"
#include "ar_rows.h"
#include "../../include/ar_protocols.h"

namespace ar {

constexpr int kNormMaxThreads = 1024;

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
  float inv_hidden;
};

// The waves' partial sums or maxima; a second array so that the maximum's
// writes need not wait for the sum's readers.
struct NormShared {
  float sum[kNormMaxThreads / kWave];
  uint32_t max[kNormMaxThreads / kWave];
};

// From the row's h in registers (chunk i of thread t: elements
// [8 * (i * threads + t), ...)) to both outputs.
// Order of the sum, fixed by hidden and the thread count: a thread's own
// elements in order, lanes by a butterfly, waves in order.
template <int FX, int FR, int FY, int NI>
__device__ __forceinline__ void norm_finish(const NormArgs& a, int64_t row, float (&h)[NI][8],
                                            NormShared& sm) {
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
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) s = __builtin_fmaf(h[i][k], h[i][k], s);
#pragma unroll
  for (int m = 1; m < kWave; m <<= 1) s += __shfl_xor(s, m, kWave);
  if (waves > 1) {
    if ((t & 63) == 0) sm.sum[wave] = s;
    __syncthreads();
    s = sm.sum[0];
    for (int w = 1; w < waves; ++w) s += sm.sum[w];
  }
  const float r = 1.0f / __builtin_sqrtf(s * a.inv_hidden + a.eps);

  const typename Elem<FX>::type* gm = static_cast<const typename Elem<FX>::type*>(a.gamma);
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int c = i * threads + t;
    float g[8];
    if (gm && c < chunks) {
      load8<FX>(gm, H, (int64_t)c * 8, g);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) g[k] = 1.0f;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) h[i][k] = (h[i][k] * r) * g[k];
    // a row whose r is not finite makes NaN of the zeros past its end
    if ((int64_t)c * 8 + 8 > H) {
#pragma unroll
      for (int k = 0; k < 8; ++k) h[i][k] = (int64_t)c * 8 + k < H ? h[i][k] : 0.0f;
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
__global__ __launch_bounds__(kNormMaxThreads) void k_residual_norm(NormArgs a) {
  __shared__ NormShared sm;
  const int64_t row = blockIdx.x;
  const int t = threadIdx.x, threads = blockDim.x;
  const int64_t H = a.hidden;
  const auto* xr = static_cast<const typename Elem<FX>::type*>(a.x) + row * a.x_stride;
  const auto* rr = a.res ? static_cast<const typename Elem<FR>::type*>(a.res) + row * a.res_stride
                         : nullptr;
  float h[NI][8];
#pragma unroll
  for (int i = 0; i < NI; ++i) load8<FX>(xr, H, ((int64_t)i * threads + t) * 8, h[i]);
  if (rr) {
    float q[NI][8];
#pragma unroll
    for (int i = 0; i < NI; ++i) load8<FR>(rr, H, ((int64_t)i * threads + t) * 8, q[i]);
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) h[i][k] = q[i][k] + h[i][k];
  }
  norm_finish<FX, FR, FY, NI>(a, row, h, sm);
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

// 8 elements [e, e + 8) (e a multiple of 8) of one rank's payload, as packed
// bf16 pairs, with the evidence that they have arrived.
template <int P>
__device__ __forceinline__ void recv8(rsrc_t rs, uint32_t slot, uint32_t e, uint32_t seq,
                                      uint32_t stale, uint32_t (&w)[4], bool& ok, bool& bad) {
  if constexpr (P == kLL) {
    const u32x4 a = ld16(rs, slot + e * 4u);
    const u32x4 b = ld16(rs, slot + e * 4u + 16u);
    bool o1, b1, o2, b2;
    classify<P>(a, seq, stale, o1, b1);
    classify<P>(b, seq, stale, o2, b2);
    ok = o1 && o2;
    bad = b1 || b2;
    w[0] = a.x; w[1] = a.z; w[2] = b.x; w[3] = b.z;
  } else if constexpr (P == kLL128) {
    // the two halves of the chunk lie in one line each (60 = 15 * 4), maybe
    // in different ones; their flags have been seen before this load
    const uint32_t l0 = e / 60u, l1 = (e + 4u) / 60u;
    const u32x2 a = ld8(rs, slot + l0 * 128u + (e - 60u * l0) * 2u);
    const u32x2 b = ld8(rs, slot + l1 * 128u + (e + 4u - 60u * l1) * 2u);
    ok = true;
    bad = false;
    w[0] = a.x; w[1] = a.y; w[2] = b.x; w[3] = b.y;
  } else {
    const u32x4 a = ld16(rs, slot + e * 2u);
    classify<P>(a, seq, stale, ok, bad);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  }
}

// The residual and the norm of a reduced row.  The formats are chosen at run
// time here: one kernel for each protocol and shape instead of eight.
template <int FR, int NI>
__device__ __forceinline__ void reduce_finish(const ReduceNormArgs& a, int64_t row, float (&h)[NI][8],
                                              NormShared& sm) {
  const int t = threadIdx.x, threads = blockDim.x;
  if (a.n.res) {
    const auto* rr = static_cast<const typename Elem<FR>::type*>(a.n.res) + row * a.n.res_stride;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float q[8];
      load8<FR>(rr, a.n.hidden, ((int64_t)i * threads + t) * 8, q);
#pragma unroll
      for (int k = 0; k < 8; ++k) h[i][k] = q[k] + h[i][k];
    }
  }
  switch (a.y_format) {
    case AR_E4M3_ROW: norm_finish<AR_BF16, FR, AR_E4M3_ROW, NI>(a.n, row, h, sm); break;
    case AR_E4M3_MX: norm_finish<AR_BF16, FR, AR_E4M3_MX, NI>(a.n, row, h, sm); break;
    case AR_E2M1_MX: norm_finish<AR_BF16, FR, AR_E2M1_MX, NI>(a.n, row, h, sm); break;
    default: norm_finish<AR_BF16, FR, AR_BF16, NI>(a.n, row, h, sm); break;
  }
}

// One workgroup per (consumer, row): every thread polls its own 8 elements
// of every rank until they carry their evidence (in whatever order the
// blocks arrive), adds them in rank order in binary32 and goes on with the
// norm; the sum is never rounded or written.
template <int P, int NMAX, int NI>
__global__ __launch_bounds__(NMAX == 16 ? 512 : kNormMaxThreads) void k_reduce_norm(ReduceNormArgs a) {
  __shared__ NormShared sm;
  __shared__ int err;
  const int t = threadIdx.x, threads = blockDim.x, lane = t & 63;
  const int c = blockIdx.x / a.rows;                       // consumer
  const int row = blockIdx.x - c * a.rows;
  const int64_t H = a.n.hidden;
  const rsrc_t rs = make_rsrc(a.scratch, a.scratch_bytes);
  const uint32_t src0 = ((uint32_t)c * 2u + a.parity) * (uint32_t)a.nranks * a.slot_bytes;
  const uint32_t stale = seq_prev(seq_prev(a.seq));
  if (t == 0) err = 0;
  __syncthreads();
  float h[NI][8];
  int st = 0;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int64_t first = ((int64_t)i * threads + t) * 8;
    const bool active = first < H;
    const uint32_t e = (uint32_t)row * (uint32_t)H + (uint32_t)first;
    uint32_t w[NMAX][4];
    Waiter wt(a.timeout_ticks, a.ctrl);
    if (P == kLL128 && st == 0) {
      // the line flags first, the data only after they have been seen
      while (true) {
        bool ok = true, bad = false;
        if (active) {
          const uint32_t l0 = e / 60u, l1 = (e + 4u) / 60u;
#pragma unroll
          for (int r = 0; r < NMAX; ++r) {
            if (r >= a.nranks) continue;
            const uint32_t slot = src0 + (uint32_t)r * a.slot_bytes;
            const u32x2 f = ld8(rs, slot + l0 * 128u + 120u);
            const u32x2 g = ld8(rs, slot + l1 * 128u + 120u);
            const bool o1 = f.x == a.seq && f.y == 0u, o2 = g.x == a.seq && g.y == 0u;
            ok = ok && o1 && o2;
            bad = bad || (!o1 && !(f.y == 0u && (f.x == 0u || f.x == stale))) ||
                  (!o2 && !(g.y == 0u && (g.x == 0u || g.x == stale)));
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
#pragma unroll
        for (int r = 0; r < NMAX; ++r) {
          if (r >= a.nranks) continue;
          bool o, b;
          recv8<P>(rs, src0 + (uint32_t)r * a.slot_bytes, e, a.seq, stale, w[r], o, b);
          ok = ok && o;
          bad = bad || b;
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
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          // rank 0 starts the sum: an addition to zero would lose a -0
          h[i][2 * k] = r == 0 ? bf_lo(w[r][k]) : h[i][2 * k] + bf_lo(w[r][k]);
          h[i][2 * k + 1] = r == 0 ? bf_hi(w[r][k]) : h[i][2 * k + 1] + bf_hi(w[r][k]);
        }
      }
    }
  }
  if (st != 0 && lane == 0) err = 1;
  __syncthreads();
  if (err) return;                                         // whole workgroup
  const int64_t orow = (int64_t)c * a.rows + row;
  if (a.res_format == AR_F32) reduce_finish<AR_F32, NI>(a, orow, h, sm);
  else reduce_finish<AR_BF16, NI>(a, orow, h, sm);
}

// ================================================================ host side

// Threads a row and 8-element steps a thread.  MX rows take whole blocks.
struct NormShape {
  int threads, ni;
};

static NormShape norm_shape(int64_t hidden, int max_threads) {
  const int64_t chunks = (hidden + 31) / 32 * 4;
  int ni = 1;
  while (ni < 8 && chunks > (int64_t)ni * max_threads) ni <<= 1;
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
  a.inv_hidden = 1.0f / (float)p->hidden;
  return a;
}

template <int FX, int FR, int FY>
static hipError_t launch_norm_ni(const NormArgs& a, int64_t rows, NormShape g, hipStream_t s) {
  const dim3 grid((unsigned)rows), block(g.threads);
  switch (g.ni) {
    case 1: return launch(k_residual_norm<FX, FR, FY, 1>, grid, block, s, a);
    case 2: return launch(k_residual_norm<FX, FR, FY, 2>, grid, block, s, a);
    case 4: return launch(k_residual_norm<FX, FR, FY, 4>, grid, block, s, a);
    default: return launch(k_residual_norm<FX, FR, FY, 8>, grid, block, s, a);
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
  const NormShape g = norm_shape(p->hidden, kNormMaxThreads);
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
  const NormShape g = norm_shape(p->hidden, d->nranks > 8 ? 512 : kNormMaxThreads);
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
