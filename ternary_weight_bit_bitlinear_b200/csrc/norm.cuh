// norm.cuh -- what a decoder layer does between two ternary products, one
// pass over each token row: residual addition and root-mean-square norm
// (norm_quant), or act(gate) * up and an optional norm (gated_norm_quant),
// then the per-token absmax int8 quantiser of quant.cuh.
//
//   h    = x, T(x + residual), or act(gate) * up (kept in fp32)
//   r    = fp32(1 / sqrt(sum h^2 / K + eps))     1 / K as a 64-bit factor
//   v    = (h * r) * w                      without the norm, v = h
//   amax = max |v|,  q = clamp(rint(v * (127 / amax)), -128, 127)
//
// The sum of squares and r are held in 64 bits and r is rounded once.  Squares
// of fp32 values are exact there, their sum is not: how the row is cut into
// threads changes it by a few 2^-53, and r, and the codes with it, only where
// that reaches across the middle of two fp32 values (2^-24 apart from either:
// about one row in 10^8).  Every other row comes out as the definition has it,
// bit for bit.  The maximum keeps inf and NaN: a row that holds either gets
// amax = NaN and q = 0.
//
// Two kernels, both reading each element once and holding it in registers from
// the load to the codes (kElems per thread, 8 to 48):
//   norm_stream_kernel  rows up to 16384 wide, one CTA per row: persistent CTAs
//                       whose next row is on its way into shared memory while
//                       the present one goes through its sum and its maximum;
//   norm_quant_kernel   wider rows, 4 or 8 CTAs of a cluster per row: sum,
//                       maximum and code sum go from every warp to every CTA
//                       of the row with asynchronous stores into the cluster's
//                       shared memories, whose bytes an mbarrier of the
//                       receiver counts.
// The waits are bounded, as everywhere.
//
// Bound by memory in fp32 with a residual (2048 x 8192: 37.6 us, 5.8 TB/s of
// the 13 bytes an element).  Rows of 16 bits are bound by the latency of one
// step after another with few warps per SM (2048 x 4096 bf16 with a residual:
// 13.3 us, 4.4 TB/s, 19 warps; gate and up 2048 x 6912: 22.9 us, 3.1 TB/s, 16):
// their 26 and 30 instructions an element fill half of the issue slots, no pipe
// is above 41 % (ALU) and DRAM is at 25 % of its peak; a warp waits for shared
// memory and shuffles, for the next row's copy and for barriers.  One token: 2.5 us at 2560, 3.2 at
// 8192 (launch to launch), 4.0 at 28672, where one CTA would take 14.6.
#pragma once

#include "element.cuh"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace bl {

struct NormParams {
  const void* a;          // x, or gate
  const void* b;          // residual (may be null), or up
  void* h;                // x + residual, written when there is a residual
  const float* weight;    // [K] or null
  int8_t* xq;
  float* amax;
  int32_t* xsum;          // may be null
  long long lda, ldb, ldh;
  double eps, inv_k;      // inv_k = 1 / K
  unsigned long long wait_ns;
  int K;
  int slice;              // norm_quant_kernel: chunks of 16 bytes of x per CTA
  int normalize;
  int act;
};

// r = 1 / sqrt(t) rounded to fp32: the hardware's fp32 estimate (22 bits) and
// two Newton steps y (3 - t y^2) / 2 in 64 bits, which leave an error of a few
// 2^-53; a quotient of a 64-bit root, which takes ten times as long, only
// where t leaves fp32's middle range.
__device__ __forceinline__ float norm_rsqrt(double t) {
  if (t > 1e-30 && t < 1e30) {
    double y = static_cast<double>(rsqrtf(static_cast<float>(t)));
    const double h = 0.5 * t;
#pragma unroll
    for (int i = 0; i < 2; ++i) y = fma(y, fma(-h * y, y, 0.5), y);
    return static_cast<float>(y);
  }
  return static_cast<float>(1.0 / sqrt(t));
}

// A thread's chunks past the end of its row hold zeros, which change no sum and
// no maximum: everything but loads and stores runs without a condition, so the
// instructions of different chunks interleave.

// The 16 bytes of x or gate, and of residual or up, that make chunk c of a row;
// zeros unless `in`.
struct NormRaw {
  uint4 a, b;
};

template <typename T>
__device__ __forceinline__ NormRaw norm_fetch(const T* a, const T* b, int c, bool in, bool two) {
  NormRaw v;
  v.a = v.b = make_uint4(0, 0, 0, 0);
  if (in) v.a = *(reinterpret_cast<const uint4*>(a) + c);
  if (in && two) v.b = *(reinterpret_cast<const uint4*>(b) + c);
  return v;
}

// Row values of chunk c as fp32; x + residual is written to h on the way.
template <typename T, bool kGated>
__device__ __forceinline__ void norm_combine(const NormParams& p, const NormRaw& v, bool two, T* h,
                                             int c, bool in, float (&f)[kVec<T>]) {
  constexpr int E = kVec<T>;
  Vec16<T> x, y;
  x.u = v.a;
  y.u = v.b;
#pragma unroll
  for (int i = 0; i < E; ++i) f[i] = Elem<T>::to_float(x.e[i]);
  if constexpr (kGated) {
    if (in) {   // (a warp with nothing left skips the activation)
      activate_exact_all(f, p.act);
#pragma unroll
      for (int i = 0; i < E; ++i) f[i] = __fmul_rn(f[i], Elem<T>::to_float(y.e[i]));
    }
  } else if (two) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      x.e[i] = Elem<T>::from_float(__fadd_rn(f[i], Elem<T>::to_float(y.e[i])));
      f[i] = Elem<T>::to_float(x.e[i]);
    }
    if (in) *(reinterpret_cast<uint4*>(h) + c) = x.u;
  }
}

// The weights of chunk c (ones without a weight): asked for before the row's
// sum is exchanged, so that they are there when r is.
template <int E>
__device__ __forceinline__ void norm_weights(const float* w, int c, bool in,
                                             float4 (&to)[E / 4]) {
  const float4* w4 = reinterpret_cast<const float4*>(w) + static_cast<int64_t>(c) * (E / 4);
#pragma unroll
  for (int i = 0; i < E / 4; ++i) {
    to[i] = make_float4(1.0f, 1.0f, 1.0f, 1.0f);
    if (in) to[i] = __ldg(w4 + i);
  }
}

template <int E>
__device__ __forceinline__ void norm_scale(bool weighted, const float4 (&w)[E / 4], float r,
                                           float (&f)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) f[i] = __fmul_rn(f[i], r);
  if (weighted) {
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      f[4 * i] = __fmul_rn(f[4 * i], w[i].x);
      f[4 * i + 1] = __fmul_rn(f[4 * i + 1], w[i].y);
      f[4 * i + 2] = __fmul_rn(f[4 * i + 2], w[i].z);
      f[4 * i + 3] = __fmul_rn(f[4 * i + 3], w[i].w);
    }
  }
}

// max(m, |v|) that keeps a NaN.
__device__ __forceinline__ float norm_max(float m, float v) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(fabsf(v)));
  return r;
}

// What a row's values are turned into codes with.
struct NormScale {
  float s;      // 127 / amax
  bool none;    // a row of zeros, or with inf or NaN: every code 0
  __device__ __forceinline__ explicit NormScale(float amax) {
    none = !(amax > 0.0f && amax < __uint_as_float(0x7F800000u));
    s = none ? 0.0f : __fdiv_rn(127.0f, amax);
  }
};

// Four codes: rint(v * s).  |v * s| <= 127 (1 + 2^-22), so adding 1.5 * 2^23
// rounds to the integer, half to even, and leaves it in the low byte: no
// conversion instruction (16 a cycle and SM, beside those of the 64-bit sum)
// and no clamp.  Where 127 / amax overflows, quant_pack4 follows the
// definition.
__device__ __forceinline__ uint32_t norm_codes(const float* f, float s, int& sum) {
  uint32_t b[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    b[i] = __float_as_uint(__fadd_rn(__fmul_rn(f[i], s), 12582912.0f));
  const uint32_t w = __byte_perm(__byte_perm(b[0], b[1], 0x0040),
                                 __byte_perm(b[2], b[3], 0x0040), 0x5410);
  sum = __dp4a(static_cast<int>(w), 0x01010101, sum);
  return w;
}

// The codes of chunks first, first + step, ... before end, R of them; which of
// the three ways is the row's.
template <int R, int E>
__device__ __forceinline__ void norm_store_codes(int8_t* out, int first, int step, int end,
                                                 const NormScale& q, const float (&v)[R][E],
                                                 int& sum) {
  auto each = [&](auto four) {
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int c = first + j * step;
      uint32_t* o = reinterpret_cast<uint32_t*>(out + static_cast<int64_t>(c) * E);
      if constexpr (E == 8) {
        const uint2 w = make_uint2(four(&v[j][0]), four(&v[j][4]));
        if (c < end) *reinterpret_cast<uint2*>(o) = w;
      } else {
        const uint32_t w = four(&v[j][0]);
        if (c < end) o[0] = w;
      }
    }
  };
  if (q.none)
    each([&](const float*) { return 0u; });
  else if (q.s < __uint_as_float(0x7F800000u))
    each([&](const float* f) { return norm_codes(f, q.s, sum); });
  else
    each([&](const float* f) {
      return quant_pack4(make_float4(f[0], f[1], f[2], f[3]), q.s, sum);
    });
}

constexpr int kNormMaxCluster = 8;

// One value per warp of the row, from all its CTAs: slot rank * W + warp.
template <typename V, int W>
struct NormExchange {
  V slot[kNormMaxCluster * W];
  uint64_t full;
};

__device__ __forceinline__ void st_async(void* p, uint64_t* bar, int rank, double v) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %2, [%1];" ::"r"(
                   map_cluster(p, rank)),
               "r"(map_cluster(bar, rank)), "l"(__double_as_longlong(v))
               : "memory");
}
__device__ __forceinline__ void st_async(void* p, uint64_t* bar, int rank, uint32_t v) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %2, [%1];" ::"r"(
                   map_cluster(p, rank)),
               "r"(map_cluster(bar, rank)), "r"(v)
               : "memory");
}

// Every lane of a warp passes the warp's value v; `to` CTAs (0 .. to - 1 of the
// cluster) receive it, all of them or the first alone.  The CTAs among them
// return combine over the row's values, in one order for all; a CTA that does
// not receive returns v.
template <int W, typename V, class Combine>
__device__ __forceinline__ V norm_exchange(NormExchange<V, W>& x, V v, int C, int to, int rank,
                                           int warp, int lane, int* abort,
                                           unsigned long long wait_ns, V none, Combine combine) {
  if (C == 1) {
    if (lane == 0) x.slot[warp] = v;
    __syncthreads();
    constexpr int P = W <= 4 ? 4 : W <= 8 ? 8 : 16;   // W is 4, 5, 8 or 16
    V s = (lane & (P - 1)) < W ? x.slot[lane & (P - 1)] : none;
#pragma unroll
    for (int o = P / 2; o > 0; o >>= 1) s = combine(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
    return s;
  }
  if (lane < to) st_async(&x.slot[rank * W + warp], &x.full, lane, v);
  if (rank >= to) return v;
  mbar_wait_warp(&x.full, 0, abort, wait_ns);   // given up: the row comes out wrong
  V s = none;
  for (int i = lane; i < C * W; i += 32) s = combine(s, x.slot[i]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s = combine(s, __shfl_xor_sync(0xFFFFFFFFu, s, o));
  return s;
}

// The row's maximum from each thread's; NaN where the row holds inf or NaN.
// (As unsigned integers the patterns of inf and NaN are above every finite's.)
template <int W>
__device__ __forceinline__ float norm_row_max(NormExchange<uint32_t, W>& x, float most, int C,
                                              int rank, int warp, int lane, int* abort,
                                              unsigned long long wait_ns) {
  const uint32_t top = norm_exchange<W>(
      x, __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(most) & 0x7FFFFFFFu), C, C, rank, warp,
      lane, abort, wait_ns, 0u, [](uint32_t a, uint32_t b) { return max(a, b); });
  return __uint_as_float(top < 0x7F800000u ? top : 0x7FC00000u);
}

// One row per cluster; p.slice <= R * kThreads.
template <typename T, int kThreads, int kElems, bool kGated>
static __global__ void __launch_bounds__(kThreads)
norm_quant_kernel(const __grid_constant__ NormParams p) {
  constexpr int E = kVec<T>;
  constexpr int R = kElems / E;
  constexpr int W = kThreads / 32;
  __shared__ NormExchange<double, W> xd;
  __shared__ NormExchange<uint32_t, W> xm, xs;
  __shared__ int abort;
  const int C = static_cast<int>(cluster_nctarank());
  const int rank = static_cast<int>(cluster_ctarank());
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) {
    abort = 0;
    mbar_init(&xd.full, 1);
    mbar_init(&xm.full, 1);
    mbar_init(&xs.full, 1);
    fence_mbar_init();
    if (p.normalize) mbar_arrive_expect_tx(&xd.full, C * W * sizeof(double));
    mbar_arrive_expect_tx(&xm.full, C * W * sizeof(uint32_t));
    if (p.xsum && rank == 0) mbar_arrive_expect_tx(&xs.full, C * W * sizeof(uint32_t));
  }
  cluster_sync();   // the barriers exist before another CTA's bytes arrive
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int64_t row = blockIdx.x / C;
  const T* a = static_cast<const T*>(p.a) + row * p.lda;
  const T* b = p.b ? static_cast<const T*>(p.b) + row * p.ldb : nullptr;
  T* h = p.h ? static_cast<T*>(p.h) + row * p.ldh : nullptr;
  int8_t* out = p.xq + row * p.K;
  // this thread's first chunk of E elements of this slice, and the slice's end
  const int c0 = p.slice * rank + tid;
  const int c1 = min(p.K / E, p.slice * (rank + 1));

  // Everything is asked for before anything is used: a store to h between two
  // loads, or a choice of activation, would leave one load in flight at a time.
  const bool two = kGated || b != nullptr;
  NormRaw raw[R];
#pragma unroll
  for (int j = 0; j < R; ++j)
    raw[j] = norm_fetch(a, b, c0 + j * kThreads, c0 + j * kThreads < c1, two);
  float v[R][E];
#pragma unroll
  for (int j = 0; j < R; ++j)
    norm_combine<T, kGated>(p, raw[j], two, h, c0 + j * kThreads, c0 + j * kThreads < c1, v[j]);
  float r = 1.0f;
  float4 w[R][E / 4];
  if (p.weight) {
#pragma unroll
    for (int j = 0; j < R; ++j)
      norm_weights<E>(p.weight, c0 + j * kThreads, c0 + j * kThreads < c1, w[j]);
  }
  if (p.normalize) {
    double ss[4] = {0.0, 0.0, 0.0, 0.0};   // four chains: the additions' latency
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const double d = static_cast<double>(v[j][i]);
        ss[i & 3] = fma(d, d, ss[i & 3]);
      }
    double t = (ss[0] + ss[1]) + (ss[2] + ss[3]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
    t = norm_exchange<W>(xd, t, C, C, rank, warp, lane, &abort, p.wait_ns, 0.0,
                         [](double x, double y) { return x + y; });
    r = norm_rsqrt(fma(t, p.inv_k, p.eps));
  }

  float most = 0.0f;
  if (p.normalize) {
#pragma unroll
    for (int j = 0; j < R; ++j) norm_scale<E>(p.weight != nullptr, w[j], r, v[j]);
  }
#pragma unroll
  for (int j = 0; j < R; ++j)
#pragma unroll
    for (int i = 0; i < E; ++i) most = norm_max(most, v[j][i]);
  const float amax = norm_row_max<W>(xm, most, C, rank, warp, lane, &abort, p.wait_ns);
  const NormScale q(amax);
  int sum = 0;
  norm_store_codes<R, E>(out, c0, kThreads, c1, q, v, sum);
  if (tid == 0 && rank == 0) p.amax[row] = amax;
  if (p.xsum) {
    const uint32_t total =
        norm_exchange<W>(xs, static_cast<uint32_t>(__reduce_add_sync(0xFFFFFFFFu, sum)), C, 1,
                         rank, warp, lane, &abort, p.wait_ns, 0u,
                         [](uint32_t x, uint32_t y) { return x + y; });
    if (tid == 0 && rank == 0) p.xsum[row] = static_cast<int32_t>(total);
  }
  // Given up: what the other CTAs may still send has landed before this one exits.
  if (tid == 0 && *static_cast<volatile int*>(&abort)) {
    if (p.normalize) mbar_drain(&xd.full, 0);
    mbar_drain(&xm.full, 0);
    if (p.xsum && rank == 0) mbar_drain(&xs.full, 0);
  }
}

// Whole rows, K <= kElems * kThreads, in persistent CTAs.  The next row
// of a CTA is on its way into shared memory (bulk copies) while the present
// one, in registers, goes through its sum and its maximum, so memory does not
// wait for the reductions (2048 x 8192 fp32 with a residual: 37.6 us against
// 62.8 with one CTA per row and no copy ahead).
template <typename T, int kThreads, int kElems, bool kGated>
static __global__ void __launch_bounds__(kThreads)
norm_stream_kernel(const __grid_constant__ NormParams p, int rows) {
  constexpr int E = kVec<T>;
  constexpr int R = kElems / E;
  constexpr int W = kThreads / 32;
  extern __shared__ __align__(128) uint8_t next_row[];   // x or gate, then residual or up
  __shared__ NormExchange<double, W> xd;
  __shared__ NormExchange<uint32_t, W> xm, xs;
  __shared__ uint64_t full;
  __shared__ int abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = p.K / E;
  const uint32_t bytes = static_cast<uint32_t>(p.K * sizeof(T));
  const bool two = kGated || p.b != nullptr;
  auto fetch = [&](int64_t row) {   // one thread
    mbar_arrive_expect_tx(&full, two ? 2 * bytes : bytes);
    bulk_load(next_row, static_cast<const T*>(p.a) + row * p.lda, bytes, &full);
    if (two) bulk_load(next_row + bytes, static_cast<const T*>(p.b) + row * p.ldb, bytes, &full);
  };
  if (tid == 0) {
    abort = 0;
    mbar_init(&full, 1);
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  if (tid == 0) fetch(blockIdx.x);
  uint32_t phase = 0;
  bool fetched = true;   // a copy is in flight (or has landed) that phase belongs to
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, phase ^= 1u) {
    const bool ok = mbar_wait(&full, phase, &abort, p.wait_ns);
    T* h = p.h ? static_cast<T*>(p.h) + row * p.ldh : nullptr;
    float v[R][E];
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int c = tid + j * kThreads;
      const NormRaw raw = norm_fetch(reinterpret_cast<const T*>(next_row),
                                     reinterpret_cast<const T*>(next_row + bytes), c, c < C, two);
      norm_combine<T, kGated>(p, raw, two, h, c, c < C, v[j]);
    }
    if (!__syncthreads_and(ok)) break;             // the row has been read, by all
    fetched = row + gridDim.x < rows;
    if (tid == 0 && fetched) fetch(row + gridDim.x);

    float r = 1.0f;
    float4 w[R][E / 4];
    if (p.weight) {
#pragma unroll
      for (int j = 0; j < R; ++j)
        norm_weights<E>(p.weight, tid + j * kThreads, tid + j * kThreads < C, w[j]);
    }
    if (p.normalize) {
      double ss[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const double d = static_cast<double>(v[j][i]);
          ss[i & 3] = fma(d, d, ss[i & 3]);
        }
      double t = (ss[0] + ss[1]) + (ss[2] + ss[3]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
      t = norm_exchange<W>(xd, t, 1, 1, 0, warp, lane, &abort, p.wait_ns, 0.0,
                           [](double x, double y) { return x + y; });
      r = norm_rsqrt(fma(t, p.inv_k, p.eps));
    }
    float most = 0.0f;
    if (p.normalize) {
#pragma unroll
      for (int j = 0; j < R; ++j) norm_scale<E>(p.weight != nullptr, w[j], r, v[j]);
    }
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int i = 0; i < E; ++i) most = norm_max(most, v[j][i]);
    const float amax = norm_row_max<W>(xm, most, 1, 0, warp, lane, &abort, p.wait_ns);
    const NormScale q(amax);
    int8_t* out = p.xq + row * p.K;
    int sum = 0;
    norm_store_codes<R, E>(out, tid, kThreads, C, q, v, sum);
    if (tid == 0) p.amax[row] = amax;
    if (p.xsum) {
      const uint32_t total =
          norm_exchange<W>(xs, static_cast<uint32_t>(__reduce_add_sync(0xFFFFFFFFu, sum)), 1, 1,
                           0, warp, lane, &abort, p.wait_ns, 0u,
                           [](uint32_t x, uint32_t y) { return x + y; });
      if (tid == 0) p.xsum[row] = static_cast<int32_t>(total);
    }
  }
  // Given up: the copy in flight has landed before the CTA exits.
  if (tid == 0 && fetched && *static_cast<volatile int*>(&abort)) mbar_drain(&full, phase);
}

}  // namespace bl
