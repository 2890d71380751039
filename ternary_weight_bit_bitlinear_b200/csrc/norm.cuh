// norm.cuh -- what a decoder layer does between two ternary products, one
// pass over each token row: residual addition and root-mean-square norm
// (norm_quant), or act(gate) * up and an optional norm (gated_norm_quant),
// then the per-token absmax int8 quantiser of quant.cuh.
//
//   h    = x, T(x + residual), or act(gate) * up (kept in fp32)
//   r    = fp32(1 / sqrt(sum h^2 / K + eps))
//   v    = (h * r) * w                      without the norm, v = h
//   amax = max |v|,  q = clamp(rint(v * (127 / amax)), -128, 127)
//
// The sum of squares and r are held in 64 bits and r is rounded once (squares
// of fp32 values are exact there), so r, and with it every code, does not
// depend on how the row is cut into threads: the result is the definition's,
// as it is for the library's other integer results.  The maximum is taken
// over the bit patterns of |v|, whose unsigned order puts inf and NaN above
// every finite value: a row that holds either gets amax = NaN and q = 0.
//
// One CTA per row.  A thread keeps its part of the row in registers from the
// load to the codes (rows up to kNormRegElems * kThreads wide are read once);
// wider rows read the rest again for each of the three passes.
#pragma once

#include "element.cuh"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace bl {

constexpr int kNormRegElems = 32;   // values of the row each thread keeps

struct NormParams {
  const void* a;          // x, or gate
  const void* b;          // residual (may be null), or up
  void* h;                // x + residual, written when there is a residual
  const float* weight;    // [K] or null
  int8_t* xq;
  float* amax;
  int32_t* xsum;          // may be null
  long long lda, ldb, ldh;
  double eps;
  int K;
  int normalize;
  int act;
};

// Row values of chunk c (kVec<T> of them) as fp32.
template <typename T, bool kGated>
__device__ __forceinline__ void norm_load(const NormParams& p, const T* a, const T* b, T* h,
                                          int c, bool first, float (&f)[kVec<T>]) {
  constexpr int E = kVec<T>;
  float g[E];
  if constexpr (kGated) {
    load_vec(a + static_cast<int64_t>(c) * E, f);
    load_vec(b + static_cast<int64_t>(c) * E, g);
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = __fmul_rn(activate(f[i], p.act), g[i]);
  } else if (b == nullptr) {
    load_vec(a + static_cast<int64_t>(c) * E, f);
  } else if (first) {
    load_vec(a + static_cast<int64_t>(c) * E, f);
    load_vec(b + static_cast<int64_t>(c) * E, g);
#pragma unroll
    for (int i = 0; i < E; ++i) f[i] = __fadd_rn(f[i], g[i]);
    store_vec(h + static_cast<int64_t>(c) * E, f);
  } else {
    load_vec(h + static_cast<int64_t>(c) * E, f);   // this thread wrote it
  }
}

template <int E>
__device__ __forceinline__ void norm_scale(const float* w, int c, float r, float (&f)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) f[i] = __fmul_rn(f[i], r);
  if (w) {
    const float4* w4 = reinterpret_cast<const float4*>(w) + static_cast<int64_t>(c) * (E / 4);
#pragma unroll
    for (int i = 0; i < E / 4; ++i) {
      const float4 t = __ldg(w4 + i);
      f[4 * i] = __fmul_rn(f[4 * i], t.x);
      f[4 * i + 1] = __fmul_rn(f[4 * i + 1], t.y);
      f[4 * i + 2] = __fmul_rn(f[4 * i + 2], t.z);
      f[4 * i + 3] = __fmul_rn(f[4 * i + 3], t.w);
    }
  }
}

template <int E>
__device__ __forceinline__ void norm_store_codes(int8_t* out, int c, float s, float (&f)[E],
                                                 int& sum) {
  uint32_t* o = reinterpret_cast<uint32_t*>(out + static_cast<int64_t>(c) * E);
  uint32_t w[E / 4];
#pragma unroll
  for (int i = 0; i < E / 4; ++i)
    w[i] = quant_pack4(make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]), s, sum);
  if constexpr (E == 8) {
    *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[1]);
  } else {
    o[0] = w[0];
  }
}

template <typename T, int kThreads, bool kGated>
static __global__ void __launch_bounds__(kThreads)
norm_quant_kernel(const __grid_constant__ NormParams p) {
  constexpr int E = kVec<T>;
  constexpr int R = kNormRegElems / E;
  constexpr int W = kThreads / 32;
  __shared__ double red_d[W];
  __shared__ uint32_t red_u[W];
  __shared__ int red_i[W];
  pdl_wait_prior_grid();
  pdl_allow_next_grid();
  const int64_t row = blockIdx.x;
  const T* a = static_cast<const T*>(p.a) + row * p.lda;
  const T* b = p.b ? static_cast<const T*>(p.b) + row * p.ldb : nullptr;
  T* h = p.h ? static_cast<T*>(p.h) + row * p.ldh : nullptr;
  int8_t* out = p.xq + row * p.K;
  const int C = p.K / E;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  float v[R][E];
  double ss = 0.0;
  auto square = [&](const float (&f)[E]) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const double d = static_cast<double>(f[i]);
      ss = fma(d, d, ss);
    }
  };
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int c = tid + j * kThreads;
    if (c < C) {
      norm_load<T, kGated>(p, a, b, h, c, true, v[j]);
      if (p.normalize) square(v[j]);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) v[j][i] = 0.0f;
    }
  }
  for (int c = tid + R * kThreads; c < C; c += kThreads) {
    float f[E];
    norm_load<T, kGated>(p, a, b, h, c, true, f);
    if (p.normalize) square(f);
  }

  float r = 1.0f;
  if (p.normalize) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    if (lane == 0) red_d[warp] = ss;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < W; ++w) t += red_d[w];
    r = static_cast<float>(1.0 / sqrt(t / static_cast<double>(p.K) + p.eps));
  }

  uint32_t top = 0;
  auto bits = [&](const float (&f)[E]) {
#pragma unroll
    for (int i = 0; i < E; ++i) top = max(top, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  };
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int c = tid + j * kThreads;
    if (c < C) {
      if (p.normalize) norm_scale(p.weight, c, r, v[j]);
      bits(v[j]);
    }
  }
  for (int c = tid + R * kThreads; c < C; c += kThreads) {
    float f[E];
    norm_load<T, kGated>(p, a, b, h, c, false, f);
    if (p.normalize) norm_scale(p.weight, c, r, f);
    bits(f);
  }
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if (lane == 0) red_u[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) top = max(top, red_u[w]);

  const bool finite = top < 0x7F800000u;
  const float amax = finite ? __uint_as_float(top) : __uint_as_float(0x7FC00000u);
  int sum = 0;
  if (top == 0u || !finite) {
    for (int c = tid; c < C; c += kThreads) {
      float z[E] = {};
      norm_store_codes<E>(out, c, 0.0f, z, sum);
    }
  } else {
    const float s = __fdiv_rn(127.0f, amax);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      const int c = tid + j * kThreads;
      if (c < C) norm_store_codes<E>(out, c, s, v[j], sum);
    }
    for (int c = tid + R * kThreads; c < C; c += kThreads) {
      float f[E];
      norm_load<T, kGated>(p, a, b, h, c, false, f);
      if (p.normalize) norm_scale(p.weight, c, r, f);
      norm_store_codes<E>(out, c, s, f, sum);
    }
  }
  if (tid == 0) p.amax[row] = amax;
  if (p.xsum) {
    sum = __reduce_add_sync(0xFFFFFFFFu, sum);
    if (lane == 0) red_i[warp] = sum;
    __syncthreads();
    if (tid == 0) {
      int t = 0;
#pragma unroll
      for (int w = 0; w < W; ++w) t += red_i[w];
      p.xsum[row] = t;
    }
  }
}

}  // namespace bl
