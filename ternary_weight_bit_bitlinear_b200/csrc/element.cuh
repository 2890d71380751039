// element.cuh -- element types of activation matrices (fp32, bf16, fp16) and
// the pointwise activations, shared by the kernels around the products
// (norm.cuh, epilogue.cuh).  Everything is computed in fp32: a value read is
// widened exactly, a value written is rounded once, to nearest even.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "bitlinear.h"

namespace bl {

template <typename T>
struct Elem;

template <>
struct Elem<float> {
  static __device__ __forceinline__ float to_float(float v) { return v; }
  static __device__ __forceinline__ float from_float(float v) { return v; }
};
template <>
struct Elem<__nv_bfloat16> {
  static __device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
  static __device__ __forceinline__ __nv_bfloat16 from_float(float v) {
    return __float2bfloat16_rn(v);
  }
};
template <>
struct Elem<__half> {
  static __device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
  static __device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }
};

// Elements of one 16-byte access.
template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));

template <typename T>
union Vec16 {
  uint4 u;
  T e[kVec<T>];
};

// max(v, 0) that keeps a NaN.
__device__ __forceinline__ float relu_nan(float v) {
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(v));
  return r;
}

// act(v), every operation a single fp32 rounding (no contraction):
//   relu   max(v, 0)          relu2  max(v, 0)^2
//   silu   v / (1 + e^-v)
//   gelu   0.5 v (1 + erf(v / sqrt 2))
//   gelu_tanh  0.5 v (1 + tanh(sqrt(2/pi) (v + 0.044715 v^3)))
// A NaN stays a NaN.
__device__ __forceinline__ float activate(float v, int act) {
  switch (act) {
    case BITLINEAR_ACT_RELU: return relu_nan(v);
    case BITLINEAR_ACT_RELU2: {
      const float r = relu_nan(v);
      return __fmul_rn(r, r);
    }
    case BITLINEAR_ACT_SILU: return __fdiv_rn(v, __fadd_rn(1.0f, expf(-v)));
    case BITLINEAR_ACT_GELU:
      return __fmul_rn(__fmul_rn(0.5f, v),
                       __fadd_rn(1.0f, erff(__fmul_rn(v, 0.7071067811865476f))));
    case BITLINEAR_ACT_GELU_TANH: {
      const float c = __fmul_rn(__fmul_rn(__fmul_rn(0.044715f, v), v), v);
      const float t = tanhf(__fmul_rn(0.7978845608028654f, __fadd_rn(v, c)));
      return __fmul_rn(__fmul_rn(0.5f, v), __fadd_rn(1.0f, t));
    }
    default: return v;
  }
}

// v / (1 + e^-t) without an overflow however far below zero t is: with
// e = e^-|t| it is v e / (1 + e) where t is negative and v / (1 + e) elsewhere.
// The divisor stays between 1 and 2, where the approximate division is within 2
// units in the last place (it gives 0 from 2^126 on).  kRefine adds one step of
// iterative refinement, q + (n - q d) / d with the residual from one fused
// operation, which leaves half a unit and a few 2^-21 of one (512 x 11008 x
// 4096, fp32 silu: 40.3 us without it, 44.8 with it, 55.0 with exact divisions,
// which spill in the GEMMs).  An infinite n stays as it is; t = v = -inf gives
// NaN.
template <bool kRefine>
__device__ __forceinline__ float times_sigmoid(float v, float t) {
  const float e = expf(-fabsf(t));
  const float n = t < 0.0f ? __fmul_rn(v, e) : v, d = __fadd_rn(1.0f, e);
  const float q = __fdividef(n, d);
  if (!kRefine) return q;
  const float r = __fmaf_rn(-q, d, n);
  return r == r ? __fadd_rn(q, __fdividef(r, d)) : q;
}

// act(v) behind a product.  silu as above with t = v; gelu_tanh in its form
// v / (1 + e^-2a), a the argument of tanh, which keeps the small values left of
// zero.  Outputs of 16 bits (kRefine false) take the approximate quotient:
// their own rounding covers it.
template <bool kRefine>
__device__ __forceinline__ float activate_product(float v, int act) {
  if (act == BITLINEAR_ACT_SILU) return times_sigmoid<kRefine>(v, v);
  if (act == BITLINEAR_ACT_GELU_TANH) {
    const float c = __fmul_rn(__fmul_rn(__fmul_rn(0.044715f, v), v), v);
    return times_sigmoid<kRefine>(v, __fmul_rn(2.0f * 0.7978845608028654f, __fadd_rn(v, c)));
  }
  return activate(v, act);
}

// activate over n values, the choice made once.
template <int n>
__device__ __forceinline__ void activate_exact_all(float (&f)[n], int act) {
  switch (act) {
#define BL_ACT_ALL(a)                                                       \
  case a: {                                                                 \
    _Pragma("unroll") for (int i = 0; i < n; ++i) f[i] = activate(f[i], a); \
    break;                                                                  \
  }
    BL_ACT_ALL(BITLINEAR_ACT_RELU)
    BL_ACT_ALL(BITLINEAR_ACT_RELU2)
    BL_ACT_ALL(BITLINEAR_ACT_SILU)
    BL_ACT_ALL(BITLINEAR_ACT_GELU)
    BL_ACT_ALL(BITLINEAR_ACT_GELU_TANH)
#undef BL_ACT_ALL
    default: break;
  }
}

// activate_product of n values that are stored as T, the choice made once.
template <typename T, int n>
__device__ __forceinline__ void activate_all(float (&f)[n], int act) {
  switch (act) {
#define BL_ACT_ALL(a)                                                          \
  case a: {                                                                    \
    _Pragma("unroll") for (int i = 0; i < n; ++i)                              \
        f[i] = activate_product<sizeof(T) == 4>(f[i], a);                      \
    break;                                                                     \
  }
    BL_ACT_ALL(BITLINEAR_ACT_RELU)
    BL_ACT_ALL(BITLINEAR_ACT_RELU2)
    BL_ACT_ALL(BITLINEAR_ACT_SILU)
    BL_ACT_ALL(BITLINEAR_ACT_GELU)
    BL_ACT_ALL(BITLINEAR_ACT_GELU_TANH)
#undef BL_ACT_ALL
    default: break;
  }
}

}  // namespace bl
