// epilogue.cuh -- what bitlinear_linear does with an accumulator before it is
// stored: bias, activation, residual, one rounding to the output's type.
//
//   y[n, m] = T(act(acc * (alpha * (amax[n] / 127)) + bias[m]) + residual[n, m])
//
// Every fp32 operation is rounded on its own.
#pragma once

#include "element.cuh"

namespace bl {

struct Epilogue {
  const float* bias;       // [M] or null
  const void* residual;    // [N, M], row stride ldr, or null
  void* y;                 // [N, M], row stride ldy
  long long ldr, ldy;
  int dtype;               // of residual and y
  int act;
};

__device__ __forceinline__ float ep_load(const void* p, int64_t o, int dtype) {
  if (dtype == BITLINEAR_F32) return static_cast<const float*>(p)[o];
  if (dtype == BITLINEAR_BF16)
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[o]);
  return __half2float(static_cast<const __half*>(p)[o]);
}

__device__ __forceinline__ void ep_store(void* p, int64_t o, int dtype, float v) {
  if (dtype == BITLINEAR_F32)
    static_cast<float*>(p)[o] = v;
  else if (dtype == BITLINEAR_BF16)
    static_cast<__nv_bfloat16*>(p)[o] = __float2bfloat16_rn(v);
  else
    static_cast<__half*>(p)[o] = __float2half_rn(v);
}

// Element (n, m) from its rescaled accumulator v.
__device__ __forceinline__ void ep_element(const Epilogue& e, int64_t n, int m, float v) {
  if (e.bias) v = __fadd_rn(v, __ldg(e.bias + m));
  v = activate(v, e.act);
  if (e.residual) v = __fadd_rn(v, ep_load(e.residual, n * e.ldr + m, e.dtype));
  ep_store(e.y, n * e.ldy + m, e.dtype, v);
}

}  // namespace bl
