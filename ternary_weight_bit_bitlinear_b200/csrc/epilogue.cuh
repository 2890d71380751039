// epilogue.cuh -- what bitlinear_linear does with an accumulator before it is
// stored: bias, activation, residual, one rounding to the output's type.
//
//   y[n, m] = T(act(acc * (alpha * (amax[n] / 127)) + bias[m]) + residual[n, m])
//
// Every fp32 operation is rounded on its own; the tensor-core kernels divide
// approximately in silu and gelu_tanh of a 16-bit output (activate_product).
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
  int vec;                 // 1: rows of y, residual and bias can be accessed 16 bytes at a time
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
  v = activate_product<true>(v, e.act);   // one form for all types: less code in a short launch
  if (e.residual) v = __fadd_rn(v, ep_load(e.residual, n * e.ldr + m, e.dtype));
  ep_store(e.y, n * e.ldy + m, e.dtype, v);
}

// One warp's part of a GEMM epilogue: blocks of kTokens tokens x 32 weight
// rows, the rescaled accumulators staged in shared memory as blk[token][row].
// Tensor memory gives each lane one weight row of all tokens; the outputs are
// token-major, so the second half of the work takes 16-byte pieces of a
// token's 32 rows instead: 8 lanes (fp32) or 4 lanes (16-bit) per token, all
// residual loads of a block in flight at once, and those of the next block
// while this one is finished.  Blocks that reach past M, and rows that are not
// on 16 bytes, go element by element, a lane per row, eight loads at a time.
// Measured in the BN = 256 kernel (11008 x 4096, 512 tokens, bf16): 33.9 us
// against 77.3 with one element per lane and step; the product with plain fp32
// stores takes 32.5.
template <typename T, int kTokens>
struct EpRows {
  static constexpr int E = kVec<T>;
  static constexpr int kLanes = 32 / E;          // lanes per token
  static constexpr int kStep = 32 / kLanes;      // tokens per iteration
  static constexpr int kIters = kTokens / kStep;
  uint4 res[kIters];                             // residual of the block to finish
  float bias[E];
  int m, lane;                                   // this lane's first row (vector path)
  bool vec, full;

  // Rows m0 .. m0+31 of a layer of M.
  __device__ __forceinline__ void begin(const Epilogue& e, int m0, int M, int lane_) {
    lane = lane_;
    full = m0 + 32 <= M;
    vec = e.vec && full;
    m = vec ? m0 + (lane % kLanes) * E : m0 + lane;
#pragma unroll
    for (int i = 0; i < E; ++i) bias[i] = 0.0f;
    if (e.bias) {
      if (vec) {
#pragma unroll
        for (int i = 0; i < E; i += 4) {
          const float4 b = __ldg(reinterpret_cast<const float4*>(e.bias + m + i));
          bias[i] = b.x, bias[i + 1] = b.y, bias[i + 2] = b.z, bias[i + 3] = b.w;
        }
      } else if (m < M) {
        bias[0] = __ldg(e.bias + m);
      }
    }
  }

  // Residual of tokens n0 .. (those before N) into `to`.
  __device__ __forceinline__ void load(const Epilogue& e, int n0, int N, uint4 (&to)[kIters]) {
    if (!vec || !e.residual) return;
    const T* r = static_cast<const T*>(e.residual) + m;
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const int n = n0 + i * kStep + lane / kLanes;
      if (n < N) to[i] = *reinterpret_cast<const uint4*>(r + static_cast<int64_t>(n) * e.ldr);
    }
  }

  __device__ __forceinline__ void finish(const Epilogue& e, const float* blk, int n0, int N,
                                         int M) {
    if (vec) {
      T* y = static_cast<T*>(e.y) + m;
#pragma unroll
      for (int i = 0; i < kIters; ++i) {
        const int t = i * kStep + lane / kLanes;
        if (n0 + t < N) {
          float f[E];
          const float4* src = reinterpret_cast<const float4*>(blk + t * 32 + (lane % kLanes) * E);
          if constexpr (E == 4) {
            const float4 v = src[0];
            f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
          } else {   // odd tokens read their second half first: no bank conflict
            const int o = (lane / kLanes) & 1;
            const float4 a = src[o], b = src[o ^ 1];
            const float4 lo = o ? b : a, hi = o ? a : b;
            f[0] = lo.x, f[1] = lo.y, f[2] = lo.z, f[3] = lo.w;
            f[4] = hi.x, f[5] = hi.y, f[6] = hi.z, f[7] = hi.w;
          }
          if (e.bias) {
#pragma unroll
            for (int q = 0; q < E; ++q) f[q] = __fadd_rn(f[q], bias[q]);
          }
          activate_all<T>(f, e.act);
          Vec16<T> v;
          v.u = res[i];
#pragma unroll
          for (int q = 0; q < E; ++q)
            v.e[q] = Elem<T>::from_float(
                e.residual ? __fadd_rn(f[q], Elem<T>::to_float(v.e[q])) : f[q]);
          *reinterpret_cast<uint4*>(y + static_cast<int64_t>(n0 + t) * e.ldy) = v.u;
        }
      }
      return;
    }
    if (m >= M) return;
    const T* r = static_cast<const T*>(e.residual) + static_cast<int64_t>(n0) * e.ldr + m;
    T* y = static_cast<T*>(e.y) + static_cast<int64_t>(n0) * e.ldy + m;
    const int nt = min(kTokens, N - n0);
#pragma unroll 1
    for (int j0 = 0; j0 < nt; j0 += 8) {
      float f[8], g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        f[j] = j0 + j < kTokens ? blk[(j0 + j) * 32 + lane] : 0.0f;
        g[j] = 0.0f;
        if (e.residual) {
          if (j0 + j < nt) g[j] = Elem<T>::to_float(*r);
          r += e.ldr;
        }
        if (e.bias) f[j] = __fadd_rn(f[j], bias[0]);
      }
      activate_all<T>(f, e.act);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j0 + j < nt) *y = Elem<T>::from_float(e.residual ? __fadd_rn(f[j], g[j]) : f[j]);
        y += e.ldy;
      }
    }
  }
};

// f(T{}) for the epilogue's element type.
template <class F>
__device__ __forceinline__ void ep_dispatch(int dtype, F&& f) {
  if (dtype == BITLINEAR_F32)
    f(float{});
  else if (dtype == BITLINEAR_BF16)
    f(__nv_bfloat16{});
  else
    f(__half{});
}

}  // namespace bl
