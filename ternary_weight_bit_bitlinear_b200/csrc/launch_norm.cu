// launch_norm.cu -- launchers of the row operators between two products
// (norm.cuh): norm + int8 output, gated activation + norm + int8 output.
#include "internal.h"
#include "norm.cuh"

namespace blh {
namespace {

template <typename T, bool kGated>
bitlinear_status launch_norm_type(int rows, const bl::NormParams& p, cudaStream_t s) {
  // The fewest threads that hold the row in registers.
  cudaError_t e;
  if (p.K <= 128 * bl::kNormRegElems)
    e = launch_pdl(bl::norm_quant_kernel<T, 128, kGated>, rows, 128, 0, s, p);
  else if (p.K <= 256 * bl::kNormRegElems)
    e = launch_pdl(bl::norm_quant_kernel<T, 256, kGated>, rows, 256, 0, s, p);
  else if (p.K <= 512 * bl::kNormRegElems)
    e = launch_pdl(bl::norm_quant_kernel<T, 512, kGated>, rows, 512, 0, s, p);
  else
    e = launch_pdl(bl::norm_quant_kernel<T, 1024, kGated>, rows, 1024, 0, s, p);
  return e == cudaSuccess ? launch_status() : BITLINEAR_ERR_CUDA;
}

template <bool kGated>
bitlinear_status launch_norm_any(int rows, int dtype, const bl::NormParams& p, cudaStream_t s) {
  switch (dtype) {
    case BITLINEAR_F32: return launch_norm_type<float, kGated>(rows, p, s);
    case BITLINEAR_BF16: return launch_norm_type<__nv_bfloat16, kGated>(rows, p, s);
    default: return launch_norm_type<__half, kGated>(rows, p, s);
  }
}

}  // namespace

bitlinear_status launch_norm(bool gated, int rows, int dtype, const bl::NormParams& p,
                             cudaStream_t s) {
  return gated ? launch_norm_any<true>(rows, dtype, p, s)
               : launch_norm_any<false>(rows, dtype, p, s);
}

}  // namespace blh
