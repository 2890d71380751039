// launch_norm.cu -- launchers of the row operators between two products
// (norm.cuh): norm + int8 output, gated activation + norm + int8 output.
#include "internal.h"
#include "norm.cuh"

namespace blh {
namespace {

// Rows up to kElems * kThreads wide: one CTA per row at a time, as many CTAs as
// are resident.
template <typename T, int kThreads, int kElems, bool kGated>
bitlinear_status launch_stream(int rows, const bl::NormParams& p, NormKernelInfo& known, int sms,
                               cudaStream_t s) {
  auto kernel = bl::norm_stream_kernel<T, kThreads, kElems, kGated>;
  constexpr int most = 2 * kThreads * kElems * static_cast<int>(sizeof(T));
  const int smem = p.K * static_cast<int>(sizeof(T)) * (kGated || p.b ? 2 : 1);
  if (!known.set) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) !=
        cudaSuccess)
      return BITLINEAR_ERR_CUDA;
    known.set = true;
  }
  int grid = rows;
  if (rows > sms) {
    int per_sm = 0;
    if (!known.per_sm.get(smem, &per_sm)) {
      if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, smem) !=
              cudaSuccess ||
          per_sm < 1)
        return BITLINEAR_ERR_CUDA;
      known.per_sm.set(smem, per_sm);
    }
    if (grid > sms * per_sm) grid = sms * per_sm;
  }
  if (launch_pdl(kernel, grid, kThreads, smem, s, p, rows) != cudaSuccess)
    return BITLINEAR_ERR_CUDA;
  return launch_status();
}

// Wider rows: a cluster of C CTAs per row, at most 2^31 - 1 CTAs per launch.
template <typename T, int kThreads, int kElems, bool kGated>
bitlinear_status launch_cluster(int64_t rows, int C, bl::NormParams p, cudaStream_t s) {
  p.slice = (p.K / bl::kVec<T> + C - 1) / C;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(C);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  constexpr int64_t most = int64_t(1) << 27;
  for (int64_t done = 0; done < rows; done += most) {
    const int64_t n = rows - done < most ? rows - done : most;
    bl::NormParams q = p;
    q.a = static_cast<const T*>(p.a) + done * p.lda;
    if (p.b) q.b = static_cast<const T*>(p.b) + done * p.ldb;
    if (p.h) q.h = static_cast<T*>(p.h) + done * p.ldh;
    q.xq = p.xq + done * p.K;
    q.amax = p.amax + done;
    if (p.xsum) q.xsum = p.xsum + done;
    cfg.gridDim = dim3(static_cast<unsigned>(n * C));
    if (cudaLaunchKernelEx(&cfg, bl::norm_quant_kernel<T, kThreads, kElems, kGated>, q) != cudaSuccess)
      return BITLINEAR_ERR_CUDA;
  }
  return launch_status();
}

// The narrowest CTA that holds a row in registers (one warp more costs every
// row its share of the reductions: 2048 x 4096 bf16 with 128 / 256 / 512
// threads 14.6 / 17.7 / 29.7 us), with few registers a thread past the row's
// end (their zeros run through all of the arithmetic: 2048 x 2560 bf16 in
// 160 threads of 16 values 10.2 us, in 128 of 32 12.2; 512 rows 4.7 and 5.6).
// Up to 12288 elements of 16 bits two CTAs of 256 threads with 48 values each
// take turns at the steps that wait, against one of 512 with 24, whose SM waits
// with it (gate and up 512 x 11008: 11.3 and 13.5 us, 2048: 30.6 and
// 39.8); one row for an SM (64: 7.5 and 5.9) and fp32 (2048: 51.5 and 49.0)
// take the wide one.  The same trade at other widths: no gain at 2048 rows of
// 5120 to 8192, 1.1 times the time at 14336 and 16384 (64 values).
// From 16384 elements on that would be 1024 threads of 64 registers, which
// spill: clusters there, of 8 CTAs while the rows leave SMs idle (one row of
// 28672: 4.0 us; 256 rows: 31 with 4 x 256 threads, 49 with 8 x 512), and
// where 4 x 256 threads do not hold the row.
template <typename T, bool kGated>
bitlinear_status launch_norm_type(int rows, const bl::NormParams& p, DeviceInfo* dev, int type,
                                  cudaStream_t s) {
  NormKernelInfo* known = dev->norm[type][kGated ? 1 : 0];
  const int K = p.K, sms = dev->sms;
  if (K <= 1024) return launch_stream<T, 128, 8, kGated>(rows, p, known[0], sms, s);
  if (K <= 2048) return launch_stream<T, 128, 16, kGated>(rows, p, known[1], sms, s);
  if (K <= 2560) return launch_stream<T, 160, 16, kGated>(rows, p, known[2], sms, s);
  if (K <= 4096) return launch_stream<T, 128, 32, kGated>(rows, p, known[3], sms, s);
  if (K <= 6144) return launch_stream<T, 256, 24, kGated>(rows, p, known[4], sms, s);
  if (K <= 8192) return launch_stream<T, 256, 32, kGated>(rows, p, known[5], sms, s);
  if constexpr (sizeof(T) == 2) {
    if (K <= 12288 && rows > sms)
      return launch_stream<T, 256, 48, kGated>(rows, p, known[8], sms, s);
  }
  if (K <= 12288) return launch_stream<T, 512, 24, kGated>(rows, p, known[6], sms, s);
  if (K <= 16384) return launch_stream<T, 512, 32, kGated>(rows, p, known[7], sms, s);
  if (K <= 32768 && rows * int64_t(8) > sms)
    return launch_cluster<T, 256, 32, kGated>(rows, 4, p, s);
  if (K <= 32768) return launch_cluster<T, 512, 8, kGated>(rows, 8, p, s);
  if (K <= 65536) return launch_cluster<T, 512, 16, kGated>(rows, 8, p, s);
  return launch_cluster<T, 512, 32, kGated>(rows, 8, p, s);
}

template <bool kGated>
bitlinear_status launch_norm_any(int rows, int dtype, const bl::NormParams& p, DeviceInfo* dev,
                                 cudaStream_t s) {
  switch (dtype) {
    case BITLINEAR_F32: return launch_norm_type<float, kGated>(rows, p, dev, 0, s);
    case BITLINEAR_BF16: return launch_norm_type<__nv_bfloat16, kGated>(rows, p, dev, 1, s);
    default: return launch_norm_type<__half, kGated>(rows, p, dev, 2, s);
  }
}

}  // namespace

bitlinear_status launch_norm(bool gated, int rows, int dtype, const bl::NormParams& p,
                             DeviceInfo* dev, cudaStream_t s) {
  return gated ? launch_norm_any<true>(rows, dtype, p, dev, s)
               : launch_norm_any<false>(rows, dtype, p, dev, s);
}

cudaError_t device_error_norm(unsigned int* v, bool clear) {
  return read_error_word(bl::g_device_error, v, clear);
}

}  // namespace blh
