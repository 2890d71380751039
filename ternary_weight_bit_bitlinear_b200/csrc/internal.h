// internal.h -- host-side pieces shared by the translation units of
// libbitlinear.so: per-device facts, the launch helper, and the launchers that
// each kernel family's unit (launch_*.cu) defines for the C ABI in
// bitlinear.cu.  Not part of the public interface.
//
// Each unit is compiled on its own (whole-program device code per unit), so
// the kernels of a family, their template instantiations and their device
// error word live in that unit only.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <utility>

#include "bitlinear.h"
#include "gemm.cuh"
#include "gemm_pair.cuh"
#include "gemm_split.cuh"
#include "gemv.cuh"
#include "gemv_quant.cuh"
#include "launch_facts.h"
#include "norm.cuh"
#include "tl2.cuh"

namespace blh {

constexpr int kMaxDevices = 64;

// A row kernel of norm.cuh: set up, and its CTAs per SM at the last
// shared-memory size asked about.
struct NormKernelInfo {
  FlagFact set{false};
  KeyedFact per_sm;   // by bytes of shared memory
};

// Per-device facts and one-time set-up flags, looked up once per device, by any
// host thread (launch_facts.h).
struct DeviceInfo {
  int sms = 0;
  FlagFact gemm_attr_set[8] = {};
  CountFact gemv_blocks_per_sm[bl::kGemvMaxTokens + 1] = {};   // 0: not set up yet
  CountFact tl2_blocks_per_sm[bl::kGemvMaxTokens + 1] = {};    // 0: not set up yet
  CountFact gq_max_dyn[bl::kGemvMaxTokens + 1] = {};   // dynamic shared memory limit
  KeyedFact gq_occ[bl::kGemvMaxTokens + 1][bl::kGqMaxWarps + 1];   // CTAs per SM, by bytes
  FlagFact gemv_split_attr_set[bl::kGemvMaxTokens + 1] = {};
  CountFact gemv_ep_blocks_per_sm[bl::kGemvEpMaxTokens + 1] = {};  // 0: not set up yet
  FlagFact gemv_ep_split_attr_set[bl::kGemvEpMaxTokens + 1] = {};
  NormKernelInfo norm[3][2][9];       // type, gated, width (launch_norm.cu)
  FlagFact split_attr_set[3] = {};    // gemm_split_kernel: 32, 64, 128 tokens
  CountFact split_clusters[3][3] = {};   // resident clusters of 1, 2, 4 pairs; 0: not asked yet
};

// The calling thread's current device.
bitlinear_status device_info(DeviceInfo** out);

// Wall-time limit every bounded wait of a launch uses (bitlinear_set_wait_limit).
unsigned long long wait_limit_ns();

// Launch with programmatic stream serialisation (see pdl_wait_prior_grid).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), int grid, int block, size_t smem,
                       cudaStream_t s, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(block));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

inline bitlinear_status launch_status() {
  return cudaGetLastError() == cudaSuccess ? BITLINEAR_OK : BITLINEAR_ERR_CUDA;
}

// ---- launchers, one unit per kernel family

// launch_gemv.cu: decode GEMV on int8 activations (tile or split-unit kernel).
bitlinear_status launch_gemv(int N, const bl::GemvParams& p, DeviceInfo* dev, cudaStream_t s);

// The few-token launch of bitlinear_linear (same kernels, with the epilogue),
// N <= kGemvEpMaxTokens.
bitlinear_status launch_gemv_ep(int N, const bl::GemvEpParams& p, DeviceInfo* dev,
                                cudaStream_t s);

// launch_norm.cu: row operators between two products.
bitlinear_status launch_norm(bool gated, int rows, int dtype, const bl::NormParams& p,
                             DeviceInfo* dev, cudaStream_t s);

// launch_gemv_quant.cu: the fused quantise + GEMV decode kernel.  CTAs of
// `warps` warps with `area` bytes of dynamic shared memory each.
bitlinear_status gemv_quant_occupancy(int N, int warps, int area, DeviceInfo* dev, int* out);
bitlinear_status gemv_quant_launch(int N, int grid, int warps, const bl::GqParams& p,
                                   cudaStream_t s);

// launch_gemm.cu: tensor-core GEMMs.  variant: 0 = 128-token tiles, 1 = CTA
// pairs, 3 = 64-token tiles (A unpacked into shared memory); 4 = 16 tokens,
// 5 = 32 tokens (A in tensor memory).
bitlinear_status launch_gemm(int variant, const bl::GemmParams& p, DeviceInfo* dev,
                             cudaStream_t s);

// The CTA-pair GEMM with an epilogue (bitlinear_linear, many tokens).
bitlinear_status launch_pair_ep(const bl::GemmEpParams& p, DeviceInfo* dev, cudaStream_t s);

// The cluster-split GEMM of bitlinear_linear, BN tokens per tile, S CTA pairs
// per cluster; split_clusters: how many such clusters the device holds at once.
bitlinear_status launch_split(int BN, int S, const bl::SplitParams& p, DeviceInfo* dev,
                              cudaStream_t s);
bitlinear_status split_clusters(int BN, int S, DeviceInfo* dev, int* out);

// launch_tl2.cu: TL2-style storage.
bitlinear_status launch_gemv_tl2(int N, const bl::Tl2Params& p, DeviceInfo* dev,
                                 cudaStream_t s);
bitlinear_status launch_tl2_convert(const uint32_t* packed, int64_t M, int64_t K, int wp,
                                    uint8_t* tl2, int grid, cudaStream_t s);

// Device error words, one per unit: read (and, with clear, reset) into *v.
cudaError_t device_error_gemv(unsigned int* v, bool clear);
cudaError_t device_error_gemv_quant(unsigned int* v, bool clear);
cudaError_t device_error_gemm(unsigned int* v, bool clear);
cudaError_t device_error_tl2(unsigned int* v, bool clear);
cudaError_t device_error_norm(unsigned int* v, bool clear);

// Shared body of the device_error_* readers (each unit passes its own symbol).
template <typename Sym>
cudaError_t read_error_word(const Sym& sym, unsigned int* v, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(v, sym, sizeof(unsigned int));
  if (e != cudaSuccess || !clear || *v == 0) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(sym, &zero, sizeof zero);
}

}  // namespace blh
