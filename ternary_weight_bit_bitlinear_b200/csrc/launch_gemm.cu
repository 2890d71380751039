// launch_gemm.cu -- launchers of the tensor-core GEMMs (gemm.cuh: one CTA per
// 128-row tile; gemm_pair.cuh: CTA pairs per 256 x 256 tile; gemm_small.cuh:
// A in tensor memory for up to 32 tokens).
#include "internal.h"
#include "gemm_small.cuh"

namespace blh {
namespace {

template <int BN, int STAGES>
bitlinear_status launch_single(const bl::GemmParams& p, DeviceInfo* dev, int slot,
                               cudaStream_t s) {
  auto kernel = bl::gemm_i8_tcgen05_kernel<BN, STAGES>;
  const int smem = static_cast<int>(sizeof(bl::GemmSmem<BN, STAGES>)) + 1024;
  if (!dev->gemm_attr_set[slot]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
        cudaSuccess)
      return BITLINEAR_ERR_CUDA;
    dev->gemm_attr_set[slot] = true;
  }
  const int grid = p.total_tiles < dev->sms ? p.total_tiles : dev->sms;
  if (launch_pdl(kernel, grid, bl::kGemmThreads, smem, s, p) != cudaSuccess)
    return BITLINEAR_ERR_CUDA;
  return launch_status();
}

// CTA-pair GEMM for wide token blocks: two CTAs (a compile-time cluster) per
// 256 x 256 tile, one pair per two SMs.
template <int STAGES, class P>
bitlinear_status launch_pair(const P& p, DeviceInfo* dev, cudaStream_t s) {
  constexpr int slot = P::kEpilogue ? 2 : 1;
  auto kernel = bl::gemm_i8_pair_kernel<STAGES, P>;
  const int smem = static_cast<int>(sizeof(bl::GemmPairSmem<STAGES>)) + 1024;
  if (!dev->gemm_attr_set[slot]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
        cudaSuccess)
      return BITLINEAR_ERR_CUDA;
    dev->gemm_attr_set[slot] = true;
  }
  const int pairs = p.total_tiles < dev->sms / 2 ? p.total_tiles : dev->sms / 2;
  if (launch_pdl(kernel, 2 * pairs, bl::kGemmThreads, smem, s, p) != cudaSuccess)
    return BITLINEAR_ERR_CUDA;
  return launch_status();
}

template <int BN>
bitlinear_status launch_small(const bl::GemmParams& p, DeviceInfo* dev, int slot,
                              cudaStream_t s) {
  auto kernel = bl::gemm_small_kernel<BN>;
  const int smem = static_cast<int>(sizeof(bl::SmallSmem<BN>)) + 1024;
  if (!dev->gemm_attr_set[slot]) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
        cudaSuccess)
      return BITLINEAR_ERR_CUDA;
    dev->gemm_attr_set[slot] = true;
  }
  const int grid = p.total_tiles < dev->sms ? p.total_tiles : dev->sms;
  if (launch_pdl(kernel, grid, bl::kSmallThreads, smem, s, p) != cudaSuccess)
    return BITLINEAR_ERR_CUDA;
  return launch_status();
}

}  // namespace

bitlinear_status launch_gemm(int variant, const bl::GemmParams& p, DeviceInfo* dev,
                             cudaStream_t s) {
  switch (variant) {
    case 0: return launch_single<128, 7>(p, dev, 0, s);
    case 1: return launch_pair<5>(p, dev, s);
    case 3: return launch_single<64, 12>(p, dev, 3, s);
    case 4: return launch_small<16>(p, dev, 4, s);
    case 5: return launch_small<32>(p, dev, 5, s);
    default: return BITLINEAR_ERR_UNSUPPORTED_SHAPE;
  }
}

bitlinear_status launch_pair_ep(const bl::GemmEpParams& p, DeviceInfo* dev, cudaStream_t s) {
  return launch_pair<5>(p, dev, s);
}

namespace {

// Index of the tile width (32, 64, 128) and of the pairs per cluster (1, 2, 4).
int split_width(int BN) { return BN == 32 ? 0 : BN == 64 ? 1 : 2; }
int split_size(int S) { return S == 1 ? 0 : S == 2 ? 1 : 2; }

struct SplitLaunch {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
};

template <int BN>
bitlinear_status split_config(int grid, int S, DeviceInfo* dev, cudaStream_t s, SplitLaunch& l) {
  const int smem = static_cast<int>(sizeof(bl::SplitSmem<BN>)) + 1024;
  FlagFact& set = dev->split_attr_set[split_width(BN)];
  if (!set) {
    if (cudaFuncSetAttribute(bl::gemm_split_kernel<BN>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
      return BITLINEAR_ERR_CUDA;
    set = true;
  }
  l.cfg.gridDim = dim3(static_cast<unsigned>(grid));
  l.cfg.blockDim = dim3(bl::kSplitThreads);
  l.cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  l.cfg.stream = s;
  l.attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  l.attr[0].val.programmaticStreamSerializationAllowed = 1;
  l.attr[1].id = cudaLaunchAttributeClusterDimension;
  l.attr[1].val.clusterDim.x = static_cast<unsigned>(2 * S);
  l.attr[1].val.clusterDim.y = 1;
  l.attr[1].val.clusterDim.z = 1;
  l.cfg.attrs = l.attr;
  l.cfg.numAttrs = 2;
  return BITLINEAR_OK;
}

template <int BN>
bitlinear_status launch_split_width(int S, const bl::SplitParams& p, DeviceInfo* dev,
                                    cudaStream_t s) {
  int clusters = 0;
  bitlinear_status st = split_clusters(BN, S, dev, &clusters);
  if (st != BITLINEAR_OK) return st;
  SplitLaunch l;
  st = split_config<BN>(2 * S * (p.total_tiles < clusters ? p.total_tiles : clusters), S, dev, s, l);
  if (st != BITLINEAR_OK) return st;
  if (cudaLaunchKernelEx(&l.cfg, bl::gemm_split_kernel<BN>, p) != cudaSuccess)
    return BITLINEAR_ERR_CUDA;
  return launch_status();
}

template <int BN>
bitlinear_status ask_clusters(int S, DeviceInfo* dev, int* out) {
  SplitLaunch l;
  const bitlinear_status st = split_config<BN>(2 * S, S, dev, nullptr, l);
  if (st != BITLINEAR_OK) return st;
  if (cudaOccupancyMaxActiveClusters(out, bl::gemm_split_kernel<BN>, &l.cfg) != cudaSuccess ||
      *out < 1)
    return BITLINEAR_ERR_CUDA;
  return BITLINEAR_OK;
}

}  // namespace

bitlinear_status split_clusters(int BN, int S, DeviceInfo* dev, int* out) {
  CountFact& known = dev->split_clusters[split_width(BN)][split_size(S)];
  int n = known;
  if (n == 0) {
    const bitlinear_status st = BN == 32   ? ask_clusters<32>(S, dev, &n)
                                : BN == 64 ? ask_clusters<64>(S, dev, &n)
                                           : ask_clusters<128>(S, dev, &n);
    if (st != BITLINEAR_OK) return st;
    known = n;
  }
  *out = n;
  return BITLINEAR_OK;
}

bitlinear_status launch_split(int BN, int S, const bl::SplitParams& p, DeviceInfo* dev,
                              cudaStream_t s) {
  switch (BN) {
    case 32: return launch_split_width<32>(S, p, dev, s);
    case 64: return launch_split_width<64>(S, p, dev, s);
    default: return launch_split_width<128>(S, p, dev, s);
  }
}

cudaError_t device_error_gemm(unsigned int* v, bool clear) {
  return read_error_word(bl::g_device_error, v, clear);
}

}  // namespace blh
