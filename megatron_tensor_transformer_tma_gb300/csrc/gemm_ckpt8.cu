// Instantiations of the tcgen05 GEMM whose saved activations are 8-bit checkpoints: fc1 writes
// the codes, dgrad reads them.
#include "gemm.cuh"
#include "kernels.h"

namespace mlpb {

template <GemmKind K>
static cudaError_t set_attr() {
  return cudaFuncSetAttribute(gemm_pair_kernel<K, false, true>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem);
}

// `clusters` clusters of kClusterM CTAs, one CTA per SM.
template <GemmKind K>
static cudaError_t launch_one(const CUtensorMap& a, const CUtensorMap& b, const GemmParams& p,
                              int clusters, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * kClusterM), 1, 1);
  cfg.blockDim = dim3(kGemmThreads, 1, 1);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kClusterM;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gemm_pair_kernel<K, false, true>, a, b, p);
}

cudaError_t gemm_ckpt8_set_smem_attrs() {
  cudaError_t e = cudaSuccess;
  if (e == cudaSuccess) e = set_attr<GemmKind::FC1_GELU>();
  if (e == cudaSuccess) e = set_attr<GemmKind::FC1_SWIGLU>();
  if (e == cudaSuccess) e = set_attr<GemmKind::DGRAD_GELU>();
  if (e == cudaSuccess) e = set_attr<GemmKind::DGRAD_SWIGLU>();
  return e;
}

cudaError_t launch_gemm_ckpt8(GemmKind kind, const CUtensorMap& a, const CUtensorMap& b,
                              const GemmParams& p, int clusters, cudaStream_t s) {
  switch (kind) {
    case GemmKind::FC1_GELU:
      return launch_one<GemmKind::FC1_GELU>(a, b, p, clusters, s);
    case GemmKind::FC1_SWIGLU:
      return launch_one<GemmKind::FC1_SWIGLU>(a, b, p, clusters, s);
    case GemmKind::DGRAD_GELU:
      return launch_one<GemmKind::DGRAD_GELU>(a, b, p, clusters, s);
    case GemmKind::DGRAD_SWIGLU:
      return launch_one<GemmKind::DGRAD_SWIGLU>(a, b, p, clusters, s);
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace mlpb
