// What the handles of the linear layer and of the updates share on the host: sizes, the device they
// are made on, tensor maps, the device error word.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "../../include/mlpb.h"

namespace mlpb {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct PlanDevice {
  int device;
  uint32_t* err;  // the device error word
  PFN_cuTensorMapEncodeTiled_v12000 encode;

  // The current device, which has to be an sm_103.
  mlpb_status find() {
    err = nullptr;
    int major = 0, minor = 0;
    if (cudaGetDevice(&device) != cudaSuccess ||
        cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, device) != cudaSuccess)
      return MLPB_ECUDA;
    if (major != 10 || minor != 3) return MLPB_EUNSUPPORTED;
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess || fn == nullptr)
      return MLPB_ECUDA;
    encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
    return MLPB_OK;
  }

  // The error word, cleared; synchronised, since streams that do not wait for that may come.
  mlpb_status allocate() {
    if (cudaMalloc(reinterpret_cast<void**>(&err), sizeof(uint32_t)) != cudaSuccess) {
      err = nullptr;
      return MLPB_ECUDA;
    }
    if (cudaMemset(err, 0, sizeof(uint32_t)) == cudaSuccess &&
        cudaStreamSynchronize(nullptr) == cudaSuccess)
      return MLPB_OK;
    release();
    return MLPB_ECUDA;
  }

  void release() {
    if (err) cudaFree(err);
    err = nullptr;
  }

  // Whether the current device is this one: a call's stream would not be one of its otherwise.
  mlpb_status current() const {
    int now = -1;
    if (cudaGetDevice(&now) != cudaSuccess) return MLPB_ECUDA;
    return now == device ? MLPB_OK : MLPB_EINVAL;
  }

  // Reads and clears the error word in order with `s`.
  mlpb_status last_error(cudaStream_t s) const {
    const mlpb_status st = current();
    if (st != MLPB_OK) return st;
    uint32_t v = 0;
    if (cudaMemcpyAsync(&v, err, sizeof(v), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
      return MLPB_ECUDA;
    if (v == 0) return MLPB_OK;
    if (cudaMemsetAsync(err, 0, sizeof(uint32_t), s) != cudaSuccess ||
        cudaStreamSynchronize(s) != cudaSuccess)
      return MLPB_ECUDA;
    return MLPB_ETIMEOUT;
  }

  // Tiles of a tensor of `rank` (2 to 4) dimensions; what is past its edges reads zero.
  bool map(CUtensorMap* m, CUtensorMapDataType type, const void* base, int rank,
           const cuuint64_t* dims, const cuuint64_t* strides, const cuuint32_t* box,
           CUtensorMapSwizzle swizzle) const {
    const cuuint32_t steps[4] = {1, 1, 1, 1};
    return encode(m, type, static_cast<cuuint32_t>(rank), const_cast<void*>(base), dims, strides,
                  box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
};

}  // namespace mlpb
