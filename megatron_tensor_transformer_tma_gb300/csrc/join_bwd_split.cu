// Backward of the join where the stream or the block's tensors are fp32.
#include "join_bwd.cuh"

namespace mlpb {

template <class XT, class YT>
static cudaError_t by_norm(const JoinParams& p, int grid, cudaStream_t s) {
  return p.post == MLPB_NORM_LAYER || p.pre == MLPB_NORM_LAYER
             ? join_bwd_pick<XT, YT, true>(p, grid, s)
             : join_bwd_pick<XT, YT, false>(p, grid, s);
}

cudaError_t launch_join_bwd_split(const JoinParams& p, bool x32, bool y32, int grid,
                                  cudaStream_t s) {
  using bf = __nv_bfloat16;
  if (x32 && y32) return by_norm<float, float>(p, grid, s);
  return x32 ? by_norm<float, bf>(p, grid, s) : by_norm<bf, float>(p, grid, s);
}

}  // namespace mlpb
