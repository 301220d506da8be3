// The join between two blocks for an fp32 stream and bf16 blocks.
#include "join_bwd.cuh"
#include "join_fwd.cuh"

namespace mlpb {

template cudaError_t join_fwd_run<float, __nv_bfloat16>(const JoinParams&, int, cudaStream_t);
template cudaError_t join_bwd_run<float, __nv_bfloat16>(
    const JoinParams&, const JoinShape&, bool, int, cudaStream_t);

}  // namespace mlpb
