// The join between two blocks for an fp32 stream and fp32 blocks.
#include "join_bwd.cuh"
#include "join_fwd.cuh"

namespace mlpb {

template cudaError_t join_fwd_run<float, float>(const JoinParams&, int, cudaStream_t);
template cudaError_t join_bwd_run<float, float>(
    const JoinParams&, const JoinShape&, bool, int, cudaStream_t);

}  // namespace mlpb
