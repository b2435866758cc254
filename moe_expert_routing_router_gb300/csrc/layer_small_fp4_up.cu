// The first kernel of the layer for few tokens, on 4-bit weights.
#include "layer_small.cuh"

namespace moe {

cudaError_t launch_small_fp4_up(const SmallLayerParams& p, int sms, cudaStream_t stream) { return launch<true, true>(p, sms, stream); }

}  // namespace moe
