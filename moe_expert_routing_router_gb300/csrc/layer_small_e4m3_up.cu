// The first kernel of the layer for few tokens, on 8-bit weights.
#include "layer_small.cuh"

namespace moe {

cudaError_t launch_small_e4m3_up(const SmallLayerParams& p, int sms, cudaStream_t stream) { return launch<false, true>(p, sms, stream); }

}  // namespace moe
