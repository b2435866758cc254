// The second kernel of the layer for few tokens, on 4-bit weights.
#include "layer_small.cuh"

namespace moe {

cudaError_t launch_small_fp4_down(const SmallLayerParams& p, int sms, cudaStream_t stream) { return launch<true, false>(p, sms, stream); }

}  // namespace moe
