// Scored, group-limited routing of fp32 logits (compiled in a unit of its own).
#include "route_kernels.cuh"

namespace moe {

cudaError_t launch_route_fwd_fp32(const RouteParams& p, int sms, cudaStream_t stream) { return fwd_elem<Fp32>(p, sms, stream); }

cudaError_t launch_route_bwd_fp32(const RouteBwdParams& p, int sms, cudaStream_t stream) { return bwd_elem<Fp32>(p, sms, stream); }

}  // namespace moe
