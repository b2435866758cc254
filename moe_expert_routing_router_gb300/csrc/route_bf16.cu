// Scored, group-limited routing of bf16 logits (compiled in a unit of its own).
#include "route_kernels.cuh"

namespace moe {

cudaError_t launch_route_fwd_bf16(const RouteParams& p, int sms, cudaStream_t stream) { return fwd_elem<Bf16>(p, sms, stream); }

cudaError_t launch_route_bwd_bf16(const RouteBwdParams& p, int sms, cudaStream_t stream) { return bwd_elem<Bf16>(p, sms, stream); }

}  // namespace moe
