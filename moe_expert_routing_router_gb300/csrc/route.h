// Launchers of the scored, group-limited routing and its gradient (route_kernels.cuh, per logit type).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kRouteLanes = 32;         // lanes that hold a row; at most as many groups

struct RouteParams {
  const void* logits;     // [T, E]
  int64_t T;
  int E, k;
  int softmax;            // scores: 0 sigmoid, 1 softmax
  int G, gs, keep;        // groups, experts per group, groups a token may use
  int top2;               // a group's score: 0 its largest choice value, 1 the sum of its two largest
  int L, chunk;           // of a warp a row (the double-precision path): lanes per group (a power of two), experts per lane
  int tshift, tchunk;     // of the kernel's lanes a row: logarithm of the lanes per group, experts per lane
  const float* bias;      // [E] or null
  int renorm;
  float scale;
  float bias_gamma;
  float* bias_out;        // [E] or null
  int32_t* idx;           // [T, k]
  float* gate;            // [T, k]
  int32_t* counts;        // [E]
};

cudaError_t launch_route_fwd_bf16(const RouteParams& p, int sms, cudaStream_t stream);
cudaError_t launch_route_fwd_fp32(const RouteParams& p, int sms, cudaStream_t stream);

struct RouteBwdParams {
  const void* logits;     // [T, E]
  int64_t T;
  int E, k;
  int softmax, renorm;
  float scale;
  const int32_t* idx;     // [T, k]
  const float* dgate;     // [T, k]
  float* dlogits;         // [T, E]
};

cudaError_t launch_route_bwd_bf16(const RouteBwdParams& p, int sms, cudaStream_t stream);
cudaError_t launch_route_bwd_fp32(const RouteBwdParams& p, int sms, cudaStream_t stream);

}  // namespace moe
