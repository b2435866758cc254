// The layer for few tokens: its scratch, and the choice of its kernels (layer_small.cuh).
#include "layer_small.h"

#include "device_common.cuh"

#include <cuda_bf16.h>

namespace moe {
namespace {

// out_t = sum_j gate_tj y_tj in the order of j: four columns a thread.  It is launched while the second
// kernel ends, and spreads the sums over the SMs.  (Joined in that kernel, by the CTA that completed a
// block of columns, they took up to 35 us for 64 tokens: the last CTAs complete most blocks.)
constexpr int kJoinThreads = 128;

__global__ void __launch_bounds__(kJoinThreads) small_join_kernel(const __grid_constant__ SmallLayerParams p) {
  const int t = blockIdx.y, c = (blockIdx.x * kJoinThreads + threadIdx.x) * 4;
  if (c >= p.H) return;
  float g[8];
  bool some[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int e = j < p.k ? p.idx[t * p.k + j] : -1;
    some[j] = e >= 0 && e < p.E;
    g[j] = some[j] ? p.gate[t * p.k + j] : 0.f;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float4 v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    v[j] = some[j] ? __ldcg(reinterpret_cast<const float4*>(p.y + int64_t(t * p.k + j) * p.H + c)) : make_float4(0.f, 0.f, 0.f, 0.f);
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    sum.x = fmaf(g[j], v[j].x, sum.x);
    sum.y = fmaf(g[j], v[j].y, sum.y);
    sum.z = fmaf(g[j], v[j].z, sum.z);
    sum.w = fmaf(g[j], v[j].w, sum.w);
  }
  const __nv_bfloat162 lo = __floats2bfloat162_rn(sum.x, sum.y), hi = __floats2bfloat162_rn(sum.z, sum.w);
  *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + int64_t(t) * p.H + c) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

cudaError_t launch_join(const SmallLayerParams& p, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((p.H / 4 + kJoinThreads - 1) / kJoinThreads), unsigned(p.T));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, small_join_kernel, p);
}

size_t up_to(size_t n) { return (n + 255) / 256 * 256; }   // pieces of the scratch

}  // namespace

size_t small_layer_work_size(int T, int H, int I, int k) {
  const size_t A = size_t(T) * k;
  return up_to(A * I * 4) + up_to(A * H * 4);
}

void small_layer_work(SmallLayerParams& p, void* work) {
  const size_t A = size_t(p.T) * p.k;
  char* at = static_cast<char*>(work);
  p.h = reinterpret_cast<float*>(at);
  p.y = reinterpret_cast<float*>(at + up_to(A * p.I * 4));
}

cudaError_t launch_layer_small(const SmallLayerParams& p, int sms, cudaStream_t stream) {
  cudaError_t e = p.w1.fp4 ? launch_small_fp4_up(p, sms, stream) : launch_small_e4m3_up(p, sms, stream);
  if (e != cudaSuccess) return e;
  e = p.w2.fp4 ? launch_small_fp4_down(p, sms, stream) : launch_small_e4m3_down(p, sms, stream);
  return e != cudaSuccess ? e : launch_join(p, stream);
}

}  // namespace moe
