// The layer for few tokens: its scratch, and the choice of its kernels (layer_small.cuh).
#include "layer_small.h"

namespace moe {
namespace {

size_t up_to(size_t n) { return (n + 255) / 256 * 256; }   // pieces of the scratch

}  // namespace

size_t small_layer_work_size(int T, int H, int I, int k) {
  const size_t A = size_t(T) * k;
  return up_to(A * I * 4) + up_to(A * H * 4) + up_to(size_t(H + kSmallJoin - 1) / kSmallJoin * 4);
}

void small_layer_work(SmallLayerParams& p, void* work) {
  const size_t A = size_t(p.T) * p.k;
  char* at = static_cast<char*>(work);
  p.h = reinterpret_cast<float*>(at);
  p.y = reinterpret_cast<float*>(at + up_to(A * p.I * 4));
  p.joined = reinterpret_cast<int*>(at + up_to(A * p.I * 4) + up_to(A * p.H * 4));
}

cudaError_t launch_layer_small(const SmallLayerParams& p, int sms, cudaStream_t stream) {
  const cudaError_t e = p.w1.fp4 ? launch_small_fp4_up(p, sms, stream) : launch_small_e4m3_up(p, sms, stream);
  if (e != cudaSuccess) return e;
  return p.w2.fp4 ? launch_small_fp4_down(p, sms, stream) : launch_small_e4m3_down(p, sms, stream);
}

}  // namespace moe
