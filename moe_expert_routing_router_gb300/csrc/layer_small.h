// Launcher of the experts of a layer for few tokens (layer_small.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kSmallTokens = 64, kSmallWidth = 16384;

// Weights of all experts: 4-bit codes [E, N, K/2] with words of four exponents
// [ceil(K/128), E N], or e4m3 codes [E, N, K] with scales [E, ceil(N/128), ceil(K/128)].
struct SmallWeights {
  int fp4;
  const uint8_t* q;
  const void* scale;
};

struct SmallLayerParams {
  const void* x;          // [T, H] bf16
  int T, H, I, E, k;
  const int32_t* idx;     // [T, k]
  const float* gate;      // [T, k]
  SmallWeights w1, w2;    // N, K: 2 I, H and H, I
  void* out;              // [T, H] bf16
  float* h;               // [T k, I]: scratch
  float* y;               // [T k, H]: scratch
};
size_t small_layer_work_size(int T, int H, int I, int k);
// Sets h and y within `work`.
void small_layer_work(SmallLayerParams& p, void* work);
// The first kernel (up) and the second by the kind of their weights.
cudaError_t launch_small_fp4_up(const SmallLayerParams& p, int sms, cudaStream_t stream);
cudaError_t launch_small_fp4_down(const SmallLayerParams& p, int sms, cudaStream_t stream);
cudaError_t launch_small_e4m3_up(const SmallLayerParams& p, int sms, cudaStream_t stream);
cudaError_t launch_small_e4m3_down(const SmallLayerParams& p, int sms, cudaStream_t stream);
cudaError_t launch_layer_small(const SmallLayerParams& p, int sms, cudaStream_t stream);

}  // namespace moe
