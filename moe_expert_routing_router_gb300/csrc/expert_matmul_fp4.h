// Launcher of the experts' 4-bit matrix products (expert_matmul_fp4.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

struct MatmulFp4Params {
  int64_t M;              // rows of a and out
  int C, K, E;            // columns of out, contraction length, experts
  const uint8_t* a;       // [M, K/2]
  const uint32_t* a_scale;// [ceil(K/128), M]: words of four exponents
  const uint8_t* b;       // [E, C, K/2]
  const uint32_t* b_scale;// [ceil(K/128), E C]
  const int32_t* offsets; // [E+1] or null (one expert with all M rows)
  const int32_t* kept;    // [E] or null
  int out_bf16;
  void* out;              // [M, C]
  int* errors;            // the device's error word
  uint64_t timeout_ns;
  unsigned extra;         // tests of the expired wait: arrivals that never come
};

// `error` receives a message when the result is cudaErrorUnknown (tensor map).
cudaError_t launch_expert_matmul_fp4(const MatmulFp4Params& p, int sms, const char** error, cudaStream_t stream);

}  // namespace moe
