// Launcher of the experts' 8-bit matrix products (expert_matmul.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// One contraction per expert e:  out_e[r, c] = sum over blocks b of 128 of
//   a_scale * b_scale * sum_k a[r, 128 b + k] * b[c, 128 b + k].
//   product:          r runs over the expert's rows of a [M, K], c over its matrix b [E, N, K];
//   weight gradient:  r and c run over the rows of a [R, width] and b [C, width], the
//                     contraction over the expert's columns of both.
struct MatmulParams {
  int wgrad;
  int64_t M;              // rows of a (product)
  int R, C;               // C: columns of out; R: rows of one expert's out (weight gradient)
  int K;                  // contraction length (product)
  int E;
  int64_t blocks;         // column blocks of a and b (weight gradient)
  const uint8_t* a;
  const float* a_scale;   // product [ceil(K/128), M]; weight gradient [blocks, R]
  const uint8_t* b;
  const float* b_scale;   // product [E, ceil(C/128), ceil(K/128)]; weight gradient [blocks, C]
  const int32_t* offsets; // [E+1] or null (product: one expert with all M rows)
  const int32_t* kept;    // [E] or null (product)
  int out_bf16;
  void* out;              // product [M, C]; weight gradient [E, R, C]
  uint64_t timeout_ns;
  unsigned extra;         // tests of the expired wait: arrivals that never come
};

// `error` receives a message when the result is cudaErrorUnknown (tensor map).
cudaError_t launch_expert_matmul(const MatmulParams& p, int sms, const char** error, cudaStream_t stream);
// Reads and clears the current device's error bits (synchronises the stream).
cudaError_t expert_matmul_errors(int* bits, cudaStream_t stream);

}  // namespace moe
