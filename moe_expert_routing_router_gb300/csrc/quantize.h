// Launchers of the block-scaled 8-bit quantisation (quantize.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

constexpr int kScaleBlock = 128;        // values that share a scale

struct QuantRowsParams {
  const void* x;          // [rows, K]
  int64_t rows, M;        // rows of x, rows of q
  int K, k;
  const int32_t* perm;    // [M] or null: row r of q is row perm[r] / k of x
  uint8_t* q;             // [M, K] e4m3
  float* scale;           // [ceil(K/128), M]
};
cudaError_t launch_quantize_rows(const QuantRowsParams& p, bool bf16, cudaStream_t stream);

struct QuantColsParams {
  const void* x;          // [rows, K]
  int64_t rows, M;
  int K, k, E;
  const int32_t* offsets; // [E+1]
  const int32_t* kept;    // [E] or null
  const int32_t* perm;    // [M] or null
  int64_t width;          // columns of q
  uint8_t* q;             // [K, width] e4m3
  float* scale;           // [width/128, K]
  int64_t share;          // tiles of a CTA, set by the launcher
};
cudaError_t launch_quantize_cols(QuantColsParams p, bool bf16, int sms, cudaStream_t stream);

struct QuantWeightsParams {
  const void* w;          // [E, N, K]
  int E, N, K;
  uint8_t* q;             // [E, N, K] e4m3 or null
  float* scale;           // [E, ceil(N/128), ceil(K/128)] or null
  uint8_t* qt;            // [E, K, N] e4m3 or null
  float* scalet;          // [E, ceil(K/128), ceil(N/128)] or null
};
cudaError_t launch_quantize_weights(const QuantWeightsParams& p, bool bf16, cudaStream_t stream);

}  // namespace moe
