// Launchers of the microscaled 4-bit quantisation (quantize_fp4.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

struct QuantFp4Params {
  const void* x;          // [rows, K]
  int64_t rows, M;        // rows of x, rows of q
  int K, k;
  const int32_t* perm;    // [M] or null: row r of q is row perm[r] / k of x
  uint8_t* q;             // [M, K/2]
  uint32_t* scale;        // [ceil(K/128), M]: four scale codes a word
};
cudaError_t launch_quantize_fp4(const QuantFp4Params& p, bool bf16, cudaStream_t stream);

struct DequantFp4Params {
  const uint8_t* q;       // [M, K/2]
  const uint32_t* scale;  // [ceil(K/128), M]
  int64_t M;
  int K;
  void* y;                // [M, K]
};
cudaError_t launch_dequantize_fp4(const DequantFp4Params& p, bool bf16, cudaStream_t stream);

}  // namespace moe
