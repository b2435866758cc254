// Launchers of the gated combine of the experts' rows (expert_combine.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

struct CombineRowsParams {
  const void* y;          // [M, H] the experts' rows in dispatch order
  int64_t T, M;
  int H, k, E;
  const int32_t* idx;     // [T, k]
  const int32_t* slot;    // [T, k] flattened, -1 for a dropped assignment
  const int32_t* offsets; // [E+1]
  const float* gate;      // [T, k] or null (all ones)
  void* out;              // [T, H]
};
cudaError_t launch_expert_combine(const CombineRowsParams& p, bool bf16, int sms, cudaStream_t stream);

struct CombineRowsBwdParams {
  const void* dout;       // [T, H]
  const void* y;          // [M, H]
  int64_t T, M;
  int H, k, E;
  const int32_t* idx;
  const int32_t* slot;
  const int32_t* offsets;
  const float* gate;      // [T, k]
  void* dy;               // [M, H]: rows of kept assignments
  float* dgate;           // [T, k]
};
cudaError_t launch_expert_combine_bwd(const CombineRowsBwdParams& p, bool bf16, int sms, cudaStream_t stream);

}  // namespace moe
