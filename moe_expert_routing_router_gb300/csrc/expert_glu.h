// Launchers of the gated activation between the experts' products (expert_glu.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

enum GluForm : int { kGluPlain = 0, kGluE4m3 = 1, kGluFp4 = 2 };

struct GluParams {
  const void* h;          // [M, 2 I]
  int64_t M;
  int I;
  int form;               // GluForm
  void* out;              // [M, I] in h's type, e4m3 codes [M, I], or 4-bit codes [M, I/2]
  void* scale;            // [ceil(I/128), M] fp32, or words of four scale codes
};
cudaError_t launch_expert_glu(const GluParams& p, bool bf16, cudaStream_t stream);

struct GluBwdParams {
  const void* h;          // [M, 2 I]
  const void* dy;         // [M, I]
  int64_t M;
  int I;
  void* dh;               // [M, 2 I]
};
cudaError_t launch_expert_glu_bwd(const GluBwdParams& p, bool bf16, cudaStream_t stream);

}  // namespace moe
