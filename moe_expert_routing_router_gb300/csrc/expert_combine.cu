// The experts' rows gathered back to their tokens and summed by gate, and the
// gradient of that sum.
//
//   out[t]      = sum_j gate[t,j] * y[row(t,j)],   row(t,j) = offsets[idx[t,j]] + slot[t,j]
//   dy[row]     = gate[t,j] * dout[t]
//   dgate[t,j]  = <dout[t], y[row]>
//
// over the assignments that were kept (slot >= 0).  Both are bound by memory:
// every row is read once, in 16-byte loads that are all in flight before the
// first is used, sums are fp32 in the order of j, and there are no atomics:
// a token's rows belong to one CTA, so repeated calls give the same bits.
#include "device_common.cuh"
#include "expert_combine.h"

#include <cuda_bf16.h>

namespace moe {
namespace {

constexpr int kMaxK = 8;

template <bool BF16, int VEC>
__device__ __forceinline__ void load_vec(const void* x, int64_t at, float* v) {
  if constexpr (VEC == 1) {
    v[0] = BF16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(x)[at]) : static_cast<const float*>(x)[at];
  } else if constexpr (BF16) {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(x) + at);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float4 u = *reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
  }
}

template <bool BF16, int VEC>
__device__ __forceinline__ void store_vec(void* x, int64_t at, const float* v) {
  if constexpr (VEC == 1) {
    if constexpr (BF16) static_cast<__nv_bfloat16*>(x)[at] = __float2bfloat16_rn(v[0]);
    else static_cast<float*>(x)[at] = v[0];
  } else if constexpr (BF16) {
    uint4 u;
    uint32_t* w = &u.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(x) + at) = u;
  } else {
    *reinterpret_cast<float4*>(static_cast<float*>(x) + at) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// The row of an assignment, or -1 when it was dropped or lies outside y.
__device__ __forceinline__ int64_t assigned_row(const int32_t* idx, const int32_t* slot, const int32_t* offsets, int64_t a,
                                                int E, int64_t M) {
  const int s = slot[a], e = idx[a];
  if (s < 0 || e < 0 || e >= E) return -1;
  const int64_t r = int64_t(offsets[e]) + s;
  return r >= 0 && r < M ? r : -1;
}

// One CTA per token and piece of blockDim.x * VEC columns.
template <bool BF16, int VEC>
__global__ void __launch_bounds__(512) expert_combine_kernel(const CombineRowsParams p) {
  __shared__ int64_t s_row[kMaxK];
  __shared__ float s_gate[kMaxK];
  const int64_t t = blockIdx.x;
  if (threadIdx.x < p.k) {
    const int64_t a = t * p.k + threadIdx.x;
    s_row[threadIdx.x] = assigned_row(p.idx, p.slot, p.offsets, a, p.E, p.M);
    s_gate[threadIdx.x] = p.gate != nullptr ? p.gate[a] : 1.f;
  }
  __syncthreads();
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * VEC;
  if (c >= p.H) return;
  float v[kMaxK][VEC];
#pragma unroll
  for (int j = 0; j < kMaxK; ++j)
    if (j < p.k && s_row[j] >= 0) load_vec<BF16, VEC>(p.y, s_row[j] * p.H + c, v[j]);
  float acc[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
#pragma unroll
  for (int j = 0; j < kMaxK; ++j)
    if (j < p.k && s_row[j] >= 0) {
      const float g = s_gate[j];
#pragma unroll
      for (int i = 0; i < VEC; ++i) acc[i] = fmaf(g, v[j][i], acc[i]);
    }
  store_vec<BF16, VEC>(p.out, t * p.H + c, acc);
}

// One CTA per token: it passes over the columns once and adds up the k dots.
template <bool BF16, int VEC>
__global__ void __launch_bounds__(256) expert_combine_bwd_kernel(const CombineRowsBwdParams p) {
  __shared__ int64_t s_row[kMaxK];
  __shared__ float s_gate[kMaxK];
  __shared__ float s_dot[kMaxK][8];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  if (threadIdx.x < p.k) {
    const int64_t a = t * p.k + threadIdx.x;
    s_row[threadIdx.x] = assigned_row(p.idx, p.slot, p.offsets, a, p.E, p.M);
    s_gate[threadIdx.x] = p.gate[a];
  }
  __syncthreads();
  float dot[kMaxK];
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) dot[j] = 0.f;
  for (int c = threadIdx.x * VEC; c < p.H; c += blockDim.x * VEC) {
    float d[VEC], v[kMaxK][VEC];
    load_vec<BF16, VEC>(p.dout, t * p.H + c, d);
#pragma unroll
    for (int j = 0; j < kMaxK; ++j)
      if (j < p.k && s_row[j] >= 0) load_vec<BF16, VEC>(p.y, s_row[j] * p.H + c, v[j]);
#pragma unroll
    for (int j = 0; j < kMaxK; ++j)
      if (j < p.k && s_row[j] >= 0) {
        const float g = s_gate[j];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          dot[j] = fmaf(d[i], v[j][i], dot[j]);
          v[j][i] = g * d[i];
        }
        store_vec<BF16, VEC>(p.dy, s_row[j] * p.H + c, v[j]);
      }
  }
#pragma unroll
  for (int j = 0; j < kMaxK; ++j)
    if (j < p.k) {
      const float s = warp_sum_f(dot[j]);
      if (lane == 0) s_dot[j][warp] = s;
    }
  __syncthreads();
  if (threadIdx.x < p.k) {
    float s = 0.f;
    for (int w = 0; w < int(blockDim.x) / kWarp; ++w) s += s_dot[threadIdx.x][w];
    p.dgate[t * p.k + threadIdx.x] = s_row[threadIdx.x] >= 0 ? s : 0.f;
  }
}

bool vec_ok(int H, int vec, const void* a, const void* b, const void* c) {
  return H % vec == 0 && (reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | reinterpret_cast<uintptr_t>(c)) % 16 == 0;
}

int threads_for(int64_t pieces, int most) {
  int t = kWarp;
  while (t < most && t < pieces) t += kWarp;
  return t;
}

template <bool BF16, int VEC>
cudaError_t combine_launch(const CombineRowsParams& p, cudaStream_t stream) {
  const int64_t pieces = (p.H + VEC - 1) / VEC;
  // Few tokens: small CTAs, so that a token's columns spread over several SMs.
  const int threads = threads_for(pieces, p.T < 256 ? 64 : 256);
  const dim3 grid(unsigned(p.T), unsigned((pieces + threads - 1) / threads));
  expert_combine_kernel<BF16, VEC><<<grid, threads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <bool BF16, int VEC>
cudaError_t combine_bwd_launch(const CombineRowsBwdParams& p, cudaStream_t stream) {
  const int threads = threads_for((p.H + VEC - 1) / VEC, 256);
  expert_combine_bwd_kernel<BF16, VEC><<<unsigned(p.T), threads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_combine(const CombineRowsParams& p, bool bf16, cudaStream_t stream) {
  if (bf16) return vec_ok(p.H, 8, p.y, p.out, nullptr) ? combine_launch<true, 8>(p, stream) : combine_launch<true, 1>(p, stream);
  return vec_ok(p.H, 4, p.y, p.out, nullptr) ? combine_launch<false, 4>(p, stream) : combine_launch<false, 1>(p, stream);
}

cudaError_t launch_expert_combine_bwd(const CombineRowsBwdParams& p, bool bf16, cudaStream_t stream) {
  if (bf16) return vec_ok(p.H, 8, p.y, p.dout, p.dy) ? combine_bwd_launch<true, 8>(p, stream) : combine_bwd_launch<true, 1>(p, stream);
  return vec_ok(p.H, 4, p.y, p.dout, p.dy) ? combine_bwd_launch<false, 4>(p, stream) : combine_bwd_launch<false, 1>(p, stream);
}

}  // namespace moe
