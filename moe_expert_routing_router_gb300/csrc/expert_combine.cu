// The experts' rows gathered back to their tokens and summed by gate, and the
// gradient of that sum.
//
//   out[t]      = sum_j gate[t,j] * y[row(t,j)],   row(t,j) = offsets[idx[t,j]] + slot[t,j]
//   dy[row]     = gate[t,j] * dout[t]
//   dgate[t,j]  = <dout[t], y[row]>
//
// over the assignments that were kept (slot >= 0).  Both are bound by memory:
// every row is read once, in 16-byte loads of which a thread has k in flight,
// sums are fp32 in the order of j, and there are no atomics: repeated calls give
// the same bits.  W warps work on a token; many tokens take one warp each (its
// index loads and row loads overlap with the other warps' of the SM), few tokens
// take up to eight.  16,384 x 6 rows of 2048 bf16, none dropped: 74 us and 133 us
// backward, 6.3 and 6.6 TB/s; an eighth dropped: 69 and 121 us, 6.1 and 6.4 TB/s of
// the rows kept.  Rows that are not whole pieces of 16 bytes take an element a load:
// of 2044 to 2047 bf16 170 and 308 us, of 2046 and 2047 fp32 197 and 405 us (2048: 145
// and 265).
#include "device_common.cuh"
#include "expert_combine.h"

#include <cuda_bf16.h>

namespace moe {
namespace {

constexpr int kMaxK = 8;
constexpr int kWarps = 8;            // of a CTA
constexpr unsigned kFull = 0xffffffffu;

// VEC neighbouring values, kept as they were loaded.
template <bool BF16, int VEC>
struct Piece {
  static constexpr int kWords = VEC == 1 ? 1 : 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const void* x, int64_t at) {
    if constexpr (VEC == 1) {
      w[0] = BF16 ? uint32_t(static_cast<const uint16_t*>(x)[at]) : static_cast<const uint32_t*>(x)[at];
    } else {
      const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const char*>(x) + at * (BF16 ? 2 : 4));
      w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (BF16) return __uint_as_float(i % 2 == 0 ? w[i / 2] << 16 : w[i / 2] & 0xffff0000u);
    else return __uint_as_float(w[i]);
  }
  __device__ __forceinline__ static void store(void* x, int64_t at, const float* v) {
    if constexpr (VEC == 1) {
      if constexpr (BF16) static_cast<__nv_bfloat16*>(x)[at] = __float2bfloat16_rn(v[0]);
      else static_cast<float*>(x)[at] = v[0];
    } else if constexpr (BF16) {
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        h[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(x) + at) = make_uint4(h[0], h[1], h[2], h[3]);
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(x) + at) = make_float4(v[0], v[1], v[2], v[3]);
    }
  }
};

// The row of an assignment, or -1 when it was dropped or lies outside y.
__device__ __forceinline__ int64_t assigned_row(const int32_t* idx, const int32_t* slot, const int32_t* offsets, int64_t a,
                                                int E, int64_t M) {
  const int s = slot[a], e = idx[a];
  if (s < 0 || e < 0 || e >= E) return -1;
  const int64_t r = int64_t(offsets[e]) + s;
  return r >= 0 && r < M ? r : -1;
}

// A warp's token, its pieces of the row, and lane j's assignment spread to all lanes.
struct Token {
  int64_t t;
  int part;                       // of the W warps of the token
  int row[kMaxK];                 // rows of y, -1 for none
  float gate[kMaxK];

  __device__ __forceinline__ void fetch(const int32_t* idx, const int32_t* slot, const int32_t* offsets, const float* g,
                                        int64_t T, int64_t M, int k, int E, int W, int lane) {
    const int64_t unit = int64_t(blockIdx.x) * kWarps + threadIdx.x / kWarp;
    t = unit / W;
    part = int(unit % W);
    int r = -1;
    float gv = 0.f;
    if (t < T && lane < k) {
      r = int(assigned_row(idx, slot, offsets, t * k + lane, E, M));
      gv = g != nullptr ? g[t * k + lane] : 1.f;
    }
#pragma unroll
    for (int j = 0; j < kMaxK; ++j) {
      row[j] = __shfl_sync(kFull, r, j);          // lanes from k on hold -1
      gate[j] = __shfl_sync(kFull, gv, j);
    }
  }
};

template <bool BF16, int VEC>
__global__ void __launch_bounds__(kWarps * kWarp) expert_combine_kernel(const CombineRowsParams p, int W) {
  using P = Piece<BF16, VEC>;
  const int lane = threadIdx.x % kWarp;
  Token tk;
  tk.fetch(p.idx, p.slot, p.offsets, p.gate, p.T, p.M, p.k, p.E, W, lane);
  if (tk.t >= p.T) return;
  for (int c = (tk.part * kWarp + lane) * VEC; c < p.H; c += W * kWarp * VEC) {
    P v[kMaxK];
#pragma unroll
    for (int j = 0; j < kMaxK; ++j)
      if (tk.row[j] >= 0) v[j].load(p.y, int64_t(tk.row[j]) * p.H + c);
    float acc[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.f;
#pragma unroll
    for (int j = 0; j < kMaxK; ++j)
      if (tk.row[j] >= 0) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] = fmaf(tk.gate[j], v[j].get(i), acc[i]);
      }
    P::store(p.out, tk.t * p.H + c, acc);
  }
}

template <bool BF16, int VEC>
__global__ void __launch_bounds__(kWarps * kWarp) expert_combine_bwd_kernel(const CombineRowsBwdParams p, int W) {
  using P = Piece<BF16, VEC>;
  __shared__ float s_dot[kWarps][kMaxK];
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  Token tk;
  tk.fetch(p.idx, p.slot, p.offsets, p.gate, p.T, p.M, p.k, p.E, W, lane);
  float dot[kMaxK];
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) dot[j] = 0.f;
  if (tk.t < p.T) {
    for (int c = (tk.part * kWarp + lane) * VEC; c < p.H; c += W * kWarp * VEC) {
      P d, v[kMaxK];
      d.load(p.dout, tk.t * p.H + c);
#pragma unroll
      for (int j = 0; j < kMaxK; ++j)
        if (tk.row[j] >= 0) v[j].load(p.y, int64_t(tk.row[j]) * p.H + c);
#pragma unroll
      for (int j = 0; j < kMaxK; ++j)
        if (tk.row[j] >= 0) {
          float o[VEC];
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            dot[j] = fmaf(d.get(i), v[j].get(i), dot[j]);
            o[i] = tk.gate[j] * d.get(i);
          }
          P::store(p.dy, int64_t(tk.row[j]) * p.H + c, o);
        }
    }
  }
  float mine = 0.f;                                             // lane j: the warp's part of dgate[t, j]
#pragma unroll
  for (int j = 0; j < kMaxK; ++j) {
    const float s = warp_sum_f(dot[j]);
    if (lane == j) mine = s;
  }
  if (W > 1) {                                                  // the token's warps are neighbours in the CTA
    if (lane < kMaxK) s_dot[warp][lane] = mine;
    __syncthreads();
    if (tk.part != 0 || lane >= kMaxK) return;
    mine = 0.f;
    for (int w = 0; w < W; ++w) mine += s_dot[warp + w][lane];
  }
  if (tk.t < p.T && lane < p.k) p.dgate[tk.t * p.k + lane] = mine;
}

bool vec_ok(int H, int vec, const void* a, const void* b, const void* c) {
  return H % vec == 0 && (reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | reinterpret_cast<uintptr_t>(c)) % 16 == 0;
}

// Warps of a token: one, and up to a CTA's eight (a power of two, at most one per
// 32 pieces) while that leaves fewer than 16 warps an SM.  One warp, this rule and
// eight, k 8, bf16: 16 tokens of 4096 10.0, 2.8 and 2.8 us (backward 16.5, 4.0, 4.0);
// 512 of 2048 6.3, 3.7, 3.7; 2048 of 2048 14.5, 13.2, 14.1; 16,384 x 6 of 2048 74.0,
// 74.0, 85.9 (backward 132.9, 132.9, 156.4).
int warps_for(int64_t T, int H, int vec, int sms) {
  const int64_t pieces = (int64_t(H) + vec - 1) / vec;
  int W = 1;
  while (W < kWarps && T * W < int64_t(sms) * 16 && int64_t(W) * kWarp < pieces) W *= 2;
  return W;
}

template <bool BF16, int VEC>
cudaError_t combine_launch(const CombineRowsParams& p, int sms, cudaStream_t stream) {
  const int W = warps_for(p.T, p.H, VEC, sms);
  expert_combine_kernel<BF16, VEC><<<unsigned((p.T * W + kWarps - 1) / kWarps), kWarps * kWarp, 0, stream>>>(p, W);
  return cudaGetLastError();
}

template <bool BF16, int VEC>
cudaError_t combine_bwd_launch(const CombineRowsBwdParams& p, int sms, cudaStream_t stream) {
  const int W = warps_for(p.T, p.H, VEC, sms);
  expert_combine_bwd_kernel<BF16, VEC><<<unsigned((p.T * W + kWarps - 1) / kWarps), kWarps * kWarp, 0, stream>>>(p, W);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_combine(const CombineRowsParams& p, bool bf16, int sms, cudaStream_t stream) {
  if (bf16) return vec_ok(p.H, 8, p.y, p.out, nullptr) ? combine_launch<true, 8>(p, sms, stream) : combine_launch<true, 1>(p, sms, stream);
  return vec_ok(p.H, 4, p.y, p.out, nullptr) ? combine_launch<false, 4>(p, sms, stream) : combine_launch<false, 1>(p, sms, stream);
}

cudaError_t launch_expert_combine_bwd(const CombineRowsBwdParams& p, bool bf16, int sms, cudaStream_t stream) {
  if (bf16) return vec_ok(p.H, 8, p.y, p.dout, p.dy) ? combine_bwd_launch<true, 8>(p, sms, stream) : combine_bwd_launch<true, 1>(p, sms, stream);
  return vec_ok(p.H, 4, p.y, p.dout, p.dy) ? combine_bwd_launch<false, 4>(p, sms, stream) : combine_bwd_launch<false, 1>(p, sms, stream);
}

}  // namespace moe
