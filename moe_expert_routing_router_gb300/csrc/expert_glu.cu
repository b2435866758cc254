// The gated activation between an expert's two products, y = g sigmoid(g) u for the halves
// g, u of a row, and its gradient.
//
//   s = sigmoid(g),  y = g s u,  du = dy g s,  dg = dy u s (1 + g (1 - s))
//
// With t = exp(-|g|) in (0, 1] the two sigmoids are 1 / (1 + t) and t / (1 + t): neither
// overflows, and 1 - s keeps its digits.  Everything is computed in fp32 and rounded once.
// y leaves in the input's type, or as the second product's operand, e4m3 with a scale for
// 128 values or 4 bits with one for 32, so that it is never written and read again.
//
// All forms are bound by memory: 32836 rows of 2048, bf16, 66 us (6.2 TB/s), the gradient 102 us (6.6 TB/s).
// Quantised, to e4m3 64 us (5.3 TB/s) and to 4 bits 66 us (4.6 TB/s), the exponential and the reciprocal of a
// value and its code take two thirds of the issue slots besides.
#include "block_values.cuh"
#include "expert_glu.h"

#include <cuda_bf16.h>

#include <cfloat>

namespace moe {
namespace {

constexpr int kThreads = 256;

// exp(-|g|).  Of bf16 values one rounding of the exponent is enough (2^-17 of the result where
// |g| <= 88); fp32 values get the accurate function.
template <bool BF16>
__device__ __forceinline__ float decay(float g) {
  if constexpr (BF16) {
    float t;
    asm("ex2.approx.f32 %0, %1;" : "=f"(t) : "f"(-fabsf(g) * kLog2e));
    return t;
  } else {
    return expf(-fabsf(g));
  }
}

// sigmoid(g) and sigmoid(-g).
template <bool BF16>
__device__ __forceinline__ float2 sigmoids(float g) {
  const float t = decay<BF16>(g);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + t));    // 1 + t is in [1, 2]
  return g >= 0.f ? make_float2(r, t * r) : make_float2(t * r, r);
}

template <bool BF16>
__device__ __forceinline__ float gated(float g, float u) { return g * sigmoids<BF16>(g).x * u; }

template <bool BF16, int N>
__device__ __forceinline__ void store(void* base, int64_t at, const float (&f)[N]) {
  uint4* to = reinterpret_cast<uint4*>(static_cast<char*>(base) + at * (BF16 ? 2 : 4));
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < N; i += 8) {
      uint32_t b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 q = __floats2bfloat162_rn(f[i + 2 * j], f[i + 2 * j + 1]);
        b[j] = *reinterpret_cast<const uint32_t*>(&q);
      }
      to[i / 8] = make_uint4(b[0], b[1], b[2], b[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      to[i / 4] = make_uint4(__float_as_uint(f[i]), __float_as_uint(f[i + 1]), __float_as_uint(f[i + 2]), __float_as_uint(f[i + 3]));
  }
}

// A piece of 8 columns of a row.
template <bool BF16>
__global__ void __launch_bounds__(kThreads) glu_kernel(const GluParams p) {
  constexpr int N = 8;
  const int per = p.I / N;
  const int64_t pieces = p.M * per, i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= pieces) return;
  const int64_t r = i / per;
  const int c = int(i - r * per) * N;
  Values<BF16, N> g, u;
  g.load(p.h, r * 2 * p.I + c);
  u.load(p.h, r * 2 * p.I + p.I + c);
  float y[N];
#pragma unroll
  for (int j = 0; j < N; ++j) y[j] = gated<BF16>(g.get(j), u.get(j));
  store<BF16>(p.out, r * p.I + c, y);
}

template <bool BF16>
__global__ void __launch_bounds__(kThreads) glu_bwd_kernel(const GluBwdParams p) {
  constexpr int N = 8;
  const int per = p.I / N;
  const int64_t pieces = p.M * per, i = int64_t(blockIdx.x) * kThreads + threadIdx.x;
  if (i >= pieces) return;
  const int64_t r = i / per;
  const int c = int(i - r * per) * N;
  Values<BF16, N> g, u, d;
  g.load(p.h, r * 2 * p.I + c);
  u.load(p.h, r * 2 * p.I + p.I + c);
  d.load(p.dy, r * p.I + c);
  float dg[N], du[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float2 s = sigmoids<BF16>(g.get(j));
    du[j] = d.get(j) * (g.get(j) * s.x);
    const float slope = s.x * fmaf(g.get(j), s.y, 1.f), both = d.get(j) * u.get(j);   // the slope is below 1.1, and may be small
    dg[j] = fabsf(both) <= FLT_MAX ? both * slope : d.get(j) * (u.get(j) * slope);
  }
  store<BF16>(p.dh, r * 2 * p.I + c, dg);
  store<BF16>(p.dh, r * 2 * p.I + p.I + c, du);
}

// Quantised: eight lanes hold 128 values of a row, 16 each, as the quantisation of rows does.
constexpr int kLanes = 8, kVals = kScaleBlock / kLanes, kTeams = kWarp / kLanes, kBlocks = 4;
constexpr int kIter = 2;                      // rows of a lane, loaded together
constexpr int kTileRows = kThreads / kWarp / kBlocks * kTeams * kIter;

template <bool BF16, bool FP4>
__global__ void __launch_bounds__(kThreads) glu_quantize_kernel(const GluParams p) {
  using V = Values<BF16, kVals>;
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp, l = lane % kLanes;
  const int kb = blockIdx.y * kBlocks + warp % kBlocks, col = kb * kScaleBlock + l * kVals;
  const int64_t r0 = int64_t(blockIdx.x) * kTileRows + warp / kBlocks * (kTeams * kIter) + lane / kLanes;
  if (kb * kScaleBlock >= p.I) return;
  V g[kIter], u[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int64_t r = r0 + i * kTeams;
    if (r < p.M && col < p.I) {
      g[i].load(p.h, r * 2 * p.I + col);
      u[i].load(p.h, r * 2 * p.I + p.I + col);
    } else {
      g[i].zero();
      u[i].zero();
    }
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    float y[kVals];
    uint32_t m = 0;                                              // as bits, a NaN above every number
#pragma unroll
    for (int j = 0; j < kVals; ++j) {
      y[j] = gated<BF16>(g[i].get(j), u[i].get(j));
      m = max(m, __float_as_uint(y[j]) & 0x7fffffffu);
    }
    m = max(m, __shfl_xor_sync(kFull, m, 1));
    const int64_t r = r0 + i * kTeams;
    if constexpr (FP4) {
      const Fp4Scale s = fp4_scale(__uint_as_float(m));
      const uint32_t word = fp4_scale_word(s.code, l);
      if (r >= p.M) continue;
      if (l == i) static_cast<uint32_t*>(p.scale)[int64_t(kb) * p.M + r] = word;
      if (col >= p.I) continue;
      const float2 inv = make_float2(s.inv, s.inv);
      uint32_t c[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float2 f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = mul2(make_float2(y[8 * h + 2 * j], y[8 * h + 2 * j + 1]), inv);
        c[h] = fp4_pack8(f[0], f[1], f[2], f[3]);
      }
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + (r * p.I + col) / 2) = make_uint2(c[0], c[1]);
    } else {
      m = max(m, __shfl_xor_sync(kFull, m, 2));
      m = max(m, __shfl_xor_sync(kFull, m, 4));
      const Pow2Scale s = pow2_scale(__uint_as_float(m));
      if (r >= p.M) continue;
      if (l == i) static_cast<float*>(p.scale)[int64_t(kb) * p.M + r] = s.scale;
      if (col >= p.I) continue;
      uint32_t c[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) c[h] = scaled4(make_float2(y[4 * h], y[4 * h + 1]), make_float2(y[4 * h + 2], y[4 * h + 3]), s.inv);
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.out) + r * p.I + col) = make_uint4(c[0], c[1], c[2], c[3]);
    }
  }
}

template <bool BF16>
cudaError_t launch(const GluParams& p, cudaStream_t stream) {
  if (p.form == kGluPlain) {
    const int64_t pieces = p.M * (p.I / 8);
    glu_kernel<BF16><<<unsigned((pieces + kThreads - 1) / kThreads), kThreads, 0, stream>>>(p);
  } else {
    const int kb = (p.I + kScaleBlock - 1) / kScaleBlock;
    const dim3 grid(unsigned((p.M + kTileRows - 1) / kTileRows), unsigned((kb + kBlocks - 1) / kBlocks));
    if (p.form == kGluFp4) glu_quantize_kernel<BF16, true><<<grid, kThreads, 0, stream>>>(p);
    else glu_quantize_kernel<BF16, false><<<grid, kThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_glu(const GluParams& p, bool bf16, cudaStream_t stream) {
  return bf16 ? launch<true>(p, stream) : launch<false>(p, stream);
}

cudaError_t launch_expert_glu_bwd(const GluBwdParams& p, bool bf16, cudaStream_t stream) {
  const int64_t pieces = p.M * (p.I / 8);
  const unsigned grid = unsigned((pieces + kThreads - 1) / kThreads);
  if (bf16) glu_bwd_kernel<true><<<grid, kThreads, 0, stream>>>(p);
  else glu_bwd_kernel<false><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace moe
