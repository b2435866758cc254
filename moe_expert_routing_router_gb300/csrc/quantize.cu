// Quantisation to e4m3 with one scale for a block of 128 values.
//
// The scale is the power of two s with 224 < max|x| / s <= 448, the largest
// e4m3 value: dividing by it is exact, so a value is rounded once (to nearest,
// ties to even, half a step of 2^-4 of itself), and a transposed block has the
// same codes.  A block of zeros has the scale 1; a block that holds an infinity
// or a NaN has the scale NaN, which every product with it then shows.
//
// All three kernels are bound by memory: every value is read once, held in
// registers while its block's maximum is found, and written once as a byte.
#include "device_common.cuh"
#include "quantize.h"

#include <cuda_bf16.h>

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;

// The block's scale and its inverse, from the bits of max|x|.
struct Pow2Scale {
  float scale, inv;
};
__device__ __forceinline__ Pow2Scale pow2_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
  if (b == 0u) return {1.f, 1.f};
  if (b >= 0x7f800000u) return {__uint_as_float(0x7fc00000u), 0.f};
  // amax = m * 2^x, 1 <= m < 2: 448 = 1.75 * 2^8, so the exponent is x - 8, one
  // more where m > 1.75, and at least -126 (a subnormal amax has it).
  const int x = int(b >> 23) - 127;
  int n = x - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  n = n < -126 ? -126 : n;                       // 2^-n <= 2^126 is finite; n <= 120
  return {__uint_as_float(uint32_t(n + 127) << 23), __uint_as_float(uint32_t(127 - n) << 23)};
}

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return uint32_t(lo) | uint32_t(hi) << 16;
}

// N neighbouring values, kept as they were loaded (bf16: two in a register).
template <bool BF16, int N>
struct Values {
  static constexpr int kWords = BF16 ? N / 2 : N;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const void* x, int64_t at) {
    const uint32_t* s = reinterpret_cast<const uint32_t*>(static_cast<const char*>(x) + at * (BF16 ? 2 : 4));
    if constexpr (kWords % 4 == 0) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 u = *reinterpret_cast<const uint4*>(s + i);
        w[i] = u.x; w[i + 1] = u.y; w[i + 2] = u.z; w[i + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 2) {
        const uint2 u = *reinterpret_cast<const uint2*>(s + i);
        w[i] = u.x; w[i + 1] = u.y;
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (BF16) return __uint_as_float(i % 2 == 0 ? w[i / 2] << 16 : w[i / 2] & 0xffff0000u);
    else return __uint_as_float(w[i]);
  }
  // Largest |x| so far, word by word: as unsigned integers (bf16: halves), so that a
  // NaN is above every number.
  __device__ __forceinline__ static uint32_t larger(uint32_t m, uint32_t w) {
    if constexpr (BF16) return __vmaxu2(m, w & 0x7fff7fffu);
    else return max(m, w & 0x7fffffffu);
  }
  // The fp32 bits of the larger half (bf16), or of the word.
  __device__ __forceinline__ static uint32_t bits(uint32_t m) {
    if constexpr (BF16) return max(m << 16, m & 0xffff0000u);
    else return m;
  }
  __device__ __forceinline__ uint32_t largest() const {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < kWords; ++i) m = larger(m, w[i]);
    return m;
  }
  // Four neighbouring values from the i-th on, scaled and rounded.
  __device__ __forceinline__ uint32_t codes(int i, float inv) const {
    return pack4(get(i) * inv, get(i + 1) * inv, get(i + 2) * inv, get(i + 3) * inv);
  }
};

// The row of x that row r of the output holds, or -1: zeros.  All rows fit int32.
__device__ __forceinline__ int source_row(const int32_t* perm, int k, int64_t r, int64_t rows) {
  if (perm == nullptr) return int(r);
  const int a = perm[r];
  const uint32_t t = uint32_t(a) / uint32_t(k);
  return a >= 0 && t < uint64_t(rows) ? int(t) : -1;
}

// ---------------------------------------------------------------------------
// Rows: blocks of 1 x 128.  Eight lanes hold a block, 16 values each.  A CTA
// takes 32 rows by 4 blocks of columns (512), so that the scales of a block
// column, which lie one row after another, leave as whole 128-byte lines.
// ---------------------------------------------------------------------------
constexpr int kRowsTile = 32, kRowsBlocks = 4, kQuantThreads = 256, kRowLanes = 8, kRowVals = kScaleBlock / kRowLanes;

template <bool BF16>
__global__ void __launch_bounds__(kQuantThreads) quantize_rows_kernel(const QuantRowsParams p) {
  using V = Values<BF16, kRowVals>;
  __shared__ float s_scale[kRowsBlocks][kRowsTile];
  const int64_t r0 = int64_t(blockIdx.x) * kRowsTile;
  constexpr int kTeams = kQuantThreads / kRowLanes, kIter = kRowsTile * kRowsBlocks / kTeams;   // 32 teams, 4 blocks each
  const int team = threadIdx.x / kRowLanes, l = threadIdx.x % kRowLanes;
  const int kb = team % kRowsBlocks;
  const int col = (blockIdx.y * kRowsBlocks + kb) * kScaleBlock + l * kRowVals;
  // Lane i of the team finds the source of its i-th block.
  static_assert(kIter <= kRowLanes, "a lane a block");
  const int64_t r = r0 + l * (kRowsTile / kIter) + team / kRowsBlocks;
  const int token = l < kIter && r < p.M ? source_row(p.perm, p.k, r, p.rows) : -1;
  V v[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int t = __shfl_sync(kFull, token, i, kRowLanes);
    if (t >= 0 && col < p.K) v[i].load(p.x, int64_t(t) * p.K + col);
    else v[i].zero();
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int row = i * (kRowsTile / kIter) + team / kRowsBlocks;
    uint32_t m = v[i].largest();
#pragma unroll
    for (int off = kRowLanes / 2; off > 0; off >>= 1) m = V::larger(m, __shfl_xor_sync(kFull, m, off));
    const Pow2Scale s = pow2_scale(__uint_as_float(V::bits(m)));
    if (l == 0) s_scale[kb][row] = s.scale;
    if (r0 + row < p.M && col < p.K)
      *reinterpret_cast<uint4*>(p.q + (r0 + row) * p.K + col) =
          make_uint4(v[i].codes(0, s.inv), v[i].codes(4, s.inv), v[i].codes(8, s.inv), v[i].codes(12, s.inv));
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kRowsBlocks * kRowsTile; i += kQuantThreads) {
    const int b = blockIdx.y * kRowsBlocks + i / kRowsTile;
    const int64_t r = r0 + i % kRowsTile;
    if (b * kScaleBlock < p.K && r < p.M) p.scale[int64_t(b) * p.M + r] = s_scale[i / kRowsTile][i % kRowsTile];
  }
}

// ---------------------------------------------------------------------------
// Columns: blocks of 128 rows of one expert by one column, written transposed
// (the rows become the contraction of a weight gradient).  Expert e's rows
// start at column 128 * (sum over e' < e of ceil(kept[e'] / 128)); its last
// block ends in zeros.  A CTA takes one block of rows by 128 columns: a thread
// holds 4 columns of 16 rows, the maxima meet in shared memory, and the bytes
// turn through shared memory into rows of 128.
// ---------------------------------------------------------------------------
constexpr int kColsTile = 128, kColsLane = kColsTile / kWarp, kColsWarps = kQuantThreads / kWarp, kColsRows = kScaleBlock / kColsWarps;

template <bool BF16>
__global__ void __launch_bounds__(kQuantThreads) quantize_cols_kernel(const QuantColsParams p) {
  __shared__ int s_where[3];                                     // first row, rows, found
  __shared__ __align__(16) uint32_t s_max[kColsWarps][kColsTile];
  __shared__ __align__(16) uint8_t s_q[kColsTile][kScaleBlock + 16];
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  const int64_t blk = blockIdx.x;
  if (threadIdx.x < kWarp) {                                     // which expert's block this is
    if (lane == 0) s_where[2] = 0;
    __syncwarp();
    int64_t before = 0;
    for (int e0 = 0; e0 < p.E && before <= blk; e0 += kWarp) {
      const int e = e0 + lane;
      int64_t lo = 0, n = 0;
      if (e < p.E) {
        lo = min(max(int64_t(p.offsets[e]), int64_t(0)), p.M);
        const int64_t hi = min(max(int64_t(p.offsets[e + 1]), lo), p.M);
        n = hi - lo;
        if (p.kept != nullptr) n = min(n, max(int64_t(p.kept[e]), int64_t(0)));
      }
      const int64_t nb = (n + kScaleBlock - 1) / kScaleBlock;
      int64_t incl = nb;
#pragma unroll
      for (int off = 1; off < kWarp; off <<= 1) {
        const int64_t o = __shfl_up_sync(kFull, incl, off);
        if (lane >= off) incl += o;
      }
      const int64_t first = before + incl - nb;
      if (blk >= first && blk < first + nb) {
        const int64_t at = (blk - first) * kScaleBlock;
        s_where[0] = int(lo + at);
        s_where[1] = int(min(n - at, int64_t(kScaleBlock)));
        s_where[2] = 1;
      }
      before += __shfl_sync(kFull, incl, kWarp - 1);
    }
  }
  __syncthreads();
  if (s_where[2] == 0) return;                                   // behind the last expert: left as it is
  // Lane i finds the source of the warp's i-th row.
  const int r = warp * kColsRows + lane;
  const int token = lane < kColsRows && r < s_where[1] ? source_row(p.perm, p.k, int64_t(s_where[0]) + r, p.rows) : -1;
  const int col = blockIdx.y * kColsTile + lane * kColsLane;
  Values<BF16, kColsLane> v[kColsRows];
#pragma unroll
  for (int i = 0; i < kColsRows; ++i) {
    const int t = __shfl_sync(kFull, token, i);
    if (t >= 0 && col < p.K) v[i].load(p.x, int64_t(t) * p.K + col);
    else v[i].zero();
  }
  using V = Values<BF16, kColsLane>;
  uint32_t m[V::kWords] = {};                                    // a column each, bf16: two
#pragma unroll
  for (int i = 0; i < kColsRows; ++i)
#pragma unroll
    for (int j = 0; j < V::kWords; ++j) m[j] = V::larger(m[j], v[i].w[j]);
#pragma unroll
  for (int j = 0; j < V::kWords; ++j) s_max[warp][lane * V::kWords + j] = m[j];
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kColsWarps; ++w)
#pragma unroll
    for (int j = 0; j < V::kWords; ++j) m[j] = V::larger(m[j], s_max[w][lane * V::kWords + j]);
  Pow2Scale s[kColsLane];
#pragma unroll
  for (int j = 0; j < kColsLane; ++j)
    s[j] = pow2_scale(__uint_as_float(BF16 ? (j % 2 == 0 ? m[j / 2] << 16 : m[j / 2] & 0xffff0000u) : m[j % V::kWords]));
  if (warp == 0 && col < p.K)
    *reinterpret_cast<float4*>(p.scale + blk * p.K + col) = make_float4(s[0].scale, s[1].scale, s[2].scale, s[3].scale);
#pragma unroll
  for (int j = 0; j < kColsLane; ++j) {
    uint32_t o[kColsRows / 4];
#pragma unroll
    for (int i = 0; i < kColsRows / 4; ++i)
      o[i] = pack4(v[4 * i].get(j) * s[j].inv, v[4 * i + 1].get(j) * s[j].inv, v[4 * i + 2].get(j) * s[j].inv, v[4 * i + 3].get(j) * s[j].inv);
    *reinterpret_cast<uint4*>(&s_q[lane * kColsLane + j][warp * kColsRows]) = make_uint4(o[0], o[1], o[2], o[3]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kColsTile * (kScaleBlock / 16); i += kQuantThreads) {
    const int c = i / (kScaleBlock / 16), part = i % (kScaleBlock / 16);
    const int64_t out_col = int64_t(blockIdx.y) * kColsTile + c;
    if (out_col < p.K)
      *reinterpret_cast<uint4*>(p.q + out_col * p.width + blk * kScaleBlock + part * 16) =
          *reinterpret_cast<const uint4*>(&s_q[c][part * 16]);
  }
}

// ---------------------------------------------------------------------------
// Weights: blocks of 128 x 128, one CTA each, 8 rounds of 16 rows by 128
// columns held in registers.  The transposed copy (the same codes and scales,
// for the product's gradient) turns through shared memory.
// ---------------------------------------------------------------------------
template <bool BF16>
__global__ void __launch_bounds__(kQuantThreads) quantize_weights_kernel(const QuantWeightsParams p) {
  __shared__ uint32_t s_max[kQuantThreads / kWarp];
  __shared__ __align__(16) uint8_t s_t[kScaleBlock][kScaleBlock + 4];
  const int e = blockIdx.z, nb = blockIdx.y, kb = blockIdx.x;
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  const int tr = threadIdx.x / 16, tc = threadIdx.x % 16 * 8;
  const int col = kb * kScaleBlock + tc;
  const int64_t matrix = int64_t(e) * p.N * p.K;
  Values<BF16, 8> v[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = nb * kScaleBlock + i * 16 + tr;
    if (row < p.N && col < p.K) v[i].load(p.w, matrix + int64_t(row) * p.K + col);
    else v[i].zero();
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m = Values<BF16, 8>::larger(m, v[i].largest());
  m = Values<BF16, 8>::bits(m);
  m = __reduce_max_sync(kFull, m);
  if (lane == 0) s_max[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQuantThreads / kWarp; ++w) m = max(m, s_max[w]);
  const Pow2Scale s = pow2_scale(__uint_as_float(m));
  const int nbs = (p.N + kScaleBlock - 1) / kScaleBlock, kbs = (p.K + kScaleBlock - 1) / kScaleBlock;
  if (threadIdx.x == 0) {
    if (p.scale != nullptr) p.scale[(int64_t(e) * nbs + nb) * kbs + kb] = s.scale;
    if (p.scalet != nullptr) p.scalet[(int64_t(e) * kbs + kb) * nbs + nb] = s.scale;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = nb * kScaleBlock + i * 16 + tr;
    uint2 o;
    o.x = v[i].codes(0, s.inv);
    o.y = v[i].codes(4, s.inv);
    if (p.q != nullptr && row < p.N && col < p.K)
      *reinterpret_cast<uint2*>(p.q + matrix + int64_t(row) * p.K + col) = o;
    if (p.qt != nullptr) {
      *reinterpret_cast<uint32_t*>(&s_t[i * 16 + tr][tc]) = o.x;
      *reinterpret_cast<uint32_t*>(&s_t[i * 16 + tr][tc + 4]) = o.y;
    }
  }
  if (p.qt == nullptr) return;
  __syncthreads();
  for (int i = threadIdx.x; i < kScaleBlock * (kScaleBlock / 16); i += kQuantThreads) {
    // neighbouring threads read neighbouring columns of one row
    const int c = i % kScaleBlock, part = i / kScaleBlock;
    const int out_row = kb * kScaleBlock + c, out_col = nb * kScaleBlock + part * 16;
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = uint32_t(s_t[part * 16 + 4 * j][c]) | uint32_t(s_t[part * 16 + 4 * j + 1][c]) << 8 |
             uint32_t(s_t[part * 16 + 4 * j + 2][c]) << 16 | uint32_t(s_t[part * 16 + 4 * j + 3][c]) << 24;
    if (out_row < p.K && out_col < p.N)
      *reinterpret_cast<uint4*>(p.qt + matrix + int64_t(out_row) * p.N + out_col) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace

cudaError_t launch_quantize_rows(const QuantRowsParams& p, bool bf16, cudaStream_t stream) {
  const int kb = (p.K + kScaleBlock - 1) / kScaleBlock;
  const dim3 grid(unsigned((p.M + kRowsTile - 1) / kRowsTile), unsigned((kb + kRowsBlocks - 1) / kRowsBlocks));
  if (bf16) quantize_rows_kernel<true><<<grid, kQuantThreads, 0, stream>>>(p);
  else quantize_rows_kernel<false><<<grid, kQuantThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_quantize_cols(const QuantColsParams& p, bool bf16, cudaStream_t stream) {
  if (p.width == 0) return cudaSuccess;
  const dim3 grid(unsigned(p.width / kScaleBlock), unsigned((p.K + kColsTile - 1) / kColsTile));
  if (bf16) quantize_cols_kernel<true><<<grid, kQuantThreads, 0, stream>>>(p);
  else quantize_cols_kernel<false><<<grid, kQuantThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_quantize_weights(const QuantWeightsParams& p, bool bf16, cudaStream_t stream) {
  const dim3 grid((p.K + kScaleBlock - 1) / kScaleBlock, (p.N + kScaleBlock - 1) / kScaleBlock, p.E);
  if (bf16) quantize_weights_kernel<true><<<grid, kQuantThreads, 0, stream>>>(p);
  else quantize_weights_kernel<false><<<grid, kQuantThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace moe
