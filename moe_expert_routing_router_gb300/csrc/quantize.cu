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
  // amax = m * 2^x, 1 <= m < 2: 448 = 1.75 * 2^8, so the exponent is x - 8, one more where
  // m > 1.75 (the addition carries), and at least -126 (a subnormal amax has it).
  const int n = max(int((b + 0x1fffffu) >> 23) - 8, 1);          // biased; 2^-126 .. 2^120
  Pow2Scale s = {__uint_as_float(uint32_t(n) << 23), __uint_as_float(uint32_t(254 - n) << 23)};
  if (b == 0u) s = {1.f, 1.f};
  if (b >= 0x7f800000u) s = {__uint_as_float(0x7fc00000u), 0.f};
  return s;
}

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return uint32_t(lo) | uint32_t(hi) << 16;
}

__device__ __forceinline__ uint32_t scaled4(float2 x, float2 y, float inv) {
  x = mul2(x, make_float2(inv, inv));
  y = mul2(y, make_float2(inv, inv));
  return pack4(x.x, x.y, y.x, y.y);
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
  // Larger |x|, word by word (bf16: half by half), a NaN above every number.  Signs are
  // whatever they are.
  __device__ __forceinline__ static uint32_t larger(uint32_t a, uint32_t b) {
    uint32_t m;
    if constexpr (BF16) asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(m) : "r"(a), "r"(b));
    else asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(*reinterpret_cast<float*>(&m)) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
    return m;
  }
  // |x| of the larger half (bf16), or of the word; of one half.
  __device__ __forceinline__ static float size(uint32_t m) {
    if constexpr (BF16) return __uint_as_float(max(m << 16 & 0x7fffffffu, m & 0x7fff0000u));
    else return __uint_as_float(m & 0x7fffffffu);
  }
  __device__ __forceinline__ static float size(uint32_t m, int half) {
    return __uint_as_float((half == 0 ? m << 16 : m) & (BF16 ? 0x7fff0000u : 0x7fffffffu));
  }
  __device__ __forceinline__ uint32_t largest() const {
    uint32_t m = w[0];
#pragma unroll
    for (int i = 1; i < kWords; ++i) m = larger(m, w[i]);
    return m;
  }
  // Four neighbouring values from the i-th on, scaled and rounded.
  __device__ __forceinline__ uint32_t codes(int i, float inv) const {
    return scaled4(make_float2(get(i), get(i + 1)), make_float2(get(i + 2), get(i + 3)), inv);
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
// Rows: blocks of 1 x 128.  Eight lanes, a team, hold a block, 16 values each; a
// warp takes 16 rows of one block column, four at a time, so that their scales,
// which lie one row after another, leave together.  A team's four maxima are
// reduced at once: every step halves what a lane holds, and lane i ends with the
// i-th.  A CTA takes 32 rows by 4 blocks of columns.  65,536 rows of 2048 bf16: 61
// us, 6.7 TB/s; 65,536 x 4096 gathered from 8192 rows: 70 us, where the reads from
// L2 and the instructions (6 a value) bound it.
// ---------------------------------------------------------------------------
constexpr int kRowsTile = 32, kRowsBlocks = 4, kQuantThreads = 256, kRowLanes = 8, kRowVals = kScaleBlock / kRowLanes;

template <bool BF16>
__global__ void __launch_bounds__(kQuantThreads) quantize_rows_kernel(const QuantRowsParams p) {
  using V = Values<BF16, kRowVals>;
  constexpr int kIter = 4, kTeams = kWarp / kRowLanes, kWarpRows = kIter * kTeams;
  static_assert(kRowsBlocks * kRowsTile == kQuantThreads / kWarp * kWarpRows, "a CTA's warps cover its tile");
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp, team = lane / kRowLanes, l = lane % kRowLanes;
  const int kb = blockIdx.y * kRowsBlocks + warp % kRowsBlocks, col = kb * kScaleBlock + l * kRowVals;
  const int64_t r0 = int64_t(blockIdx.x) * kRowsTile + warp / kRowsBlocks * kWarpRows + team;
  if (kb * kScaleBlock >= p.K) return;
  // Lane i of the team finds the source of its i-th row.
  const int64_t mine = r0 + (l % kIter) * kTeams;
  const int token = l < kIter && mine < p.M ? source_row(p.perm, p.k, mine, p.rows) : -1;
  V v[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int t = __shfl_sync(kFull, token, i, kRowLanes);
    if (t >= 0 && col < p.K) v[i].load(p.x, int64_t(t) * p.K + col);
    else v[i].zero();
  }
  uint32_t m[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) m[i] = v[i].largest();
  const bool odd = l & 1, upper = l & 2;
  const uint32_t a = V::larger(odd ? m[1] : m[0], __shfl_xor_sync(kFull, odd ? m[0] : m[1], 1));
  const uint32_t b = V::larger(odd ? m[3] : m[2], __shfl_xor_sync(kFull, odd ? m[2] : m[3], 1));
  uint32_t top = V::larger(upper ? b : a, __shfl_xor_sync(kFull, upper ? a : b, 2));
  top = V::larger(top, __shfl_xor_sync(kFull, top, 4));
  const Pow2Scale s = pow2_scale(V::size(top));
  if (l < kIter && mine < p.M) p.scale[int64_t(kb) * p.M + mine] = s.scale;
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const float inv = __shfl_sync(kFull, s.inv, i, kRowLanes);
    const int64_t r = r0 + i * kTeams;
    if (r < p.M && col < p.K)
      *reinterpret_cast<uint4*>(p.q + r * p.K + col) = make_uint4(v[i].codes(0, inv), v[i].codes(4, inv), v[i].codes(8, inv), v[i].codes(12, inv));
  }
}

// ---------------------------------------------------------------------------
// Columns: blocks of 128 rows of one expert by one column, written transposed
// (the rows become the contraction of a weight gradient).  Expert e's rows
// start at column 128 * (sum over e' < e of ceil(kept[e'] / 128)); its last
// block ends in zeros.  A tile is one block of rows by 128 columns: a lane holds
// 8 columns of 8 rows, the maxima meet in shared memory, and the bytes turn
// through shared memory into rows of 128.  A CTA stays, takes neighbouring
// tiles, those of one block of rows first, and loads the next tile as soon as
// the codes of this one are in shared memory.  30,018 x 2048 bf16, a fourteenth of
// the rows dropped: 35 us, 4.9 TB/s
// (39 us with a CTA a tile and lanes of 4 columns); the loads' latency between the
// barriers bounds it.
// ---------------------------------------------------------------------------
constexpr int kColsTile = 128, kColsLane = 8, kColsRows = 8, kColsWarps = kQuantThreads / kWarp, kColsWarpRows = kScaleBlock / kColsWarps;
static_assert(kColsTile / kColsLane * 2 == kWarp && kColsWarpRows == 2 * kColsRows, "half a warp a row, the other half the rows behind");

// CTAs of an SM: what the registers of a tile leave room for.
template <bool BF16>
constexpr int kColsCtas = BF16 ? 4 : 2;

// The rows of block `blk` of the output, by all lanes of a warp: the first row and how
// many (0: behind the last expert).
__device__ __forceinline__ void cols_block(const QuantColsParams& p, int blk, int lane, int64_t& row, int& rows) {
  rows = 0;
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
    const int64_t first = before + incl - nb, at = (blk - first) * kScaleBlock;
    const unsigned here = __ballot_sync(kFull, blk >= first && blk < first + nb);
    if (here != 0u) {
      row = __shfl_sync(kFull, lo + at, __ffs(here) - 1);
      rows = int(__shfl_sync(kFull, min(n - at, int64_t(kScaleBlock)), __ffs(here) - 1));
      return;
    }
    before += __shfl_sync(kFull, incl, kWarp - 1);
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kQuantThreads, kColsCtas<BF16>) quantize_cols_kernel(const QuantColsParams p) {
  using V = Values<BF16, kColsLane>;
  constexpr int kCols = BF16 ? 2 : 1;                            // columns of a word
  __shared__ __align__(16) uint32_t s_max[kColsWarps][kColsTile / kCols];
  __shared__ __align__(16) float s_inv[kColsTile];
  // Column c's pieces of 16 bytes in the order part ^ (c / 8 % 8), their halves exchanged
  // from column 64 on: neither side meets bank conflicts.
  __shared__ __align__(16) uint8_t s_q[kColsTile][kScaleBlock];
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp, cl = lane % 16, half = lane / 16;
  const int ct = (p.K + kColsTile - 1) / kColsTile;
  const int64_t tiles = p.width / kScaleBlock * ct, from = blockIdx.x * p.share;
  int left = int(min(p.share, tiles - from)), blk = int(from / ct), known = -1;
  int c0 = int(from - int64_t(blk) * ct) * kColsTile, rows = 0, token = -1;
  V v[kColsRows];
  const auto fetch = [&]() {                                     // the same in all warps: whether the block has rows
    if (blk != known) {
      known = blk;
      int64_t row = 0;
      cols_block(p, blk, lane, row, rows);
      // Lane i finds the source of the warp's i-th row.
      const int r = warp * kColsWarpRows + lane;
      token = lane < kColsWarpRows && r < rows ? source_row(p.perm, p.k, row + r, p.rows) : -1;
    }
    if (rows == 0) return;
    const int col = c0 + cl * kColsLane;
#pragma unroll
    for (int i = 0; i < kColsRows; ++i) {
      const int t = __shfl_sync(kFull, token, half * kColsRows + i);
      if (t >= 0 && col < p.K) v[i].load(p.x, int64_t(t) * p.K + col);
      else v[i].zero();
    }
  };
  fetch();
  while (left > 0) {
    const int to = blk * kScaleBlock, to_c0 = c0;
    const bool there = rows != 0;                                // behind the last expert: left as it is
    if (there) {
#pragma unroll
      for (int j = 0; j < V::kWords; ++j) {                      // a word of columns each
        uint32_t m = v[0].w[j];
#pragma unroll
        for (int i = 1; i < kColsRows; ++i) m = V::larger(m, v[i].w[j]);
        m = V::larger(m, __shfl_xor_sync(kFull, m, 16));
        if (half == j % 2) s_max[warp][cl * V::kWords + j] = m;
      }
      __syncthreads();
      if (threadIdx.x < kColsTile / kCols) {
        uint32_t m = s_max[0][threadIdx.x];
#pragma unroll
        for (int w = 1; w < kColsWarps; ++w) m = V::larger(m, s_max[w][threadIdx.x]);
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
          const Pow2Scale s = pow2_scale(V::size(m, BF16 ? j : 1));
          const int c = threadIdx.x * kCols + j;
          s_inv[c] = s.inv;
          if (c0 + c < p.K) p.scale[int64_t(blk) * p.K + c0 + c] = s.scale;
        }
      }
      __syncthreads();
      float4 inv4;
#pragma unroll
      for (int j = 0; j < kColsLane; ++j) {
        if (j % 4 == 0) inv4 = *reinterpret_cast<const float4*>(&s_inv[cl * kColsLane + j]);
        const float inv = j % 4 == 0 ? inv4.x : j % 4 == 1 ? inv4.y : j % 4 == 2 ? inv4.z : inv4.w;
        uint2 o;
        o.x = scaled4(make_float2(v[0].get(j), v[1].get(j)), make_float2(v[2].get(j), v[3].get(j)), inv);
        o.y = scaled4(make_float2(v[4].get(j), v[5].get(j)), make_float2(v[6].get(j), v[7].get(j)), inv);
        *reinterpret_cast<uint2*>(&s_q[cl * kColsLane + j][(warp ^ (cl & 7)) * 16 + (half ^ cl >> 3) * 8]) = o;
      }
    }
    if ((c0 += kColsTile) >= p.K) {
      c0 = 0;
      ++blk;
    }
    if (--left > 0) fetch();
    if (!there) continue;
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kColsTile * (kScaleBlock / 16) / kQuantThreads; ++n) {
      const int c = threadIdx.x / (kScaleBlock / 16) + n * (kQuantThreads / (kScaleBlock / 16)), part = threadIdx.x % (kScaleBlock / 16);
      uint4 o = *reinterpret_cast<const uint4*>(&s_q[c][(part ^ (c / kColsLane & 7)) * 16]);
      if (c >= kColsTile / 2) o = make_uint4(o.z, o.w, o.x, o.y);
      if (to_c0 + c < p.K) *reinterpret_cast<uint4*>(p.q + int64_t(to_c0 + c) * p.width + to + part * 16) = o;
    }                                                            // read before the next barrier, behind which it is written again
  }
}

// ---------------------------------------------------------------------------
// Weights: blocks of 128 x 128, one CTA each, 8 rounds of 16 rows by 128
// columns held in registers.  The transposed copy (the same codes and scales,
// for the product's gradient) turns through shared memory.  16 x 2048 x 4096 bf16:
// 58 us, 7.0 TB/s; with the transposed copy 84 us, 6.4 TB/s.
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
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int row = nb * kScaleBlock + i * 16 + tr;
    if (row < p.N && col < p.K) v[i].load(p.w, matrix + int64_t(row) * p.K + col);
    else v[i].zero();
  }
  uint32_t m = v[0].largest();
#pragma unroll
  for (int i = 1; i < 8; ++i) m = Values<BF16, 8>::larger(m, v[i].largest());
  // as bits, a NaN above every number
  m = __reduce_max_sync(kFull, __float_as_uint(Values<BF16, 8>::size(m)));
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

cudaError_t launch_quantize_cols(QuantColsParams p, bool bf16, int sms, cudaStream_t stream) {
  const int64_t tiles = p.width / kScaleBlock * ((p.K + kColsTile - 1) / kColsTile);
  const int64_t ctas = int64_t(sms) * (bf16 ? kColsCtas<true> : kColsCtas<false>);
  if (tiles == 0) return cudaSuccess;
  p.share = (tiles + ctas - 1) / ctas;
  const unsigned grid = unsigned((tiles + p.share - 1) / p.share);
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
