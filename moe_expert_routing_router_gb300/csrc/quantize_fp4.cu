// Quantisation to 4 bits (e2m1: 0, 1/2, 1, 3/2, 2, 3, 4, 6 and their negatives) with one
// scale for a block of 32 values of a row, and the values of such blocks.
//
// The scale is the power of two s with 3 < max|x| / s <= 6: dividing by it is exact, no
// value saturates, and each is rounded once (to nearest, ties to even: by at most a fifth
// of itself, or a fourth of s).  It is held as its exponent, a byte; those of the four
// blocks of 128 columns lie in one word, and the words of one block column one row after
// another, as the tiles of a product read them.
//
// Both kernels are bound by memory and move every value once.  Quantising, a team of eight lanes
// holds 128 values of a row, 16 each, so that a block is two neighbouring lanes'.  65560 rows of 4096, bf16:
// 108 us (6.3 TB/s); gathered, eight of each row, 76 us, where the rows come from L2 and 70 percent of the
// issue slots are taken (96, 80, 76 and 76 us with 1, 2, 4 and 8 rows a lane).
#include "block_values.cuh"
#include "quantize_fp4.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace moe {
namespace {

constexpr int kThreads = 256, kLanes = 8, kVals = kScaleBlock / kLanes, kTeams = kWarp / kLanes;
constexpr int kBlocks = 4;                    // columns of a CTA, in blocks of 128
constexpr int kIter = 4;                      // rows of a lane, loaded together
constexpr int kTileRows = kThreads / kWarp / kBlocks * kTeams * kIter;

// Where a lane works: its block column, its first column, and its team's first row.
struct Place {
  int l, kb, col;
  int64_t r0;
  __device__ __forceinline__ Place() {
    const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
    l = lane % kLanes;
    kb = blockIdx.y * kBlocks + warp % kBlocks;
    col = kb * kScaleBlock + l * kVals;
    r0 = int64_t(blockIdx.x) * kTileRows + warp / kBlocks * (kTeams * kIter) + lane / kLanes;
  }
};

template <bool BF16>
__global__ void __launch_bounds__(kThreads) quantize_fp4_kernel(const QuantFp4Params p) {
  using V = Values<BF16, kVals>;
  const Place at;
  if (at.kb * kScaleBlock >= p.K) return;
  // Lane i of the team finds the source of its i-th row.
  const int64_t mine = at.r0 + at.l % kIter * kTeams;
  const int token = at.l < kIter && mine < p.M ? source_row(p.perm, p.k, mine, p.rows) : -1;
  V v[kIter];
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    const int t = __shfl_sync(kFull, token, i, kLanes);
    if (t >= 0 && at.col < p.K) v[i].load(p.x, int64_t(t) * p.K + at.col);
    else v[i].zero();
  }
#pragma unroll
  for (int i = 0; i < kIter; ++i) {
    uint32_t m = v[i].largest();
    m = V::larger(m, __shfl_xor_sync(kFull, m, 1));
    const Fp4Scale s = fp4_scale(V::size(m));
    const uint32_t word = fp4_scale_word(s.code, at.l);
    const int64_t r = at.r0 + i * kTeams;
    if (r >= p.M) continue;
    if (at.l == i) p.scale[int64_t(at.kb) * p.M + r] = word;
    if (at.col >= p.K) continue;
    uint32_t c[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 inv = make_float2(s.inv, s.inv);
      float2 f[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = mul2(make_float2(v[i].get(8 * h + 2 * j), v[i].get(8 * h + 2 * j + 1)), inv);
      c[h] = fp4_pack8(f[0], f[1], f[2], f[3]);
    }
    *reinterpret_cast<uint2*>(p.q + (r * p.K + at.col) / 2) = make_uint2(c[0], c[1]);
  }
}

// A lane writes 8 neighbouring values and a warp 256, so that its stores are whole lines: 129 us for
// 65560 rows of 4096, bf16 (5.3 TB/s, four fifths of it writing), where teams as above took 145.
constexpr int kPiece = 8, kPieces = 4;        // of a lane, loaded together
constexpr int kFp4Block = 32;                 // values that share a scale

template <bool BF16>
__global__ void __launch_bounds__(kThreads) dequantize_fp4_kernel(const DequantFp4Params p) {
  const int per = p.K / kPiece;
  const int64_t pieces = p.M * per, first = int64_t(blockIdx.x) * kPieces * kThreads + threadIdx.x;
  uint32_t c[kPieces], code[kPieces];
#pragma unroll
  for (int n = 0; n < kPieces; ++n) {
    const int64_t i = first + n * kThreads;
    if (i >= pieces) break;
    const int64_t r = i / per;
    const int block = int(i - r * per) / (kFp4Block / kPiece);
    c[n] = reinterpret_cast<const uint32_t*>(p.q)[i];
    code[n] = p.scale[int64_t(block / 4) * p.M + r] >> (block % 4 * 8) & 255u;
  }
#pragma unroll
  for (int n = 0; n < kPieces; ++n) {
    const int64_t i = first + n * kThreads;
    if (i >= pieces) break;
    const float s = fp4_scale_value(code[n]);
    uint32_t u[4];
    fp4_unpack8(c[n], u);
    float2 f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = mul2(__half22float2(*reinterpret_cast<const __half2*>(&u[j])), make_float2(s, s));
    uint4* to = reinterpret_cast<uint4*>(static_cast<char*>(p.y) + i * (kPiece * (BF16 ? 2 : 4)));
    if constexpr (BF16) {                                        // exact: two digits and a power of two
      uint32_t b[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __nv_bfloat162 q = __floats2bfloat162_rn(f[j].x, f[j].y);
        b[j] = *reinterpret_cast<const uint32_t*>(&q);
      }
      to[0] = make_uint4(b[0], b[1], b[2], b[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        to[j] = make_uint4(__float_as_uint(f[2 * j].x), __float_as_uint(f[2 * j].y), __float_as_uint(f[2 * j + 1].x), __float_as_uint(f[2 * j + 1].y));
    }
  }
}

dim3 tiles(int64_t M, int K) {
  const int kb = (K + kScaleBlock - 1) / kScaleBlock;
  return dim3(unsigned((M + kTileRows - 1) / kTileRows), unsigned((kb + kBlocks - 1) / kBlocks));
}

}  // namespace

cudaError_t launch_quantize_fp4(const QuantFp4Params& p, bool bf16, cudaStream_t stream) {
  if (bf16) quantize_fp4_kernel<true><<<tiles(p.M, p.K), kThreads, 0, stream>>>(p);
  else quantize_fp4_kernel<false><<<tiles(p.M, p.K), kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_dequantize_fp4(const DequantFp4Params& p, bool bf16, cudaStream_t stream) {
  const unsigned ctas = unsigned((p.M * (p.K / kPiece) + kPieces * kThreads - 1) / (kPieces * kThreads));
  if (bf16) dequantize_fp4_kernel<true><<<ctas, kThreads, 0, stream>>>(p);
  else dequantize_fp4_kernel<false><<<ctas, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace moe
