// The experts of a layer for the few tokens of a decode step:
//
//   h_a = glu(W1_e x_t),  out_t = sum_j gate_tj W2_e h_a      a = (t, j), e = idx_tj
//
// in two kernels (and a small one), of which each reads the weights of the experts that have tokens once;
// that reading is what bounds them.  (The tensor core's own 4-bit and 8-bit products take
// 128 rows at a time and quantised activations; here an expert has a token or two.)
//
// Both kernels have the same body.  A tile is 16 rows of one expert's weights; the tiles of
// all experts with tokens are split evenly, in order, over one CTA per SM, and the warps of a
// CTA share the contraction of a tile, in units of 128.  Weights go from memory into registers,
// 16 bytes of a row a lane, 4 KB a warp ahead; codes become fp16, which holds them exactly, and
// meet the tokens in mma.sync m16n8k16 with the weights' rows as M and the tokens as N.
// The order of the contraction is free, so a lane's 16 bytes are its share of the steps as they lie.
//   e4m3:    a scale stands for a unit; a product's eight columns are eight tokens.
//   4 bits:  a lane's 16 bytes are one block of 32, with a scale of its own, and the four lanes of
//            a row hold the four blocks of a unit, which one product would add up.
//            Up to 4 tokens: a token takes four of the eight columns, and each sees one block: the
//            other lanes' part of its column is zero.  Sums come out by block, and are multiplied by its scale.
//            More: the codes are multiplied, as fp16, by their scale over the largest of the four,
//            a power of two (exact down to 2^-23 of it), whose own multiplies the unit's sum.  Tiles with a scale
//            that is 2^-16 of it or less are left to `run_far`.
// The tokens' values are staged in shared memory as fp16 with a power of two for each 128, so that
// their largest is between 2^14 and 2^15: bf16 values are exact down to 2^-28 of it, and the fp32
// values of h are rounded to 11 bits (three more than bf16 has).  All sums are fp32.
// A unit's sum, of codes times such values, is multiplied by the token's power and then by the weights' scale.  Where a
// power is so far from one that the first product could leave fp32 though the second comes back, `run_far` takes the
// tiles, in an order that cannot.
//
// What is under way waits in L1, so that shared memory is kept small: eight tokens of an expert are
// staged at a time, or up to 16, and more take the same tiles again, some at a time, from L2.
// (64 tokens, 8 of 64 experts of 4096 and 2048, 8 bits: 309 us with 144 KB of shared memory, 351 with 182 KB.)
// Copies to shared memory were slower, in an earlier form that took 231 us for 16 tokens: of 16 bytes a lane 320, tensor copies
// of 8 x 128 bytes by each warp 298, of 8 x 2048 by a producer warp 268, bulk copies of rows 309.
//
// The first kernel's tiles are 8 rows of the gate and the 8 rows of the other half that go
// with them.  The second one's sums go to memory by assignment, and a third, small kernel adds
// them up by gate, in the order of j: no result depends on an order of arrival.  Each is launched while
// the one before it ends (programmatic dependent launch); the second has its first weights under way
// when the first one is done.
//
// 8 of 64 experts of 4096 and 2048, a call in a graph, with the share of the measured copy rate at which weights are read:
//            1 token        4             16             32             64 tokens
//   4 bits   30 us, 53 %    73 us, 68 %   165 us, 67 %   226 us, 56 %   303 us, 42 %
//   8 bits   42 us, 73 %                  217 us, 96 %                  309 us, 78 %
// About 10 us of each are the launches, the lists and the sums over experts.  4 bits: unpacking and scaling beside the loads, for
// every time that a tile is taken; from 12 tokens of an expert on that costs more than 8-bit weights' reading.  Other sizes:
// 16 tokens, 8 of 128 experts of 2048 and 768: 73 us (4 bits) and 90 (8), a floor of 29 and 55, since 10 of 16 warps have no unit of
// the second contraction; 8 of 128 of 7168 and 2048, 4 bits: 363 us, a floor of 273.
#pragma once

#include "block_values.cuh"
#include "layer_small.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

namespace moe {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / kWarp;
constexpr int kRows = 16;                     // of a tile
constexpr int kUnit = 128;                    // of the contraction, taken by a warp at a time
constexpr int kTokens = 8;                    // columns of a product
constexpr int kFew = 4;                       // tokens that take four columns each
constexpr int kChunk = 16;                    // tiles that are taken again for more tokens
constexpr int kMaxE = 1024, kMaxA = kSmallTokens * 8;
constexpr int kZeros = 2 * kUnit;             // bytes: a token's unit where there is none
constexpr uint32_t kOnes = 0x01010101u;       // a byte each
constexpr int kMaxSlots = 8;                  // tiles whose parts are added up together

extern __shared__ __align__(16) uint8_t s_dyn[];                 // begins with kZeros bytes of zeros

struct Lists {
  int order[kMaxA];                           // assignments by expert
  int count[kMaxE];                           // the place of an expert's first assignment
  int share[2 * kWarps];                      // assignments and experts of a warp's share of the experts
  int expert[kMaxA], start[kMaxA + 1];        // of the experts that have tokens: which, and where theirs start
  int work[kMaxA];                            // what stands before them, by tile
  int tile0[kMaxA], tile1[kMaxA];             // their tiles that are this CTA's
  int far, apart;                             // a power of the staged tokens is far from one; four scales are far from one another
  int active, run0, run1;                     // experts that have tokens; the first and last of which this CTA has tiles
};

// What a tile of an expert with n tokens takes, in eighths of one that its weights' reading
// bounds: `cap` tokens are taken at a time.  (Of 64 experts of 4096 and 2048 with 1, 4, 8, 12 and 16 tokens
// each one takes, 13 or 14 at a time, 2.7, 3.5, 3.6, 5.6 and 9.8 us at 4 bits, 4.0, 4.1, 4.4, 5.3 and 9.1 at 8.  Where
// experts' tokens differ, of 64 with 8 of 64 experts each, 8 more for a time over the tiles that is not the last
// share the work best: 304 us, with 2 more 336, in the form of that time.)
template <bool FP4>
__device__ __forceinline__ int tile_cost(int n, int cap) {
  const auto pass = [](int tokens) {
    if (tokens <= kFew / 2) return 8;
    if (tokens <= kFew) return FP4 ? 11 : 8;
    if (tokens <= kTokens) return FP4 ? 11 : 9;
    return FP4 ? 16 : 11;
  };
  const int passes = (n + cap - 1) / cap, rest = n - (passes - 1) * cap;
  return (passes - 1) * (pass(cap) + 8) + pass(rest);
}

__device__ __forceinline__ int warp_prefix(int v, int lane) {    // with the lane's own
#pragma unroll
  for (int off = 1; off < kWarp; off <<= 1) {
    const int o = __shfl_up_sync(kFull, v, off);
    if (lane >= off) v += o;
  }
  return v;
}

// The experts that have tokens, their assignments in order, and which of their tiles are this CTA's.  All threads.
template <bool FP4>
__device__ __forceinline__ void plan(Lists& s, const SmallLayerParams& p, int tiles, int cap) {
  const int A = p.T * p.k, lane = threadIdx.x % kWarp;
  const unsigned below = (1u << lane) - 1u;
  int e = threadIdx.x < A ? p.idx[threadIdx.x] : -1;             // A is kThreads at most
  if (e < 0 || e >= p.E) e = -1;
  if (A <= kWarp) {                                              // one warp: groups of equal experts, by their first
    if (threadIdx.x < kWarp) {
      const unsigned peers = __match_any_sync(kFull, e);
      const int leader = e >= 0 ? __ffs(peers) - 1 : -1;
      const unsigned leaders = __ballot_sync(kFull, leader == lane);
      const int n = leader == lane ? __popc(peers) : 0, start = warp_prefix(n, lane) - n;
      const int first = __shfl_sync(kFull, start, max(leader, 0));
      if (e >= 0) s.order[first + __popc(peers & below)] = lane;
      if (leader == lane) {
        s.expert[__popc(leaders & below)] = e;
        s.start[__popc(leaders & below)] = start;
      }
      if (lane == kWarp - 1) {
        s.active = __popc(leaders);
        s.start[__popc(leaders)] = start + n;
      }
    }
  } else {
    // How many of an expert's assignments each warp has, in a byte; the warps list 32 experts at a time each.
    uint4* const table = reinterpret_cast<uint4*>(s_dyn + kZeros);
    for (int i = threadIdx.x; i < p.E; i += kThreads) table[i] = make_uint4(0u, 0u, 0u, 0u);
    const unsigned peers = __match_any_sync(kFull, e);
    const int warp = threadIdx.x / kWarp;
    __syncthreads();
    if (e >= 0 && __ffs(peers) - 1 == lane) reinterpret_cast<uint8_t*>(table + e)[warp] = uint8_t(__popc(peers));
    __syncthreads();
    const auto sum = [](uint4 v) { return int(__dp4a(v.x, kOnes, __dp4a(v.y, kOnes, __dp4a(v.z, kOnes, __dp4a(v.w, kOnes, 0u))))); };
    constexpr int kGroups = kMaxE / kThreads;                    // of 32 experts, of a warp
    const int e0 = warp * kGroups * kWarp + lane;
    int n[kGroups], incl[kGroups], all = 0, some = 0;
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      n[i] = e0 + i * kWarp < p.E ? sum(table[e0 + i * kWarp]) : 0;
      incl[i] = all + warp_prefix(n[i], lane);
      all = __shfl_sync(kFull, incl[i], kWarp - 1);
      some += __popc(__ballot_sync(kFull, n[i] > 0));
    }
    if (lane == 0) {
      s.share[warp] = all;
      s.share[kWarps + warp] = some;
    }
    int place = __popc(peers & below);                           // among the assignments of its expert
    if (e >= 0) {
      uint4 v = table[e];
      const auto before = [&](int i) { return warp / 4 > i ? 0xffffffffu : warp / 4 == i ? (1u << warp % 4 * 8) - 1u : 0u; };
      place += sum(make_uint4(v.x & before(0), v.y & before(1), v.z & before(2), v.w & before(3)));
    }
    __syncthreads();
    const int shares = lane < kWarps ? s.share[lane] : 0, experts = lane < kWarps ? s.share[kWarps + lane] : 0;
    const int first = __reduce_add_sync(kFull, lane < warp ? shares : 0);
    int at = __reduce_add_sync(kFull, lane < warp ? experts : 0);
#pragma unroll
    for (int i = 0; i < kGroups; ++i) {
      const unsigned mask = __ballot_sync(kFull, n[i] > 0);
      if (n[i] > 0) {
        const int to = at + __popc(mask & below);
        s.expert[to] = e0 + i * kWarp;
        s.start[to] = s.count[e0 + i * kWarp] = first + incl[i] - n[i];
      }
      at += __popc(mask);
    }
    if (warp == kWarps - 1 && lane == 0) {
      s.active = at;
      s.start[at] = first + all;
    }
    __syncthreads();
    if (e >= 0) s.order[s.count[e] + place] = threadIdx.x;
  }
  if (threadIdx.x < kWarp) {
    __syncwarp();
    const int active = s.active;
    int all = 0;
    for (int at0 = 0; at0 < active; at0 += kWarp) {
      const int at = at0 + lane, c = at < active ? tile_cost<FP4>(s.start[at + 1] - s.start[at], cap) : 0, incl = warp_prefix(c, lane);
      if (at < active) s.work[at] = (all + incl - c) * tiles;
      all += __shfl_sync(kFull, incl, kWarp - 1);
    }
    // the tiles whose work, in order, begins in the CTA's share; all of it is less than 2^24
    const int from = int(uint32_t(all * tiles) * blockIdx.x / gridDim.x), to = int(uint32_t(all * tiles) * (blockIdx.x + 1) / gridDim.x);
    int run0 = kMaxA, run1 = -1;
    for (int at0 = 0; at0 < active; at0 += kWarp) {
      const int at = at0 + lane;
      int t0 = 0, t1 = 0;
      if (at < active) {
        const int w = s.work[at], c = tile_cost<FP4>(s.start[at + 1] - s.start[at], cap);
        t0 = from > w ? min((from - w + c - 1) / c, tiles) : 0;
        t1 = to > w ? min((to - w + c - 1) / c, tiles) : 0;
        s.tile0[at] = t0;
        s.tile1[at] = t1;
      }
      const unsigned some = __ballot_sync(kFull, t0 < t1);
      if (some != 0u) {
        run0 = min(run0, at0 + __ffs(some) - 1);
        run1 = at0 + kWarp - 1 - __clz(some);
      }
    }
    if (lane == 0) {
      s.run0 = run0;
      s.run1 = run1;
    }
  }
  __syncthreads();
}
static_assert(kMaxA <= kThreads && kWarps == 16 && kMaxE % kThreads == 0, "an assignment a thread, a byte a warp");

// Where a CTA's shared memory lies behind the lists.
struct Staged {
  int x;                                      // offset of [cap] rows of `pitch` bytes: fp16
  float* power;                               // [units][columns]: what a token's 128 values were divided by
  float* red;                                 // [tiles][warps][tokens][16]: the warps' parts of tiles
  int pitch, columns, units;
  int slots;                                  // tiles times tokens that `red` holds
};

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A unit's sum is at most 2^31 and a multiple of 2^-33: its product with a power in [2^-93, 2^96], one over
// 2^(up - 127), is exact, and then any scale may follow.
constexpr uint32_t kNearest = 127 - 96, kFarthest = 127 + 93;
// to + sum power scale, rounded once, for any power.
__device__ __forceinline__ float add_scaled(float sum, float power, float scale, float to) {
  const float c = power * scale;                                 // exact where it is a normal number
  if ((fabsf(c) >= 0x1p-126f && fabsf(c) < __int_as_float(0x7f800000)) || scale == 0.f) return fmaf(sum, c, to);
  return fmaf(sum * power, scale, to);                           // both are above 1; or power is below 2^24, and where it is below 1 so is scale
}

// Rows `order[first ..]` of the tokens (UP: bf16 x) or of the assignments (h), as fp16, in pieces of a
// unit of a row a warp, four at a time; the rest of the last unit is zero.
constexpr int kPieces = 4;
template <bool UP>
__device__ __forceinline__ void fetch(const SmallLayerParams& p, const Lists& s, const Staged& m, int first, int n, int i0, uint32_t (&v)[kPieces][UP ? 2 : 4]) {
  const int K = UP ? p.H : p.I, lane = threadIdx.x % kWarp;
#pragma unroll
  for (int d = 0; d < kPieces; ++d) {
    const int i = i0 + d * kWarps, row = i / m.units, c = (i - row * m.units) * kUnit + lane * 4;
#pragma unroll
    for (int j = 0; j < (UP ? 2 : 4); ++j) v[d][j] = 0u;
    if (row < n && c < K) {                                      // K is a multiple of 16
      const int a = s.order[first + row];
      if constexpr (UP) {
        const void* x = static_cast<const __nv_bfloat16*>(p.x) + int64_t(a / p.k) * K + c;   // in front of the weights' loads
        asm volatile("ld.global.nc.v2.u32 {%0, %1}, [%2];" : "=r"(v[d][0]), "=r"(v[d][1]) : "l"(x));
      } else {
        const uint4 w = __ldcg(reinterpret_cast<const uint4*>(p.h + int64_t(a) * K + c));
        v[d][0] = w.x;
        v[d][1] = w.y;
        v[d][2] = w.z;
        v[d][3] = w.w;
      }
    }
  }
}
template <bool UP>
__device__ __forceinline__ void put(Lists& s, const Staged& m, int n, int i0, const uint32_t (&v)[kPieces][UP ? 2 : 4]) {
  const int lane = threadIdx.x % kWarp;
#pragma unroll
  for (int d = 0; d < kPieces; ++d) {
    const int i = i0 + d * kWarps, row = i / m.units, u = i - row * m.units;
    if (row >= n) break;                                         // the whole warp
    uint32_t f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = UP ? (j % 2 == 0 ? v[d][j / 2] << 16 : v[d][j / 2] & 0xffff0000u) : v[d][UP ? 0 : j];
    const uint32_t top = __reduce_max_sync(kFull, max(max(f[0] & 0x7fffffffu, f[1] & 0x7fffffffu), max(f[2] & 0x7fffffffu, f[3] & 0x7fffffffu)));
    // 2^14 over the power of two at or below the largest, as far as both it and its inverse are normal
    const uint32_t up = min(268u - (top >> 23), 253u);
    const float by = __uint_as_float(up << 23);
    *reinterpret_cast<uint2*>(s_dyn + m.x + row * m.pitch + (u * kUnit + lane * 4) * 2) =
        make_uint2(pack_half2(__uint_as_float(f[0]) * by, __uint_as_float(f[1]) * by), pack_half2(__uint_as_float(f[2]) * by, __uint_as_float(f[3]) * by));
    if (lane == 0) m.power[u * m.columns + row] = __uint_as_float((254u - up) << 23);
    if (up - kNearest > kFarthest - kNearest && top != 0u && top < 0x7f800000u) s.far = 1;   // zeros and infinities stay so in any order
  }
}

__device__ __forceinline__ uint4 load_weights(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t load_scale(const void* p) {
  uint32_t v;
  asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// Four e4m3 codes as fp16.
__device__ __forceinline__ void e4m3_half(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(uint16_t(codes)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(uint16_t(codes >> 16)));
}
// Two exponents' powers of two, 255 a NaN.
__device__ __forceinline__ float2 two_scales(uint32_t both) {
  uint32_t b;
  asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(b) : "h"(uint16_t(both)));
  return make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
}
// The largest of a word's four exponents; the word becomes what they lack to it.
__device__ __forceinline__ uint32_t largest_scale(uint32_t& w) {
  const uint32_t top = max(max(w & 255u, w >> 8 & 255u), max(w >> 16 & 255u, w >> 24));
  w = top * 0x01010101u - w;
  return top;
}
// The power of two that the t-th of them lacks, in both halves.
__device__ __forceinline__ uint32_t lacking(uint32_t w, int t) {
  const float f = __uint_as_float((127u - min(__byte_perm(w, 0u, 0x4440u + t), 126u)) << 23);
  return pack_half2(f, f);
}
__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
  asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
  return a;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// Within |g| + 8 roundings of 2^-24, of a value that is rounded to 11 bits.
__device__ __forceinline__ float silu(float g) {
  const float t = __expf(-fabsf(g)), r = 1.f / (1.f + t);
  return g * (g >= 0.f ? r : t * r);
}

// The sums of `tiles` tiles from the `done`-th on, of the warps' parts in their order, to where they belong.
template <bool UP>
__device__ __forceinline__ void add_parts(const SmallLayerParams& p, const Lists& s, const float* red, int done, int tiles, int first, int n) {
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  for (int o0 = warp * kWarp; o0 < tiles * n * kRows; o0 += kThreads) {
    const int o = o0 + lane, at = o / (n * kRows), in = o - at * n * kRows, row = in % kRows;
    const bool live = at < tiles;
    float sum = 0.f;
    if (live) {
#pragma unroll
      for (int i = 0; i < kWarps; ++i) sum += red[(at * kWarps + i) * n * kRows + in];
    }
    const int64_t a = live ? s.order[first + in / kRows] : 0;
    if constexpr (UP) {
      const float other = __shfl_down_sync(kFull, sum, 8);
      if (live && row < 8) p.h[a * p.I + (done + at) * 8 + row] = silu(sum) * other;
    } else {
      if (live) p.y[a * p.H + (done + at) * kRows + row] = sum;
    }
  }
}

// Tiles [tile0, tile1) of expert e for the `n` tokens whose assignments are order[first ..],
// which are staged meanwhile.  A warp has PER units of each tile, next to one another; WHOLE: all warps
// have, and no unit ends inside.  NT products are side by side, of eight tokens each or (FEW, 4 bits) of two.
template <bool FP4, bool UP, int PER, bool WHOLE, bool FEW, int NT>
__device__ __forceinline__ void run_tiles(const SmallLayerParams& p, Lists& s, const Staged& m, int e, int tile0, int tile1, int first, int n) {
  constexpr int L = FP4 ? 1 : 2, UB = 64 * L;                    // 16-byte pieces a lane, and bytes, of a row's unit
  constexpr int D = FP4 && (FEW || NT == 1) ? 4 : 2;             // units under way
  constexpr int kTile = UP ? 8 : kRows;                          // rows from a tile to the next
  constexpr int TPI = PER < D ? D / PER : 1;                     // tiles of a round, which takes whole turns of the ring
  constexpr int SW = FP4 ? (PER + 1) / 2 : 1;                    // a lane's scale words of a tile
  constexpr bool kHeld = NT * PER <= 2;                          // the tokens' values stay in registers
  constexpr int V = FEW ? 2 : 4;                                 // sums of a lane in a product
  static_assert(FP4 || !FEW, "blocks of a column");
  const int K = UP ? p.H : p.I, N = UP ? 2 * p.I : p.H;
  const SmallWeights& w = UP ? p.w1 : p.w2;
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp, g = lane / 4, t = lane % 4;
  const int row_bytes = FP4 ? K / 2 : K;
  const int others = UP ? p.I : 8;                               // from a tile's first 8 rows to its others
  const int kblocks = (K + 127) / 128;
  const int u0 = warp * PER;
  const uint32_t last_used = WHOLE || K % kUnit == 0 ? 0xffffffffu : (1u << K % kUnit / 4) - 1u;   // of the last unit's scales: others may be anything

  uint4 ring[D][2 * L];
  uint32_t scale[TPI + 1][SW];                                   // of a round's tiles; PER >= D: of this tile and the next
  uint32_t fresh[kPieces][UP ? 2 : 4];
  if constexpr (UP) fetch<UP>(p, s, m, first, n, warp, fresh);   // in front of the weights, behind which it would wait
  int off[PER * L];                                              // not WHOLE: of the lane's pieces in a row; those behind its end,
#pragma unroll                                                   // which meet zeros, are its first
  for (int i = 0; i < PER * L; ++i) {
    const int c = u0 * UB + i * 64 + t * 16;
    off[i] = WHOLE || c < row_bytes ? c : 0;
  }
  const int64_t row0 = int64_t(e) * N + tile0 * kTile;
  const uint8_t* from = w.q + (row0 + g) * row_bytes + (WHOLE ? u0 * UB + t * 16 : 0);
  const uint8_t* from2 = from + int64_t(others) * row_bytes;
  const int tile_bytes = kTile * row_bytes;
  // A lane's share of a tile's scales.  4 bits: lanes t = 0 and 1 the words of rows g and g + 8
  // of a unit, t = 2 and 3 those of the next; e4m3: lane l that of the first (l even) or the other rows of unit l / 2.
  const uint32_t* words = nullptr;
  const float* blocks = nullptr;
  int64_t word_step = 0;
  if constexpr (FP4) {
    words = static_cast<const uint32_t*>(w.scale) + int64_t(min(u0 + (PER > 1 ? t / 2 : 0), m.units - 1)) * p.E * N + row0 + g + (t % 2) * others;
    word_step = int64_t(p.E) * N;
  } else {
    blocks = static_cast<const float*>(w.scale) + int64_t(e) * ((N + 127) / 128) * kblocks + min(u0 + lane / 2 % PER, m.units - 1);
  }
  int lt = tile0;                                                // the tile that is loaded from
  const auto load = [&](uint4 (&to)[2 * L], int lu) {
#pragma unroll
    for (int i = 0; i < L; ++i) {
      to[2 * i] = load_weights(from + (WHOLE ? lu * UB + i * 64 : off[lu * L + i]));
      to[2 * i + 1] = load_weights(from2 + (WHOLE ? lu * UB + i * 64 : off[lu * L + i]));
    }
  };
  const auto load_scales = [&](uint32_t (&sc)[SW]) {
    if constexpr (FP4) {
#pragma unroll
      for (int i = 0; i < SW; ++i) {
        const uint32_t* q = words + i * 2 * word_step;
        if (!WHOLE && i > 0 && u0 + i * 2 + t / 2 >= m.units) q = words;   // of no unit
        sc[i] = load_scale(q);
      }
    } else {
      sc[0] = load_scale(blocks + (lt * kTile + lane % 2 * others) / 128 * kblocks);
    }
  };
  const auto next_tile = [&]() {                                 // behind the last one, again that
    if (++lt < tile1) {
      from += tile_bytes;
      from2 += tile_bytes;
      if constexpr (FP4) words += kTile;
    } else {
      lt = tile1 - 1;
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) {
    if (d % PER == 0) load_scales(scale[d / PER]);
    load(ring[d], d % PER);
    if (d % PER == PER - 1) next_tile();
  }
  if constexpr (!UP) {
    asm volatile("griddepcontrol.wait;" ::: "memory");           // h is there
    fetch<UP>(p, s, m, first, n, warp, fresh);
  }
  if (threadIdx.x == 0) s.far = s.apart = 0;                               // all have read what it was: they have met since
  __syncthreads();                                               // the tokens before, and their parts, are no longer read
  put<UP>(s, m, n, warp, fresh);
  for (int i = warp + kPieces * kWarps; i < n * m.units; i += kPieces * kWarps) {
    fetch<UP>(p, s, m, first, n, i, fresh);
    put<UP>(s, m, n, i, fresh);
  }
  __syncthreads();
  if (s.far) return;                                             // run_far takes the tiles

  // The values of the lane's token, and the powers of those whose sums it gets: zeros where there is no token or unit.
  const auto values = [&](int j, int lu) {
    const int row = FEW ? j * 2 + g / 4 : j * kTokens + g, u = u0 + lu;
    const bool there = row < n && (!FEW || g % 4 == t) && (WHOLE || u < m.units);
    return s_dyn + (there ? m.x + row * m.pitch + u * (2 * kUnit) + t * (FP4 ? 64 : 32) : 0);
  };
  const auto power = [&](int j, int lu) {
    const float* f = m.power + (WHOLE ? u0 + lu : min(u0 + lu, m.units - 1)) * m.columns;
    if constexpr (FEW) return make_float2(f[j * 2 + t / 2], 0.f);
    else return *reinterpret_cast<const float2*>(f + j * kTokens + t * 2);
  };
  constexpr auto piece = [](int i) { return FP4 ? i * 16 : i / 2 * 128 + i % 2 * 16; };
  uint4 held[kHeld ? NT * PER : 1][4];
  float2 held_power[kHeld ? NT * PER : 1];
  if constexpr (kHeld) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int lu = 0; lu < PER; ++lu) {
        held_power[j * PER + lu] = power(j, lu);
#pragma unroll
        for (int i = 0; i < 4; ++i) held[j * PER + lu][i] = *reinterpret_cast<const uint4*>(values(j, lu) + piece(i));
      }
  }
  float acc[NT][V];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int v = 0; v < V; ++v) acc[j][v] = 0.f;
  const int slots = min(m.slots / n, kMaxSlots);                 // tiles whose parts are added up together: TPI at least
  int slot = 0;
  float* red = m.red;                                            // of two, in turn
  uint32_t lacks = 0u;                                           // of all units' scales to the largest of their four

  for (int tile = tile0; tile < tile1; tile += TPI) {
    uint32_t top = 0u;
#pragma unroll
    for (int i0 = 0; i0 < TPI * PER; ++i0) {
      const int d = i0 % D, lu = i0 % PER, ti = i0 / PER;
      if (lu == 0 && tile + ti >= tile1) break;
      float2 s0, s1;                                             // scales of rows g and g + 8: of a unit, or (FEW) of the lane's two blocks
      uint32_t factor[2];
      const bool there = WHOLE || u0 + lu < m.units;
      if constexpr (FP4) {
        if (lu % 2 == 0) {                                       // the lane's own word, of one of two units
          const int u = u0 + lu + (PER > 1 ? t / 2 : 0);
          const uint32_t used = WHOLE || u + 1 < m.units ? 0xffffffffu : u + 1 == m.units ? last_used : 0u;
          if (!WHOLE) scale[ti][lu / 2] &= used;
          if constexpr (!FEW) {
            top = largest_scale(scale[ti][lu / 2]);
            if (!WHOLE) scale[ti][lu / 2] &= used;
            lacks |= scale[ti][lu / 2];
          }
        }
        const int lane0 = lane / 4 * 4 + (PER > 1 ? lu % 2 * 2 : 0);
        const uint32_t w0 = __shfl_sync(kFull, scale[ti][lu / 2], lane0), w1 = __shfl_sync(kFull, scale[ti][lu / 2], lane0 + 1);
        if constexpr (FEW) {
          s0 = two_scales(w0 >> (t % 2 * 16));
          s1 = two_scales(w1 >> (t % 2 * 16));
        } else {
          factor[0] = lacking(w0, t);
          factor[1] = lacking(w1, t);
          const float2 both = two_scales(__shfl_sync(kFull, top, lane0) | __shfl_sync(kFull, top, lane0 + 1) << 8);
          s0 = make_float2(both.x, both.x);
          s1 = make_float2(both.y, both.y);
        }
      } else {
        const float a = __uint_as_float(__shfl_sync(kFull, scale[ti][0], lu * 2)), b = __uint_as_float(__shfl_sync(kFull, scale[ti][0], lu * 2 + 1));
        s0 = there ? make_float2(a, a) : make_float2(0.f, 0.f);
        s1 = there ? make_float2(b, b) : make_float2(0.f, 0.f);
      }
      float dot[NT][4];                                          // one chain of products for any NT, so that a token's sums are alike
      const uint8_t* at[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int v = 0; v < 4; ++v) dot[j][v] = 0.f;
        if constexpr (!kHeld) at[j] = values(j, lu);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {                              // 16 bytes of a token's values: 8 codes
        uint32_t a[2][4];                                        // of rows g and g + 8
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if constexpr (FP4) {
            fp4_unpack8(word(ring[d][r], i), a[r]);
            if constexpr (!FEW) {
#pragma unroll
              for (int v = 0; v < 4; ++v) a[r][v] = half2_mul(a[r][v], factor[r]);
            }
          } else {
            e4m3_half(word(ring[d][i / 2 * 2 + r], i % 2 * 2), a[r][0], a[r][1]);
            e4m3_half(word(ring[d][i / 2 * 2 + r], i % 2 * 2 + 1), a[r][2], a[r][3]);
          }
        }
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint4 b;
          if constexpr (kHeld) b = held[j * PER + lu][i];
          else b = *reinterpret_cast<const uint4*>(at[j] + piece(i));
          mma_f16(dot[j], a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
          mma_f16(dot[j], a[0][2], a[1][2], a[0][3], a[1][3], b.z, b.w);
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const float2 f = kHeld ? held_power[j * PER + lu] : power(j, lu);
        if constexpr (FEW) {
          acc[j][0] = fmaf(dot[j][0] * f.x, s0.x, fmaf(dot[j][1] * f.x, s0.y, acc[j][0]));
          acc[j][1] = fmaf(dot[j][2] * f.x, s1.x, fmaf(dot[j][3] * f.x, s1.y, acc[j][1]));
        } else {
          acc[j][0] = fmaf(dot[j][0] * f.x, s0.x, acc[j][0]);
          acc[j][1] = fmaf(dot[j][1] * f.y, s0.x, acc[j][1]);
          acc[j][2] = fmaf(dot[j][2] * f.x, s1.x, acc[j][2]);
          acc[j][3] = fmaf(dot[j][3] * f.y, s1.x, acc[j][3]);
        }
      }
      // What is loaded into this unit's place: the D-th behind it.
      const int next = (i0 + D) % PER;
      if constexpr (PER < D) {
        if (lu == PER - 1) load_scales(scale[ti]);               // the tile's own are used up; those of the one TPI behind
      } else {
        if (next == 0) load_scales(scale[1]);
      }
      load(ring[d], next);
      if (next == PER - 1) next_tile();
      if (lu < PER - 1) continue;
      // The tile's end: the warps' parts go to shared memory.
      if constexpr (PER >= D) {
#pragma unroll
        for (int i = 0; i < SW; ++i) scale[0][i] = scale[1][i];
      }
      float* part_of = red + ((slot + ti) * kWarps + warp) * n * kRows;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if constexpr (FEW) {                                     // the other two blocks are the neighbour's
          const float a = acc[j][0] + __shfl_xor_sync(kFull, acc[j][0], 1), b = acc[j][1] + __shfl_xor_sync(kFull, acc[j][1], 1);
          if (j * 2 + t / 2 < n) part_of[(j * 2 + t / 2) * kRows + t % 2 * 8 + g] = t % 2 == 0 ? a : b;
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int row = j * kTokens + t * 2 + v % 2;
            if (row < n) part_of[row * kRows + v / 2 * 8 + g] = acc[j][v];
          }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) acc[j][v] = 0.f;
      }
    }
    slot += min(TPI, tile1 - tile);
    if (slot + TPI <= slots && tile + TPI < tile1) continue;
    if (FP4 && !FEW && (lacks & 0xf0f0f0f0u) != 0u) s.apart = 1; // of 16 or more
    // Those of some tiles are there: they are added in the order of the warps.  The next ones go
    // elsewhere, and here again only behind the next barrier.
    __syncthreads();
    add_parts<UP>(p, s, red, min(tile + TPI, tile1) - slot, slot, first, n);
    slot = 0;
    red = red == m.red ? m.red + m.slots * kWarps * kRows : m.red;
  }
}

// What run_tiles leaves, or has got wrong: the same tiles and tokens, which are staged.  4 bits: one block at a time, for which the
// other lanes' codes are 0.  Where run_tiles is right these are its bits (4 bits: those for up to 4 tokens), so that a
// far token does not change the others of its expert.  Nothing is under way ahead of its use: 8 of 64 experts of 4096 and 2048,
// 16 tokens that are all far, 4 bits 546 us (174 otherwise), 8 bits 343 (229), calls outside a graph.
template <bool FP4, bool UP>
__device__ __noinline__ void run_far(const SmallLayerParams& p, const Lists& s, const Staged m, int per, int e, int tile0, int tile1, int first, int n) {
  constexpr int L = FP4 ? 1 : 2, UB = 64 * L;                    // as in run_tiles
  const int K = UP ? p.H : p.I, N = UP ? 2 * p.I : p.H, row_bytes = FP4 ? K / 2 : K, others = UP ? p.I : 8;
  const SmallWeights& w = UP ? p.w1 : p.w2;
  const uint32_t* const scales = static_cast<const uint32_t*>(w.scale);
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp, g = lane / 4, t = lane % 4;
  float* red = m.red;
  __syncthreads();                                               // run_tiles' parts are no longer read
  for (int tile = tile0; tile < tile1; ++tile) {
    const int in = tile * (UP ? 8 : kRows);                      // the tile's first row
    const int64_t row0 = int64_t(e) * N + in + g;
    float* const part_of = red + warp * n * kRows;
    for (int j0 = 0; j0 < n; j0 += kTokens) {
      float acc[2][4] = {};                                      // 4 bits: of the first two blocks and of the others
      for (int u = warp * per; u < min((warp + 1) * per, m.units); ++u) {
        const uint8_t* values = s_dyn + (j0 + g < n ? m.x + (j0 + g) * m.pitch + u * (2 * kUnit) + t * (FP4 ? 64 : 32) : 0);
        const float2 f = *reinterpret_cast<const float2*>(m.power + u * m.columns + j0 + t * 2);
        uint4 codes[2][L];                                       // of rows g and g + 8
        uint32_t scale[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll
          for (int i = 0; i < L; ++i) {
            const int c = u * UB + i * 64 + t * 16;
            codes[r][i] = c < row_bytes ? load_weights(w.q + (row0 + r * others) * row_bytes + c) : make_uint4(0u, 0u, 0u, 0u);
          }
          scale[r] = load_scale(scales + (FP4 ? int64_t(u) * p.E * N + row0 + r * others
                                              : (int64_t(e) * ((N + 127) / 128) + (in + r * others) / 128) * m.units + u));
        }
        const auto add = [&](float (&to)[4], int b) {
          if (FP4 && u * kUnit + b * 32 >= K) return;
          float dot[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t a[2][4];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if constexpr (FP4) {
                fp4_unpack8(t == b ? word(codes[r][0], i) : 0u, a[r]);
              } else {
                e4m3_half(word(codes[r][i / 2], i % 2 * 2), a[r][0], a[r][1]);
                e4m3_half(word(codes[r][i / 2], i % 2 * 2 + 1), a[r][2], a[r][3]);
              }
            }
            const uint4 v = *reinterpret_cast<const uint4*>(values + (FP4 ? i * 16 : i / 2 * 128 + i % 2 * 16));
            mma_f16(dot, a[0][0], a[1][0], a[0][1], a[1][1], v.x, v.y);
            mma_f16(dot, a[0][2], a[1][2], a[0][3], a[1][3], v.z, v.w);
          }
          const float2 two = FP4 ? two_scales((scale[0] >> b * 8 & 255u) | (scale[1] >> b * 8 & 255u) << 8)
                                 : make_float2(__uint_as_float(scale[0]), __uint_as_float(scale[1]));
          to[0] = add_scaled(dot[0], f.x, two.x, to[0]);
          to[1] = add_scaled(dot[1], f.y, two.x, to[1]);
          to[2] = add_scaled(dot[2], f.x, two.y, to[2]);
          to[3] = add_scaled(dot[3], f.y, two.y, to[3]);
        };
        if constexpr (FP4) {
          add(acc[0], 1);
          add(acc[0], 0);
          add(acc[1], 3);
          add(acc[1], 2);
        } else {
          add(acc[0], 0);
        }
      }
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (j0 + t * 2 + v % 2 < n) part_of[(j0 + t * 2 + v % 2) * kRows + v / 2 * 8 + g] = acc[0][v] + acc[1][v];
    }
    __syncthreads();
    add_parts<UP>(p, s, red, tile, 1, first, n);                 // the next tile's go elsewhere
    red = red == m.red ? m.red + m.slots * kWarps * kRows : m.red;
  }
}

template <bool FP4, bool UP, int PER, bool WHOLE>
__global__ void __launch_bounds__(kThreads, 1) layer_small_kernel(const __grid_constant__ SmallLayerParams p, int cap, int columns, int pitch, int slots) {
  __shared__ Lists s;
  Staged m;
  m.units = ((UP ? p.H : p.I) + kUnit - 1) / kUnit;
  m.pitch = pitch;
  m.columns = columns;
  m.slots = slots;
  m.power = reinterpret_cast<float*>(s_dyn + kZeros);
  m.red = m.power + m.units * columns;
  m.x = kZeros + (m.units * columns + 2 * slots * kWarps * kRows) * 4;
  if (threadIdx.x < kZeros / 4) reinterpret_cast<uint32_t*>(s_dyn)[threadIdx.x] = 0u;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if constexpr (UP) {
    const int64_t line = (int64_t(blockIdx.x) * kThreads + threadIdx.x) * 128;
    if (line < int64_t(p.T) * p.H * 2) asm volatile("prefetch.global.L2 [%0];" :: "l"(static_cast<const char*>(p.x) + line));
  }
  const int tiles = UP ? p.I / 8 : p.H / kRows;                  // of an expert
  plan<FP4>(s, p, tiles, cap);
  const int run0 = s.run0, run1 = s.run1;
  for (int at = run0; at <= run1; ++at) {
    const int tile0 = s.tile0[at], tile1 = s.tile1[at], e = s.expert[at], end = s.start[at + 1];
    if (tile0 >= tile1) continue;
    const int chunk = end - s.start[at] > cap ? kChunk : tile1 - tile0;
    for (int t0 = tile0; t0 < tile1; t0 += chunk) {
      const int t1 = min(t0 + chunk, tile1);
      for (int first = s.start[at]; first < end; first += cap) {
        const int n = min(cap, end - first);
        if (FP4 && n <= kFew / 2) run_tiles<FP4, UP, PER, WHOLE, FP4, 1>(p, s, m, e, t0, t1, first, n);
        else if (FP4 && n <= kFew) run_tiles<FP4, UP, PER, WHOLE, FP4, FP4 ? 2 : 1>(p, s, m, e, t0, t1, first, n);
        else if (n <= kTokens) run_tiles<FP4, UP, PER, WHOLE, false, 1>(p, s, m, e, t0, t1, first, n);
        else run_tiles<FP4, UP, PER, WHOLE, false, 2>(p, s, m, e, t0, t1, first, n);
        if (s.far || (FP4 && s.apart)) run_far<FP4, UP>(p, s, m, PER, e, t0, t1, first, n);
      }
    }
  }
  if constexpr (!UP) asm volatile("griddepcontrol.wait;" ::: "memory");   // where it had no tile: the third kernel ends behind the first
}

// Of dynamic shared memory: what leaves L1 room for the weights under way.
constexpr size_t kShared = 144 * 1024;

template <bool FP4, bool UP, int PER, bool WHOLE>
cudaError_t launch_per(const SmallLayerParams& p, int sms, cudaStream_t stream) {
  const int K = UP ? p.H : p.I, units = (K + kUnit - 1) / kUnit;
  const int pitch = units * kUnit * 2 + 16;                      // rows' same pieces lie in different banks
  // Tokens of an expert that are staged at once, and parts of tiles: of a round's tiles at least, of eight at most.
  // More of them, which leave L1 less, where experts have more than four on average.  (8 of 64 experts of 4096 and 2048: 64 tokens,
  // 8 bits 398 us with 8 at once, 309 with 14, 4 bits 351 and 303; 16 tokens, 8 bits 217 and 222, 4 bits 165 and 165.)
  int cap = p.T * p.k > 4 * p.E ? 2 * kTokens : kTokens, columns = 0, slots = 0;
  if (cap > p.T) cap = p.T;
  size_t smem = 0;
  for (;; --cap) {
    constexpr int kAhead = FP4 ? 4 : 2, kRound = PER < kAhead ? kAhead / PER : 1, kRound2 = PER < 2 ? 2 / PER : 1;
    columns = cap > kTokens ? 2 * kTokens : kTokens;
    const int least = cap > kTokens && kRound2 * cap > kRound * kTokens ? kRound2 * cap : kRound * (cap < kTokens ? cap : kTokens);
    slots = cap > kTokens || least > 2 * kTokens ? least : 2 * kTokens;
    if (slots > kMaxSlots * cap) slots = kMaxSlots * cap;
    smem = kZeros + size_t(units) * columns * 4 + size_t(cap) * pitch + size_t(slots) * 2 * kWarps * kRows * 4;
    if (smem <= kShared) break;
  }
  if (smem < kZeros + size_t(p.E) * kWarps) smem = kZeros + size_t(p.E) * kWarps;   // the lists' table
  const auto kernel = layer_small_kernel<FP4, UP, PER, WHOLE>;
  // The limit of shared memory is raised once on each device: the host's time is a good part of a small call's.
  static std::atomic<uint64_t> raised{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (dev > 63 || (raised.load(std::memory_order_relaxed) & bit) == 0) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kShared));
    if (e != cudaSuccess) return e;
    raised.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = UP ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, cap, columns, pitch, slots);
}

// PER by the length of the contraction, and whether it fills the warps' units: then no address or scale is checked against
// its end.  (Without that form: 8 experts of 16384 and 4096, 16 tokens, 8 bits 599 us instead of 449, 4 bits 409 and 400; 64 of
// 4096 and 2048, 64 tokens, 8 bits 318 and 311, one token, 4 bits 30.6 and 29.8.)
template <bool FP4, bool UP, int PER>
cudaError_t launch_units(const SmallLayerParams& p, int sms, cudaStream_t stream) {
  return (UP ? p.H : p.I) == PER * kWarps * kUnit ? launch_per<FP4, UP, PER, true>(p, sms, stream) : launch_per<FP4, UP, PER, false>(p, sms, stream);
}
template <bool FP4, bool UP>
cudaError_t launch(const SmallLayerParams& p, int sms, cudaStream_t stream) {
  const int units = ((UP ? p.H : p.I) + kUnit - 1) / kUnit, per = (units + kWarps - 1) / kWarps;
  if (per <= 1) return launch_units<FP4, UP, 1>(p, sms, stream);
  if (per <= 2) return launch_units<FP4, UP, 2>(p, sms, stream);
  return per <= 4 ? launch_units<FP4, UP, 4>(p, sms, stream) : launch_units<FP4, UP, 8>(p, sms, stream);
}

}  // namespace
}  // namespace moe
