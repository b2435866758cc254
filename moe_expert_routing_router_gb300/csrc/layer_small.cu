// The experts of a layer for the few tokens of a decode step:
//
//   h_a = glu(W1_e x_t),  out_t = sum_j gate_tj W2_e h_a      a = (t, j), e = idx_tj
//
// in two kernels, of which each reads the weights of the experts that have tokens once;
// that reading is what bounds them.  (The tensor core's own 4-bit and 8-bit products take
// 128 rows at a time and quantised activations; here an expert has a token or two.)
//
// Both kernels have the same body.  A tile is 16 rows of one expert's weights; the tiles of
// all experts with tokens are split evenly, in order, over one CTA per SM, and the warps of a
// CTA share the contraction of a tile.  Weights go from memory into registers, 16 bytes of a
// row a lane, some steps ahead; codes become fp16, which holds them exactly, and meet the
// tokens in mma.sync m16n8k16 with the weights' rows as M.  The order of the contraction is
// free, so a lane's 16 bytes are its share of the steps as they lie.
//   4 bits:  a lane's 16 bytes are one block of 32, with a scale of its own, and the four
//            lanes of a row hold four blocks, which one product would add up.  So a token
//            takes four of the eight columns, and each sees one block: the other lanes' part
//            of its column is zero.  Sums come out by block, and scales are multiplied there.
//   e4m3:    a scale stands for 128 of the contraction; the columns are eight tokens.
// The tokens' values are staged in shared memory as fp16 with a power of two for each 128, so
// that their largest is between 2^14 and 2^15: bf16 values are exact down to 2^-28 of it, and
// the fp32 values of h are rounded to 11 bits (three more than bf16 has).  All sums are fp32.
//
// The first kernel's tiles are 8 rows of the gate and the 8 rows of the other half that go
// with them.  The second one's sums go to memory by assignment, and the CTA that completes
// a block of 128 columns adds them up by gate, in the order of j: no result depends on an order of
// arrival.  It is launched while the first one ends (programmatic dependent launch).
#include "block_values.cuh"
#include "layer_small.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace moe {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / kWarp;
constexpr int kRows = 16;                     // of a tile
constexpr int kUnit = 128;                    // of the contraction, taken by a warp at a time
constexpr int kMaxE = 1024, kMaxA = kSmallTokens * 8;
constexpr int kJoin = 128;                    // columns that are joined together

template <bool FP4>
struct Kind {
  static constexpr int kTokens = FP4 ? 2 : 8;                    // tokens of a product's eight columns
  static constexpr int kMaxTiles = FP4 ? 8 : 4;                  // products side by side
  static constexpr int kLoads = FP4 ? 1 : 2;                     // 16-byte pieces of a row's unit a lane
  static constexpr int kAhead = FP4 ? 4 : 2;                     // units under way
};

struct Lists {
  int idx[kMaxA];                             // the assignments' experts, -1 for none
  int order[kMaxA];                           // assignments by expert
  int count[kMaxE];                           // of an expert; then the place of its next assignment
  int expert[kMaxA], start[kMaxA + 1];        // of the experts that have tokens: which, and where theirs start
  int active;
  int ready[kSmallWidth / kJoin], n_ready;    // blocks of columns that this CTA joins
};

// The experts that have tokens, and their assignments.  All threads.
__device__ void sort_assignments(Lists& s, const SmallLayerParams& p) {
  const int A = p.T * p.k;
  for (int e = threadIdx.x; e < p.E; e += kThreads) s.count[e] = 0;
  for (int a = threadIdx.x; a < A; a += kThreads) {
    const int e = p.idx[a];
    s.idx[a] = e >= 0 && e < p.E ? e : -1;
  }
  __syncthreads();
  for (int a = threadIdx.x; a < A; a += kThreads)
    if (s.idx[a] >= 0) atomicAdd(&s.count[s.idx[a]], 1);
  __syncthreads();
  if (threadIdx.x < kWarp) {
    const int lane = threadIdx.x;
    int active = 0, before = 0;
    for (int e0 = 0; e0 < p.E; e0 += kWarp) {
      const int c = e0 + lane < p.E ? s.count[e0 + lane] : 0;
      const unsigned some = __ballot_sync(kFull, c > 0);
      if (some == 0u) continue;
      int incl = c;
#pragma unroll
      for (int off = 1; off < kWarp; off <<= 1) {
        const int o = __shfl_up_sync(kFull, incl, off);
        if (lane >= off) incl += o;
      }
      if (c > 0) {
        const int at = active + __popc(some & ((1u << lane) - 1u));
        s.expert[at] = e0 + lane;
        s.start[at] = before + incl - c;
        s.count[e0 + lane] = before + incl - c;
      }
      active += __popc(some);
      before += __shfl_sync(kFull, incl, kWarp - 1);
    }
    if (lane == 0) {
      s.active = active;
      s.start[active] = before;
    }
  }
  __syncthreads();
  // The order within an expert is that of arrival: it decides a column, and no column's sum.
  for (int a = threadIdx.x; a < A; a += kThreads)
    if (s.idx[a] >= 0) s.order[atomicAdd(&s.count[s.idx[a]], 1)] = a;
  __syncthreads();
}

// Where a CTA's shared memory lies behind the lists.
struct Staged {
  int x;                                      // offset of [cap] rows of `pitch` bytes: fp16
  float* power;                               // [units][columns]: what a token's 128 values were divided by
  float* red;                                 // [warps][cap][16]: the warps' parts of a tile
  int pitch, columns, units;
};
extern __shared__ __align__(16) uint8_t s_dyn[];                 // begins with 16 bytes of zeros

__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Rows `order[first ..]` of the tokens (UP: bf16 x) or of the assignments (h), as fp16.  A warp
// takes a unit of a row; the rest of the last unit is zero.
template <bool UP>
__device__ __forceinline__ void stage(const SmallLayerParams& p, const Lists& s, const Staged& m, int first, int n) {
  const int K = UP ? p.H : p.I, warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  for (int i = warp; i < n * m.units; i += kWarps) {
    const int row = i / m.units, u = i - row * m.units, a = s.order[first + row], c = u * kUnit + lane * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (c < K) {                                                 // K is a multiple of 16
      if constexpr (UP) {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.x) + int64_t(a / p.k) * K + c);
        v = make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u));
      } else {
        v = __ldcg(reinterpret_cast<const float4*>(p.h + int64_t(a) * K + c));
      }
    }
    uint32_t top = max(max(__float_as_uint(v.x) & 0x7fffffffu, __float_as_uint(v.y) & 0x7fffffffu),
                       max(__float_as_uint(v.z) & 0x7fffffffu, __float_as_uint(v.w) & 0x7fffffffu));
    top = __reduce_max_sync(kFull, top);
    // 2^14 over the power of two at or below the largest, as far as both it and its inverse are normal
    const uint32_t up = min(268u - (top >> 23), 253u);
    const float f = __uint_as_float(up << 23);
    *reinterpret_cast<uint2*>(s_dyn + m.x + row * m.pitch + (u * kUnit + lane * 4) * 2) = make_uint2(pack_half2(v.x * f, v.y * f), pack_half2(v.z * f, v.w * f));
    if (lane == 0) m.power[u * m.columns + row] = __uint_as_float((254u - up) << 23);
  }
}

__device__ __forceinline__ uint4 load_weights(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
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
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

__device__ __forceinline__ float silu(float g) {
  const float t = __expf(-fabsf(g)), r = 1.f / (1.f + t);
  return g * (g >= 0.f ? r : t * r);
}

// Tiles [tile0, tile1) of expert e for the `n` staged tokens, whose assignments are
// order[first ..].  NT products side by side hold them.
template <bool FP4, bool UP, int NT>
__device__ __forceinline__ void run_tiles(const SmallLayerParams& p, const Lists& s, const Staged& m, int e, int tile0, int tile1, int first, int n) {
  using KD = Kind<FP4>;
  constexpr int D = KD::kAhead, L = KD::kLoads;
  const int K = UP ? p.H : p.I, N = UP ? 2 * p.I : p.H;
  const SmallWeights& w = UP ? p.w1 : p.w2;
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp, g = lane / 4, t = lane % 4;
  const int per = (m.units + kWarps - 1) / kWarps;               // units of a warp: warp, warp + 16, ...
  const int row_bytes = FP4 ? K / 2 : K, row_tiles = tile1 - tile0;
  const int rows_up = UP ? p.I : 8;                              // from a tile's first 8 rows to its others
  const int64_t base = int64_t(e) * N;
  const int nblocks = (N + 127) / 128, kblocks = (K + 127) / 128;
  const uint32_t last_used = K % kUnit == 0 ? 0xffffffffu : (1u << K % kUnit / 4) - 1u;   // scales of the last unit: others may be anything

  uint4 ring[D][2 * L];
  uint32_t scale[D][2];
  // The next unit to load.
  int lt = tile0, lu = 0;
  const auto load = [&](uint4 (&to)[2 * L], uint32_t (&sc)[2]) {
    const int u = warp + lu * kWarps;
#pragma unroll
    for (int i = 0; i < 2 * L; ++i) to[i] = make_uint4(0u, 0u, 0u, 0u);
    sc[0] = sc[1] = 0u;
    if (lt < tile1 && u < m.units) {
      const int row = UP ? lt * 8 : lt * kRows;
      const int64_t r = base + row + g;
#pragma unroll
      for (int i = 0; i < L; ++i) {
        const int c = FP4 ? u * 64 + t * 16 : u * 128 + i * 64 + t * 16;
        if (c < row_bytes) {
          const uint8_t* q = w.q + r * row_bytes + c;
          to[2 * i] = load_weights(q);
          to[2 * i + 1] = load_weights(q + int64_t(rows_up) * row_bytes);
        }
      }
      if constexpr (FP4) {
        const uint32_t* q = static_cast<const uint32_t*>(w.scale) + int64_t(u) * p.E * N + r;
        sc[0] = __ldg(q);
        sc[1] = __ldg(q + rows_up);
      } else {
        const float* q = static_cast<const float*>(w.scale) + int64_t(e) * nblocks * kblocks + u;
        sc[0] = __float_as_uint(__ldg(q + int64_t(row / 128) * kblocks));
        sc[1] = __float_as_uint(__ldg(q + int64_t((row + rows_up) / 128) * kblocks));
      }
    }
    if (++lu == per) {
      lu = 0;
      ++lt;
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load(ring[d], scale[d]);

  // A lane's token in each product's column, and where its values lie.
  constexpr int V = FP4 ? 2 : 4;                                 // sums of a lane in a product
  float acc[NT][V];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int v = 0; v < V; ++v) acc[j][v] = 0.f;
  const int column = FP4 ? g / 4 : g;
  const bool mine = !FP4 || g % 4 == t;

  int ct = tile0, cu = 0;                                        // the unit at work
  const int steps = row_tiles * per;
  for (int i0 = 0; i0 < steps; i0 += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (i0 + d >= steps) break;
      const int u = warp + cu * kWarps;
      if (u < m.units) {
        float dot[NT][4];
        int at[NT], step[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
          for (int v = 0; v < 4; ++v) dot[j][v] = 0.f;
          const int row = j * KD::kTokens + column;
          const bool there = mine && row < n;
          at[j] = there ? m.x + row * m.pitch + u * (2 * kUnit) + t * (FP4 ? 64 : 32) : 0;
          step[j] = there ? -1 : 0;
        }
#pragma unroll
        for (int i = 0; i < L; ++i)
#pragma unroll
          for (int k = 0; k < 4; k += FP4 ? 1 : 2) {             // 16 bytes of a token's values: 8 codes
            uint32_t a[2][4];                                    // of rows g and g + 8
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if constexpr (FP4) {
                fp4_unpack8(word(ring[d][r], k), a[r]);
              } else {
                e4m3_half(word(ring[d][2 * i + r], k), a[r][0], a[r][1]);
                e4m3_half(word(ring[d][2 * i + r], k + 1), a[r][2], a[r][3]);
              }
            }
            const int off = FP4 ? k * 16 : i * 128 + k * 8;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              const uint4 b = *reinterpret_cast<const uint4*>(s_dyn + at[j] + (off & step[j]));
              mma_f16(dot[j], a[0][0], a[1][0], a[0][1], a[1][1], b.x, b.y);
              mma_f16(dot[j], a[0][2], a[1][2], a[0][3], a[1][3], b.z, b.w);
            }
          }
        if constexpr (FP4) {
          const uint32_t used = u + 1 == m.units ? last_used : 0xffffffffu;
          const float2 s0 = two_scales((scale[d][0] & used) >> (t % 2 * 16)), s1 = two_scales((scale[d][1] & used) >> (t % 2 * 16));
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const float f = m.power[u * m.columns + j * 2 + t / 2];
            acc[j][0] = fmaf(dot[j][0] * f, s0.x, fmaf(dot[j][1] * f, s0.y, acc[j][0]));
            acc[j][1] = fmaf(dot[j][2] * f, s1.x, fmaf(dot[j][3] * f, s1.y, acc[j][1]));
          }
        } else {
          const float s0 = __uint_as_float(scale[d][0]), s1 = __uint_as_float(scale[d][1]);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            const float2 f = *reinterpret_cast<const float2*>(&m.power[u * m.columns + j * 8 + t * 2]);
            acc[j][0] = fmaf(dot[j][0] * f.x, s0, acc[j][0]);
            acc[j][1] = fmaf(dot[j][1] * f.y, s0, acc[j][1]);
            acc[j][2] = fmaf(dot[j][2] * f.x, s1, acc[j][2]);
            acc[j][3] = fmaf(dot[j][3] * f.y, s1, acc[j][3]);
          }
        }
      }
      load(ring[d], scale[d]);
      if (++cu < per) continue;
      // The tile's end: the warps' parts meet in shared memory, and are added in their order.
      __syncthreads();                                           // the parts of the tile before have been read
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        if constexpr (FP4) {
          float a = acc[j][0], b = acc[j][1];
          a += __shfl_xor_sync(kFull, a, 1);
          b += __shfl_xor_sync(kFull, b, 1);
          const int row = j * 2 + t / 2;
          if (row < n) m.red[(warp * n + row) * kRows + (t % 2) * 8 + g] = t % 2 == 0 ? a : b;
        } else {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            const int row = j * 8 + t * 2 + v % 2;
            if (row < n) m.red[(warp * n + row) * kRows + v / 2 * 8 + g] = acc[j][v];
          }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) acc[j][v] = 0.f;
      }
      __syncthreads();
      for (int o0 = warp * kWarp; o0 < n * kRows; o0 += kThreads) {   // whole warps: 2 tokens each
        const int o = o0 + lane, live = o < n * kRows;
        float sum = 0.f;
        if (live) {
#pragma unroll
          for (int i = 0; i < kWarps; ++i) sum += m.red[i * n * kRows + o];
        }
        const int row = o % kRows;
        if constexpr (UP) {
          const float other = __shfl_down_sync(kFull, sum, 8);
          if (live && row < 8) p.h[int64_t(s.order[first + o / kRows]) * p.I + ct * 8 + row] = silu(sum) * other;
        } else {
          if (live) p.y[int64_t(s.order[first + o / kRows]) * p.H + ct * kRows + row] = sum;
        }
      }
      cu = 0;
      ++ct;
    }
  }
}

template <bool FP4, bool UP>
__global__ void __launch_bounds__(kThreads, 1) layer_small_kernel(const __grid_constant__ SmallLayerParams p, int cap, int columns, int pitch) {
  using KD = Kind<FP4>;
  __shared__ Lists s;
  Staged m;
  m.units = ((UP ? p.H : p.I) + kUnit - 1) / kUnit;
  m.pitch = pitch;
  m.columns = columns;
  m.power = reinterpret_cast<float*>(s_dyn + 16);
  m.red = m.power + m.units * columns;
  m.x = 16 + (m.units * columns + kWarps * cap * kRows) * 4;
  if (threadIdx.x < 4) reinterpret_cast<uint32_t*>(s_dyn)[threadIdx.x] = 0u;
  if constexpr (UP) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  sort_assignments(s, p);
  if constexpr (UP) {
    for (int i = blockIdx.x * kThreads + threadIdx.x; i < (p.H + kJoin - 1) / kJoin; i += gridDim.x * kThreads) p.joined[i] = 0;
  } else {
    asm volatile("griddepcontrol.wait;" ::: "memory");           // h, and joined, are there
  }

  const int tiles = UP ? p.I / 8 : p.H / kRows;                  // of an expert
  const int64_t all = int64_t(s.active) * tiles;
  const int64_t from = all * blockIdx.x / gridDim.x, to = all * (blockIdx.x + 1) / gridDim.x;
  for (int64_t i = from; i < to;) {
    const int at = int(i / tiles), tile0 = int(i - int64_t(at) * tiles), tile1 = int(min(int64_t(tiles), tile0 + to - i));
    for (int first = s.start[at]; first < s.start[at + 1]; first += cap) {
      const int n = min(cap, s.start[at + 1] - first);
      __syncthreads();                                           // the tokens before are no longer read
      stage<UP>(p, s, m, first, n);
      __syncthreads();
      const int e = s.expert[at];
      if (n <= KD::kTokens) run_tiles<FP4, UP, 1>(p, s, m, e, tile0, tile1, first, n);
      else if (n <= 2 * KD::kTokens) run_tiles<FP4, UP, 2>(p, s, m, e, tile0, tile1, first, n);
      else if (n <= 4 * KD::kTokens) run_tiles<FP4, UP, 4>(p, s, m, e, tile0, tile1, first, n);
      else if constexpr (KD::kMaxTiles == 8) run_tiles<FP4, UP, 8>(p, s, m, e, tile0, tile1, first, n);
    }
    i += tile1 - tile0;
  }
  if constexpr (UP) return;

  // Blocks of columns whose last sums are this CTA's are joined by it.
  const int blocks = (p.H + kJoin - 1) / kJoin, in_block = kJoin / kRows;
  if (threadIdx.x == 0) s.n_ready = 0;
  __threadfence();                                               // this thread's sums, before the count
  __syncthreads();
  for (int b = threadIdx.x; b < blocks; b += kThreads) {
    const int b0 = b * in_block, b1 = min(tiles, b0 + in_block);
    int done = 0;
    for (int64_t i = from; i < to;) {
      const int at = int(i / tiles), tile0 = int(i - int64_t(at) * tiles), tile1 = int(min(int64_t(tiles), tile0 + to - i));
      done += max(0, min(tile1, b1) - max(tile0, b0));
      i += tile1 - tile0;
    }
    const int want = s.active * (b1 - b0);
    const bool mine = want == 0 ? blockIdx.x == 0 : done > 0 && atomicAdd(&p.joined[b], done) + done == want;
    if (mine) s.ready[atomicAdd(&s.n_ready, 1)] = b;
  }
  __threadfence();
  __syncthreads();
  const int n_ready = s.n_ready;
  constexpr int kPieces = kJoin / 4;
  for (int i = threadIdx.x; i < n_ready * p.T * kPieces; i += kThreads) {
    const int c = s.ready[i / (p.T * kPieces)] * kJoin + i % kPieces * 4, t = i / kPieces % p.T;
    if (c >= p.H) continue;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j >= p.k || s.idx[t * p.k + j] < 0) continue;
      const float g = p.gate[t * p.k + j];
      const float4 v = __ldcg(reinterpret_cast<const float4*>(p.y + int64_t(t * p.k + j) * p.H + c));
      sum.x = fmaf(g, v.x, sum.x);
      sum.y = fmaf(g, v.y, sum.y);
      sum.z = fmaf(g, v.z, sum.z);
      sum.w = fmaf(g, v.w, sum.w);
    }
    const __nv_bfloat162 lo = __floats2bfloat162_rn(sum.x, sum.y), hi = __floats2bfloat162_rn(sum.z, sum.w);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + int64_t(t) * p.H + c) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

constexpr size_t kShared = 232448 - sizeof(Lists) - 1024;

template <bool FP4, bool UP>
cudaError_t launch(const SmallLayerParams& p, int sms, cudaStream_t stream) {
  using KD = Kind<FP4>;
  const int K = UP ? p.H : p.I, units = (K + kUnit - 1) / kUnit;
  const int pitch = units * kUnit * 2 + 16;                      // rows' same pieces lie in different banks
  // Tokens of an expert that are staged at once.
  int cap = p.T < KD::kTokens * KD::kMaxTiles ? p.T : KD::kTokens * KD::kMaxTiles, columns = 0;
  size_t smem = 0;
  for (;; --cap) {
    columns = KD::kTokens < 4 ? 4 : KD::kTokens;                 // whole pieces of 16 bytes in front of x
    while (columns < cap) columns *= 2;
    smem = 16 + size_t(units) * columns * 4 + size_t(kWarps) * cap * kRows * 4 + size_t(cap) * pitch;
    if (smem <= kShared) break;
  }
  const auto kernel = layer_small_kernel<FP4, UP>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kShared));
  if (e != cudaSuccess) return e;
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
  return cudaLaunchKernelEx(&cfg, kernel, p, cap, columns, pitch);
}

size_t up_to(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace

size_t small_layer_work_size(int T, int H, int I, int k) {
  const size_t A = size_t(T) * k;
  return up_to(A * I * 4) + up_to(A * H * 4) + up_to(size_t(H + kJoin - 1) / kJoin * 4);
}

void small_layer_work(SmallLayerParams& p, void* work) {
  const size_t A = size_t(p.T) * p.k;
  char* at = static_cast<char*>(work);
  p.h = reinterpret_cast<float*>(at);
  p.y = reinterpret_cast<float*>(at + up_to(A * p.I * 4));
  p.joined = reinterpret_cast<int*>(at + up_to(A * p.I * 4) + up_to(A * p.H * 4));
}

cudaError_t launch_layer_small(const SmallLayerParams& p, int sms, cudaStream_t stream) {
  const cudaError_t e = p.w1.fp4 ? launch<true, true>(p, sms, stream) : launch<false, true>(p, sms, stream);
  if (e != cudaSuccess) return e;
  return p.w2.fp4 ? launch<true, false>(p, sms, stream) : launch<false, false>(p, sms, stream);
}

}  // namespace moe
