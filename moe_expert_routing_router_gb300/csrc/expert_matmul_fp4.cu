// The experts' 4-bit matrix products on the fifth-generation tensor cores.
//
// Operands are e2m1 codes, two in a byte, with one power-of-two scale for 32 values along
// the contraction.  tcgen05.mma of kind mxf4 takes both operands' codes from shared
// memory and their scales from tensor memory, and multiplies a block's products by its two
// scales itself: a tile's sum stays in tensor memory over the whole contraction, in fp32,
// and is read once.
//
// One persistent CTA per SM, 12 warps: a TMA producer and an MMA issuer (one thread each),
// two warps that bring the scales, and 8 epilogue warps of 32 rows by half of the tile's
// columns.  A stage of the ring in shared memory holds 256 values of the contraction of
// both operands (rows of 128 bytes, 128-byte swizzled) and their scales.  Those lie in
// memory as words of four, of 128 values each, one row behind another; the tensor core
// wants the words of rows r, r + 32, r + 64 and r + 96 beside one another in lane r of tensor
// memory, for each of its four quarters.  So a scale warp puts a row's four words into one
// 16-byte piece of shared memory, and the issuer copies 32 such pieces to all quarters with
// one tcgen05.cp in front of the products that read them.  A stage's scales have columns
// of their own in tensor memory, so that their reuse is ordered by the stage's.
//
// Every wait is bounded: when one runs out, the CTA records the pipeline's error
// bit, drains its copies and returns.
#include "expert_matmul_fp4.h"
#include "tensor_core.cuh"

#include <cuda_bf16.h>

namespace moe {
namespace {

constexpr int kBM = 128;                      // rows of a tile
constexpr int kBK = 256;                      // values of the contraction in a stage: 128 bytes of codes, two words of scales
constexpr int kMmaK = 64;                     // of them, taken by one instruction
constexpr int kBox = 32;                      // rows of one copy of a ragged tile, which copies only those it needs
constexpr int kScaleWarps = 2, kEpiWarps = 8, kFirstEpi = 4;
constexpr int kThreads = (kFirstEpi + kEpiWarps) * kWarp;
constexpr int kMaxE = 1024;
constexpr int kGroupM = 16;                   // row tiles of an expert that are taken before the next column tile
constexpr int kAtomBytes = 512;               // scales of 128 rows by 128 values

// ---- instructions -------------------------------------------------------------------
// d [128, N] (+)= the products of 64 values, each 32 times its scales of a and of b.
__device__ __forceinline__ void tc_mma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t scale_a, uint32_t scale_b, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}"
      :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(scale_a), "r"(scale_b), "r"(accumulate) : "memory");
}

// 32 pieces of 16 bytes to four columns of tensor memory, in each of its quarters.
__device__ __forceinline__ void tc_copy_scales(uint32_t to, uint64_t desc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" :: "r"(to), "l"(desc) : "memory");
}

// Shared-memory descriptor of such pieces, one behind another: groups of 8 lie 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(const void* p) {
  return uint64_t((smem_addr(p) >> 4) & 0x3fffu) | uint64_t(128 >> 4) << 32 | uint64_t(1) << 46;
}

__device__ __forceinline__ void copy_word(uint32_t to, const uint32_t* from, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" :: "r"(to), "l"(from), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

// 32 columns of the warp's 32 rows, asynchronously.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31"
      "}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr) : "memory");
}
// Waits for the thread's loads; the values pass through, so that no use of them moves before it.
__device__ __forceinline__ void tmem_ld32_wait(uint32_t* r) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
        "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
        "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
        "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
      :: "memory");
}

// ---- the kernel ----------------------------------------------------------------------
template <int BN>
struct Tile {
  static constexpr int kCodeBytes = (kBM + BN) * kRowBytes;
  static constexpr int kScaleBytes = (kBM + BN) / 128 * 2 * kAtomBytes;
  static constexpr int kStageBytes = kCodeBytes + kScaleBytes;
  // codes need 1024-byte alignment, so all stages' codes lie before all stages' scales
  static constexpr int kStages = BN == 256 ? 4 : 6;
  static constexpr int kBufs = BN == 256 ? 1 : 2;                // tiles' sums in tensor memory
  static constexpr int kScaleCols = (kBM + BN) / 32 * 2;         // of a stage: four columns an atom
  static constexpr int kFirstScale = kBufs * BN;
  static constexpr int kCols = BN / 2;                           // columns of one epilogue warp
  static_assert(kFirstScale + kStages * kScaleCols <= kTmemCols, "tensor memory");
};

struct Shared {
  uint64_t full[8], done[8];                  // a stage's operands are there; its products have been formed
  uint64_t ready[2], tempty[2], drain;        // a tile's sum is there; it has been read
  uint32_t tmem;
  int abort;
  int row[kMaxE], count[kMaxE], first[kMaxE + 1];   // an expert's first row and rows; tiles before it
};

__device__ __forceinline__ bool wait(Shared& sh, const MatmulFp4Params& p, uint64_t* bar, uint32_t parity,
                                     uint64_t* bar2 = nullptr, uint32_t parity2 = 0) {
  return pipeline_wait(&sh.abort, p.errors, p.timeout_ns, bar, parity, bar2, parity2);
}

__device__ __forceinline__ int boxes(int rows) { return (rows + kBox - 1) / kBox; }

// A tile of the persistent loop, walked in ascending order by every role.
struct Walk {
  int e = 0;
  int row0 = 0, rows = 0;                     // of a: the first one and how many are the tile's
  int col0 = 0, cols = 0;                     // of out within the expert

  template <int BN>
  __device__ __forceinline__ void at(const MatmulFp4Params& p, const Shared& sh, int tile) {
    const int ct = (p.C + BN - 1) / BN;
    for (;;) {                                                   // the expert that has the tile: 32 at a time, by the whole warp
      const int next = e + 1 + int(threadIdx.x % kWarp);
      const unsigned past = __ballot_sync(kFull, next <= p.E && sh.first[next] <= tile);
      e += __popc(past);
      if (past != kFull) break;
    }
    const int i = tile - sh.first[e], rt = (sh.first[e + 1] - sh.first[e]) / ct;
    // kGroupM row tiles by all column tiles at a time, rows fastest: the CTAs at
    // work share both operands' tiles in L2.
    const int group = i / (kGroupM * ct), in = i - group * kGroupM * ct;
    const int gm = min(kGroupM, rt - group * kGroupM);
    const int r0 = (group * kGroupM + in % gm) * kBM;
    col0 = in / gm * BN;
    cols = min(BN, p.C - col0);
    row0 = sh.row[e] + r0;
    rows = min(kBM, sh.count[e] - r0);
  }
};

template <int BN, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
expert_matmul_fp4_kernel(const __grid_constant__ MatmulFp4Params p, const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                         const __grid_constant__ CUtensorMap whole_a, const __grid_constant__ CUtensorMap whole_b) {
  using TL = Tile<BN>;
  extern __shared__ uint8_t s_dyn[];
  __shared__ Shared sh;
  uint8_t* ring = s_dyn + (1024 - smem_addr(s_dyn) % 1024) % 1024;
  uint8_t* scales = ring + TL::kStages * TL::kCodeBytes;
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const int stages = (p.K + kBK - 1) / kBK;                      // of a tile

  if (warp == 0) {
    if (lane == 0) {
      for (const CUtensorMap* m : {&map_a, &map_b, &whole_a, &whole_b})
        asm volatile("prefetch.tensormap [%0];" :: "l"(m) : "memory");
      for (int i = 0; i < TL::kStages; ++i) {
        mbar_init(&sh.full[i], 1 + kScaleWarps + p.extra);
        mbar_init(&sh.done[i], 1);
      }
      for (int i = 0; i < TL::kBufs; ++i) {
        mbar_init(&sh.ready[i], 1);
        mbar_init(&sh.tempty[i], kEpiWarps);
      }
      mbar_init(&sh.drain, 1);
      mbar_fence_init();
      sh.abort = *static_cast<volatile int*>(p.errors) != 0;     // an error that the host has not read yet: write nothing
    }
  } else if (warp == 1) {
    tmem_alloc(&sh.tmem);
    tc_fence_before();
  } else if (warp == 2) {                                        // tiles before each expert
    const int ct = (p.C + BN - 1) / BN;
    int tiles = 0;
    float sum = 0.f;                                             // of the tiles, where ranges that overlap pass an int
    for (int e0 = 0; e0 < p.E; e0 += kWarp) {
      int t = 0;
      if (e0 + lane < p.E) {
        int64_t start, n;
        expert_rows(p, e0 + lane, &start, &n);
        sh.row[e0 + lane] = int(start);
        sh.count[e0 + lane] = int(n);
        t = int((n + kBM - 1) / kBM) * ct;
        sum += float(t);
      }
      int ti = t;
#pragma unroll
      for (int off = 1; off < kWarp; off <<= 1) {
        const int to = __shfl_up_sync(kFull, ti, off);
        if (lane >= off) ti += to;
      }
      if (e0 + lane < p.E) sh.first[e0 + lane] = tiles + ti - t;
      tiles += __shfl_sync(kFull, ti, kWarp - 1);
    }
    if (warp_sum_f(sum) > 2e9f) tiles = 0;                       // such offsets give nothing
    if (lane == 0) sh.first[p.E] = tiles;
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int n_tiles = sh.abort == 0 ? sh.first[p.E] : 0;
  __syncthreads();                                               // every thread has seen abort before a role sets it

  // The single-thread roles run as whole warps, of which one elected thread issues.
  if (warp == 0) {
    // ---- producer: the codes ----
    int s = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    Walk w;
    for (int tile = blockIdx.x; tile < n_tiles && ok; tile += gridDim.x) {
      w.at<BN>(p, sh, tile);
      const int na = boxes(w.rows), nb = boxes(w.cols), b_row = w.e * p.C + w.col0;
      for (int b = 0; b < stages; ++b) {
        ok = __all_sync(kFull, wait(sh, p, &sh.done[s], phase ^ 1u));
        if (!ok) break;
        if (elect_one()) {
          uint64_t* bar = &sh.full[s];
          uint8_t *sa = ring + s * TL::kCodeBytes, *sb = sa + kBM * kRowBytes;
          const int x = b * kRowBytes;
          mbar_arrive_expect_tx(bar, uint32_t((na + nb) * kBox * kRowBytes));
          if (na == kBM / kBox) tma_2d(sa, &whole_a, x, w.row0, bar);
          else for (int i = 0; i < na; ++i) tma_2d(sa + i * kBox * kRowBytes, &map_a, x, w.row0 + i * kBox, bar);
          if (nb == BN / kBox) tma_2d(sb, &whole_b, x, b_row, bar);
          else for (int i = 0; i < nb; ++i) tma_2d(sb + i * kBox * kRowBytes, &map_b, x, b_row + i * kBox, bar);
        }
        __syncwarp();
        ++issued;
        if (++s == TL::kStages) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok) {                                                   // copies in flight land before shared memory goes
      for (int i = 0; i < TL::kStages && i < issued; ++i) {
        const int back = issued - 1 - i;
        mbar_wait(&sh.full[back % TL::kStages], uint32_t(back / TL::kStages) & 1u, p.timeout_ns);
      }
    }
  } else if (warp == 1) {
    // ---- MMA issuer ----
    // D fp32; A and B e2m1, both K-major; scales are exponents (bit 23); N = BN, M = 128
    constexpr uint32_t idesc = 1u << 7 | 1u << 10 | uint32_t(BN / 8) << 17 | 1u << 23 | uint32_t(kBM / 16) << 24;
    const uint64_t desc0 = smem_desc(ring), sdesc0 = scale_desc(scales);
    int s = 0, t = 0;
    uint32_t phase = 0, tphase = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < n_tiles && ok; tile += gridDim.x) {
      for (int b = 0; b < stages; ++b) {
        ok = __all_sync(kFull, wait(sh, p, &sh.full[s], phase, b == 0 ? &sh.tempty[t] : nullptr, tphase ^ 1u));
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t da = desc0 + uint64_t(s * TL::kCodeBytes >> 4), db = da + (kBM * kRowBytes >> 4);
          const uint64_t ds = sdesc0 + uint64_t(s * TL::kScaleBytes >> 4);
          const uint32_t sc = tmem + TL::kFirstScale + s * TL::kScaleCols;
#pragma unroll
          for (int i = 0; i < TL::kScaleBytes / kAtomBytes; ++i) tc_copy_scales(sc + 4 * i, ds + i * (kAtomBytes >> 4));
          const int steps = min(kBK / kMmaK, (p.K - b * kBK + kMmaK - 1) / kMmaK);
#pragma unroll
          for (int k = 0; k < kBK / kMmaK; ++k) {                // 32 bytes along the row: 2 units of 16; half a word of scales
            if (k >= steps) break;
            const uint32_t half = uint32_t(k % 2) * 2;
            const uint32_t at = sc + k / 2 * ((kBM + BN) / 32);
            tc_mma_fp4(tmem + t * BN, da + k * 2, db + k * 2, idesc | half << 4 | half << 29, at, at + kBM / 32, b > 0 || k > 0);
          }
          tc_commit(&sh.done[s]);                                // the stage is free
          if (b + 1 == stages) tc_commit(&sh.ready[t]);
        }
        __syncwarp();
        if (++s == TL::kStages) {
          s = 0;
          phase ^= 1u;
        }
      }
      if (++t == TL::kBufs) {
        t = 0;
        tphase ^= 1u;
      }
    }
    if (!ok) {                                                   // products in flight end before tensor memory goes
      if (elect_one()) tc_commit(&sh.drain);
      __syncwarp();
      mbar_wait(&sh.drain, 0, p.timeout_ns);
    }
  } else if (warp < kFirstEpi) {
    // ---- scales: this warp's words are those of the stage's first or second 128 values ----
    const int half = warp - 2, words = (p.K + 127) / 128;
    int s = 0, last = -1;                                        // last: the stage whose copies are under way
    uint32_t phase = 0;
    bool ok = true;
    Walk w;
    const auto arrive = [&]() {                                  // of stage `last`
      async_proxy_fence();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.full[last]);
    };
    for (int tile = blockIdx.x; tile < n_tiles && ok; tile += gridDim.x) {
      w.at<BN>(p, sh, tile);
      const int64_t rows_b = int64_t(p.E) * p.C, a0 = w.row0, b0 = int64_t(w.e) * p.C + w.col0;
      for (int b = 0; b < stages; ++b) {
        ok = __all_sync(kFull, wait(sh, p, &sh.done[s], phase ^ 1u));
        if (!ok) break;
        uint8_t* to = scales + s * TL::kScaleBytes + half * (TL::kScaleBytes / 2) + lane * 16;
        const int kw = 2 * b + half;
        const int blocks = (p.K - kw * 128) / 32;                // of this word, where it is the last
#pragma unroll
        for (int atom = 0; atom < (kBM + BN) / 128; ++atom)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int64_t row = (atom == 0 ? a0 : b0 + (atom - 1) * 128) + i * 32 + lane, n = atom == 0 ? p.M : rows_b;
            const uint32_t* from = (atom == 0 ? p.a_scale : p.b_scale) + (kw < words && row < n ? int64_t(kw) * n + row : 0);
            const bool there = kw < words && row < n;
            if (blocks >= 4 || blocks <= 0) {
              copy_word(smem_addr(to + atom * kAtomBytes + i * 4), from, there);
            } else {                                             // bytes behind the last value's may be anything
              *reinterpret_cast<uint32_t*>(to + atom * kAtomBytes + i * 4) = there ? *from & ((1u << 8 * blocks) - 1u) : 0u;
            }
          }
        copy_commit();
        if (last >= 0) {                                         // the stage before: its words have had this one's wait to land
          copy_wait<1>();
          arrive();
        }
        last = s;
        if (++s == TL::kStages) {
          s = 0;
          phase ^= 1u;
        }
      }
    }
    copy_wait<0>();
    if (ok && last >= 0) arrive();
  } else {
    // ---- epilogue: rows 32 * quad + lane, kCols columns ----
    const int quad = warp % 4, part = (warp - kFirstEpi) / 4;
    int t = 0;
    uint32_t tphase = 0;
    Walk w;
    for (int tile = blockIdx.x; tile < n_tiles; tile += gridDim.x) {
      w.at<BN>(p, sh, tile);
      if (!__all_sync(kFull, wait(sh, p, &sh.ready[t], tphase))) break;
      tc_fence_after();
      const auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.tempty[t]);
      };
      const int c0 = w.col0 + part * TL::kCols;
      if (quad * 32 < w.rows && c0 < p.C) {
        const uint32_t addr = tmem + t * BN + part * TL::kCols + (uint32_t(quad * 32) << 16);
        // Pieces of 16 bytes, NP of which are turned among NP lanes at a time.
        constexpr int kPer = BF16 ? 8 : 4, NP = 8, kStep = kPer * NP;
#pragma unroll
        for (int c = 0; c < TL::kCols; c += kStep) {
          uint32_t u[kStep];
#pragma unroll
          for (int i = 0; i < kStep; i += 32) tmem_ld32(addr + c + i, u + i);
#pragma unroll
          for (int i = 0; i < kStep; i += 32) tmem_ld32_wait(u + i);
          if (c + kStep == TL::kCols) release();
          uint4 v[NP];
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const uint32_t* a = u + i * kPer;
            if constexpr (BF16) {
              uint32_t b2[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 q = __floats2bfloat162_rn(__uint_as_float(a[2 * j]), __uint_as_float(a[2 * j + 1]));
                b2[j] = *reinterpret_cast<const uint32_t*>(&q);
              }
              v[i] = make_uint4(b2[0], b2[1], b2[2], b2[3]);
            } else {
              v[i] = make_uint4(a[0], a[1], a[2], a[3]);
            }
          }
          turn<NP>(v, lane);
          const int col = c0 + c + lane % NP * kPer;               // C is a multiple of 16: a piece is whole
#pragma unroll
          for (int r = 0; r < NP; ++r) {
            const int to = quad * 32 + lane / NP * NP + r;
            if (to < w.rows && col < p.C)
              *reinterpret_cast<uint4*>(static_cast<char*>(p.out) + (int64_t(w.row0 + to) * p.C + col) * (BF16 ? 2 : 4)) = v[r];
          }
        }
      } else {
        release();
      }
      if (++t == TL::kBufs) {
        t = 0;
        tphase ^= 1u;
      }
    }
  }
  __syncwarp();                                                  // the roles' single threads are back
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_free(tmem);
}

template <int BN, bool BF16>
cudaError_t launch(const MatmulFp4Params& p, int sms, const char** error, cudaStream_t stream) {
  using TL = Tile<BN>;
  CUtensorMap ma, mb, wa, wb;
  const uint64_t cols = uint64_t(p.K) / 2, rows_b = uint64_t(p.E) * p.C;
  if (!make_map(&ma, p.a, uint64_t(p.M), cols, kBox) || !make_map(&mb, p.b, rows_b, cols, kBox) ||
      !make_map(&wa, p.a, uint64_t(p.M), cols, kBM) || !make_map(&wb, p.b, rows_b, cols, BN)) {
    *error = "cuTensorMapEncodeTiled refused an operand";
    return cudaErrorUnknown;
  }
  constexpr size_t smem = size_t(TL::kStages) * TL::kStageBytes + 1024;
  static_assert(TL::kStages <= 8 && sizeof(Shared) + smem <= 232448, "shared memory of one CTA");
  const auto kernel = expert_matmul_fp4_kernel<BN, BF16>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  // At most this many tiles: every expert's last row tile may be ragged.
  const int64_t ct = (p.C + BN - 1) / BN;
  int64_t rt = p.M / kBM + p.E;
  if (rt > p.M) rt = p.M;
  kernel<<<unsigned(rt * ct < sms ? rt * ct : sms), kThreads, smem, stream>>>(p, ma, mb, wa, wb);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_matmul_fp4(const MatmulFp4Params& p, int sms, const char** error, cudaStream_t stream) {
  const bool narrow = p.M <= int64_t(p.E) * 200;
  if (p.out_bf16) return narrow ? launch<128, true>(p, sms, error, stream) : launch<256, true>(p, sms, error, stream);
  return narrow ? launch<128, false>(p, sms, error, stream) : launch<256, false>(p, sms, error, stream);
}

}  // namespace moe
