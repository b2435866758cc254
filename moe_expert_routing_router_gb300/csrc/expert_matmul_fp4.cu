// The experts' 4-bit matrix products on the fifth-generation tensor cores.
//
// Operands are e2m1 codes, two in a byte, with one power-of-two scale for 32 values along
// the contraction.  tcgen05.mma of kind mxf4 takes both operands' codes from shared
// memory and their scales from tensor memory, and multiplies a block's products by its two
// scales itself: a tile's sum stays in tensor memory over the whole contraction, in fp32,
// and is read once.
//
// One persistent CTA per SM, 12 warps: a producer of codes and one of scales, an MMA issuer,
// one that mends a last product's scales, and 8 epilogue warps of 32 rows by half of the
// tile's columns.  A stage of the ring in shared memory holds 256 values of the contraction
// of both operands (rows of 128 bytes, 128-byte swizzled) and their scales.  Those lie in
// memory as words of four, of 128 values each, one row behind another; the tensor core
// wants the words of rows r, r + 32, r + 64 and r + 96 beside one another in lane r of tensor
// memory, for each of its four quarters: 16-byte pieces in shared memory, of which one
// tcgen05.cp copies 32 to all quarters in front of the products that read them.
//   b: the words of rows 4 r .. 4 r + 3 make a piece as they lie, so that tensor copies bring
//      them, and row 4 r + j of the codes is brought to row 32 j + r; the epilogue reads the
//      sum's columns accordingly.  (With all scales as a's: 345 us instead of 217, of 64 experts
//      of 2048 by 4096 and 1024 rows each, when that was changed.)
//   a: its rows start anywhere, so a warp copies word by word.
// A stage's scales have columns of their own in tensor memory, so that their reuse is
// ordered by the stage's.
//
// What bounds it: with few rows of an expert the weights' reading, 50 us for 64 experts of 2048 by
// 4096 (285 MB, 5.7 TB/s; 8 rows each).  With many, 1024 each, 208 us and 5.3 PFLOP/s: no limit is shown to be met.
// A stage's products would take 390 cycles by the nominal rate, and the tensor pipe is busy half of the time; the stages of all
// SMs bring 16 TB/s from L2.  Over seconds such calls meet the power limit (1363 W): 223 us, 910 cycles a stage at 1762 MHz.
// Narrow tiles do not (327 us, 784 cycles a stage at 2070 MHz and 1290 W).  CTA pairs, which bring 35 KB a stage instead of 52,
// were no more than 6 percent faster with 1024 rows each, and slower with 256; their clock was not recorded.
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
constexpr int kEpiWarps = 8, kFirstEpi = 4;
constexpr int kThreads = (kFirstEpi + kEpiWarps) * kWarp;
// Registers of a thread: as launched, of the first four warps then, and of the others, which
// take a tile's sums out of tensor memory at once, so that the next tile's products can start.
constexpr int kLaunchRegs = 168, kRegs = 72, kEpiRegs = 216;
static_assert(kFirstEpi * kRegs + kEpiWarps * kEpiRegs <= (kFirstEpi + kEpiWarps) * kLaunchRegs, "registers of the launch");
constexpr int kMaxE = 1024;
constexpr int kGroupM = 16;                   // row tiles of an expert that are taken before the next column tile
constexpr int kAtomBytes = 512;               // scales of 128 rows by 128 values
constexpr int kBox = 32;                      // rows of a in one copy: a ragged tile copies only those that it needs
constexpr int kGroup = 4;                     // rows of b whose scales make one piece

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

template <int N>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N)); }
template <int N>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N)); }

__device__ __forceinline__ void copy_word(uint32_t to, const uint32_t* from, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" :: "r"(to), "l"(from), "r"(there ? 4 : 0) : "memory");
}
// Arrives on the barrier when the thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void tma_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int v, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];"
      :: "r"(smem_addr(dst)), "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(y), "r"(z), "r"(v) : "memory");
}

// Whether the phase has completed, without waiting.
__device__ __forceinline__ bool mbar_peek(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(smem_addr(bar)), "r"(parity) : "memory");
  return ok != 0;
}

// ---- the kernel ----------------------------------------------------------------------
template <int BN>
struct Tile {
  static constexpr int kCodeBytes = (kBM + BN) * kRowBytes;
  static constexpr int kScaleBytes = (kBM + BN) / 128 * 2 * kAtomBytes;   // of a: two words, of b: two words of each atom
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
  uint64_t fixed[8];                          // a stage's scales are as the products need them
  uint32_t tmem;
  int abort;
  int row[kMaxE], count[kMaxE], first[kMaxE + 1];   // an expert's first row and rows; tiles before it
};

__device__ __forceinline__ bool wait(Shared& sh, const MatmulFp4Params& p, uint64_t* bar, uint32_t parity) {
  return mbar_test(bar, parity) || pipeline_wait(&sh.abort, p.errors, p.timeout_ns, bar, parity);
}

// A place in the ring.
template <int N>
struct Slot {
  int s;
  uint32_t phase;
  __device__ __forceinline__ explicit Slot(int64_t stage) : s(int(stage % N)), phase(uint32_t(stage / N) & 1u) {}
  __device__ __forceinline__ void next() {
    if (++s == N) {
      s = 0;
      phase ^= 1u;
    }
  }
};

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
    const int i = tile - sh.first[e], rt = int((unsigned(sh.count[e]) + kBM - 1) / kBM);
    // kGroupM row tiles by all column tiles at a time, rows fastest: the CTAs at
    // work share both operands' tiles in L2.
    const int group = rt <= kGroupM ? 0 : i / (kGroupM * ct), in = i - group * kGroupM * ct;
    const int gm = min(kGroupM, rt - group * kGroupM);
    const int col = int(__fdividef(float(in) + 0.5f, float(gm)));   // in / gm, of at most 2^17: off by less than 1 / 32
    const int r0 = (group * kGroupM + in - col * gm) * kBM;
    col0 = col * BN;
    cols = min(BN, p.C - col0);
    row0 = sh.row[e] + r0;
    rows = min(kBM, sh.count[e] - r0);
  }
};

template <int BN, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
expert_matmul_fp4_kernel(const __grid_constant__ MatmulFp4Params p, const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                         const __grid_constant__ CUtensorMap whole_a, const __grid_constant__ CUtensorMap whole_b,
                         const __grid_constant__ CUtensorMap map_sb) {
  using TL = Tile<BN>;
  extern __shared__ uint8_t s_dyn[];
  __shared__ Shared sh;
  uint8_t* ring = s_dyn + (1024 - smem_addr(s_dyn) % 1024) % 1024;
  uint8_t* scales = ring + TL::kStages * TL::kCodeBytes;
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;
  const int stages = (p.K + kBK - 1) / kBK;                      // of a tile

  for (int e = threadIdx.x; e < p.E; e += kThreads) {
    int64_t start, n;
    expert_rows(p, e, &start, &n);
    sh.row[e] = int(start);
    sh.count[e] = int(n);
  }
  if (warp == 0) {
    if (lane == 0) {
      for (const CUtensorMap* m : {&map_a, &map_b, &whole_a, &whole_b, &map_sb})
        asm volatile("prefetch.tensormap [%0];" :: "l"(m) : "memory");
      for (int i = 0; i < TL::kStages; ++i) {
        mbar_init(&sh.full[i], 2 + kWarp + p.extra);
        mbar_init(&sh.done[i], 1);
        mbar_init(&sh.fixed[i], 1);
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
  }
  __syncthreads();
  if (warp == 2) {                                               // tiles before each expert
    const int ct = (p.C + BN - 1) / BN;
    int tiles = 0;
    float sum = 0.f;                                             // of the tiles, where ranges that overlap pass an int
    for (int e0 = 0; e0 < p.E; e0 += kWarp) {
      int t = 0;
      if (e0 + lane < p.E) {
        t = int((int64_t(sh.count[e0 + lane]) + kBM - 1) / kBM) * ct;
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

  // A warp finds its tile together; one elected thread runs through the tile's stages.
  // `at` counts the stages before the tile, `issued` those of which copies have been started.
  const auto drain = [&](int64_t issued) {                       // copies in flight land before shared memory goes
    for (int64_t i = issued > TL::kStages ? issued - TL::kStages : 0; i < issued; ++i) {
      const Slot<TL::kStages> q(i);
      mbar_wait(&sh.full[q.s], q.phase, p.timeout_ns);
    }
  };
  bool ok = true;
  int64_t at = 0;
  if (warp < kFirstEpi) fewer_registers<kRegs>();
  if (warp == 0) {
    // ---- producer: the codes ----
    Walk w;
    for (int tile = blockIdx.x; tile < n_tiles && ok; tile += gridDim.x) {
      w.at<BN>(p, sh, tile);
      int n = 0;
      if (elect_one()) {
        const int b_row = w.e * p.C + w.col0, atoms = (w.cols + 127) / 128;
        const int boxes = (w.rows + kBox - 1) / kBox;
        const uint32_t bytes = (boxes * kBox + atoms * 128) * kRowBytes;
        Slot<TL::kStages> q(at);
        for (; n < stages; ++n, q.next()) {
          if (!wait(sh, p, &sh.done[q.s], q.phase ^ 1u)) break;
          uint64_t* bar = &sh.full[q.s];
          uint8_t *sa = ring + q.s * TL::kCodeBytes, *sb = sa + kBM * kRowBytes;
          mbar_arrive_expect_tx(bar, bytes);
          if (boxes == kBM / kBox) tma_2d(sa, &whole_a, n * kRowBytes, w.row0, bar);
          else for (int i = 0; i < boxes; ++i) tma_2d(sa + i * kBox * kRowBytes, &map_a, n * kRowBytes, w.row0 + i * kBox, bar);
          if (w.cols == BN) tma_4d(sb, &whole_b, n * kRowBytes, b_row / kGroup, 0, 0, bar);
          else for (int i = 0; i < atoms; ++i) tma_4d(sb + i * 128 * kRowBytes, &map_b, n * kRowBytes, b_row / kGroup + i * 32, 0, 0, bar);
        }
      }
      n = __reduce_max_sync(kFull, n);
      ok = n == stages;
      at += n;
    }
    if (!ok) drain(at);
  } else if (warp == 1) {
    // ---- MMA issuer ----
    // D fp32; A and B e2m1, both K-major; scales are exponents (bit 23); N = BN, M = 128
    constexpr uint32_t idesc = 1u << 7 | 1u << 10 | uint32_t(BN / 8) << 17 | 1u << 23 | uint32_t(kBM / 16) << 24;
    const uint64_t desc0 = smem_desc(ring), sdesc0 = scale_desc(scales);
    const int last_steps = (p.K - (stages - 1) * kBK + kMmaK - 1) / kMmaK;
    uint64_t* full = p.K % kMmaK != 0 ? sh.fixed : sh.full;
    int t = 0;
    uint32_t tphase = 0;
    for (int tile = blockIdx.x; tile < n_tiles && ok; tile += gridDim.x) {
      int n = 0;
      if (elect_one() && wait(sh, p, &sh.tempty[t], tphase ^ 1u)) {
        Slot<TL::kStages> q(at);
        bool there = false;
        for (; n < stages; ++n) {
          if (!there && !wait(sh, p, &full[q.s], q.phase)) break;
          const bool last = n + 1 == stages;
          async_proxy_fence();                                   // the words that the scale warp's copies wrote
          tc_fence_after();
          const uint64_t da = desc0 + uint64_t(q.s * TL::kCodeBytes >> 4), db = da + (kBM * kRowBytes >> 4);
          const uint64_t ds = sdesc0 + uint64_t(q.s * TL::kScaleBytes >> 4);
          const uint32_t sc = tmem + TL::kFirstScale + q.s * TL::kScaleCols;
          uint64_t* done = &sh.done[q.s];
          q.next();
          there = !last && mbar_peek(&full[q.s], q.phase);
#pragma unroll
          for (int i = 0; i < TL::kScaleBytes / kAtomBytes; ++i) tc_copy_scales(sc + 4 * i, ds + i * (kAtomBytes >> 4));
#pragma unroll
          for (int k = 0; k < kBK / kMmaK; ++k) {                // 32 bytes along the row: 2 units of 16; half a word of scales
            if (last && k >= last_steps) break;
            const uint32_t half = uint32_t(k % 2) * 2;
            tc_mma_fp4(tmem + t * BN, da + k * 2, db + k * 2, idesc | half << 4 | half << 29, sc + k / 2 * (kBM / 32),
                       sc + 2 * (kBM / 32) + k / 2 * (BN / 32), n > 0 || k > 0);
          }
          tc_commit(done);                                       // the stage is free
          if (last) tc_commit(&sh.ready[t]);
        }
      }
      n = __reduce_max_sync(kFull, n);
      ok = n == stages;
      at += n;
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
  } else if (warp == 2) {
    // ---- producer: the scales, those of a by the whole warp ----
    const int words = (p.K + 127) / 128;
    Walk w;
    for (int tile = blockIdx.x; tile < n_tiles && ok; tile += gridDim.x) {
      w.at<BN>(p, sh, tile);
      const int b_row = w.e * p.C + w.col0;
      int n = 0;
      for (Slot<TL::kStages> q(at); n < stages && __all_sync(kFull, wait(sh, p, &sh.done[q.s], q.phase ^ 1u)); ++n, q.next()) {
        uint8_t* ss = scales + q.s * TL::kScaleBytes;
        if (elect_one()) {
          mbar_arrive_expect_tx(&sh.full[q.s], TL::kScaleBytes - 2 * kAtomBytes);
          tma_2d(ss + 2 * kAtomBytes, &map_sb, b_row, 2 * n, &sh.full[q.s]);
        }
        __syncwarp();
        const uint32_t to = smem_addr(ss + lane * 16);
        const uint32_t* from = p.a_scale + 2 * n * p.M + w.row0 + lane;
        const bool two = 2 * n + 1 < words;
        for (int i = 0; i * kBox < w.rows; ++i, from += kBox) {
          const bool there = w.row0 + int64_t(i) * kBox + lane < p.M;   // nothing is read, and zero written, where it is not
          copy_word(to + i * 4, there ? from : p.a_scale, there);
          copy_word(to + kAtomBytes + i * 4, there && two ? from + p.M : p.a_scale, there && two);
        }
        copies_arrive(&sh.full[q.s]);
      }
      n = __reduce_max_sync(kFull, n);
      ok = n == stages;
      at += n;
    }
    copies_wait();
    if (!ok) drain(at);
  } else if (warp == 3) {
    // ---- where the last product's second block is not there: its scale may be anything, and becomes the smallest ----
    const int blocks = (p.K - (stages - 1) * kBK) / 32;
    Slot<TL::kStages> q(0);
    for (int tile = blockIdx.x; tile < n_tiles && ok && p.K % kMmaK != 0; tile += gridDim.x) {
      for (int n = 0; n < stages; ++n, q.next()) {
        ok = __all_sync(kFull, wait(sh, p, &sh.full[q.s], q.phase));
        if (!ok) break;
        if (n + 1 == stages) {
          uint32_t *sa = reinterpret_cast<uint32_t*>(scales + q.s * TL::kScaleBytes), *sb = sa + 2 * kBM;
          for (int i = lane; i < kBM; i += kWarp) sa[blocks / 4 * kBM + i] &= ~(0xffu << blocks % 4 * 8);
          for (int i = lane; i < BN; i += kWarp) sb[blocks / 4 * BN + i] &= ~(0xffu << blocks % 4 * 8);
          async_proxy_fence();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(&sh.fixed[q.s]);
      }
    }
  } else {
    // ---- epilogue: 32 rows, kCols columns ----
    more_registers<kEpiRegs>();
    const int quad = warp % 4, part = (warp - kFirstEpi) / 4;
    int t = 0;
    uint32_t tphase = 0;
    Walk w;
    for (int tile = blockIdx.x; tile < n_tiles; tile += gridDim.x) {
      w.at<BN>(p, sh, tile);
      if (!__all_sync(kFull, wait(sh, p, &sh.ready[t], tphase))) break;
      tc_fence_after();
      const int c0 = w.col0 + part * TL::kCols;
      const bool any = quad * 32 < w.rows && c0 < p.C;
      // Pieces of 16 bytes, NP of which are turned among NP lanes at a time.
      constexpr int kPer = BF16 ? 8 : 4, NP = 8, kPieces = TL::kCols / kPer;
      uint32_t u[TL::kCols / 64][4][16];
      if (any) {
        // column 4 l + j of 128 lies in column 32 j + l of tensor memory
        const uint32_t addr = tmem + t * BN + (BN == 256 ? part * 128 : part * 16) + (uint32_t(quad * 32) << 16);
#pragma unroll
        for (int c = 0; c < TL::kCols / 64; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) tmem_ld16(addr + j * 32 + c * 16, u[c][j]);
#pragma unroll
        for (int c = 0; c < TL::kCols / 64; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) tmem_ld_wait(u[c][j]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.tempty[t]);                 // the next tile's products may start
      if (any) {
#pragma unroll
        for (int i = 0; i < kPieces; i += NP) {
          uint4 v[NP];
#pragma unroll
          for (int n = 0; n < NP; ++n) {
            const int c = (i + n) * kPer / 64, l = (i + n) * kPer % 64 / 4;
            if constexpr (BF16) {
              uint32_t b2[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t* from = &u[c][j % 2 * 2][l + j / 2];
                const __nv_bfloat162 q = __floats2bfloat162_rn(__uint_as_float(from[0]), __uint_as_float(from[16]));
                b2[j] = *reinterpret_cast<const uint32_t*>(&q);
              }
              v[n] = make_uint4(b2[0], b2[1], b2[2], b2[3]);
            } else {
              v[n] = make_uint4(u[c][0][l], u[c][1][l], u[c][2][l], u[c][3][l]);
            }
          }
          turn<NP>(v, lane);
          const int col = c0 + (i + lane % NP) * kPer;               // C is a multiple of 16: a piece is whole
#pragma unroll
          for (int r = 0; r < NP; ++r) {
            const int to = quad * 32 + lane / NP * NP + r;
            if (to < w.rows && col < p.C)
              *reinterpret_cast<uint4*>(static_cast<char*>(p.out) + (int64_t(w.row0 + to) * p.C + col) * (BF16 ? 2 : 4)) = v[r];
          }
        }
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

// Codes [rows, K/2] of b in boxes of 128 bytes by 128 rows: row 4 l + j of them is brought to row 32 j + l.
// `blocks` such boxes at once have to lie inside the rows.
bool grouped_map(CUtensorMap* map, const void* base, uint64_t rows, int K, cuuint32_t blocks) {
  const uint64_t row = uint64_t(K) / 2;
  const cuuint64_t dims[4] = {row, rows / kGroup, kGroup, blocks}, strides[3] = {row * kGroup, row, row * 128};
  const cuuint32_t box[4] = {kRowBytes, 128 / kGroup, kGroup, blocks}, ones[4] = {1, 1, 1, 1};
  return encode_fn() != nullptr &&
         encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scales [words, rows] in boxes of two words of n rows.
bool scale_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t words, cuuint32_t n) {
  const cuuint64_t dims[2] = {rows, words}, strides[1] = {rows * 4};
  const cuuint32_t box[2] = {n, 2}, ones[2] = {1, 1};
  return encode_fn() != nullptr &&
         encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, bool BF16>
cudaError_t launch(const MatmulFp4Params& p, int sms, const char** error, cudaStream_t stream) {
  using TL = Tile<BN>;
  CUtensorMap ma, mb, wa, wb, sb;
  const uint64_t cols = uint64_t(p.K) / 2, rows_b = uint64_t(p.E) * p.C, words = (uint64_t(p.K) + 127) / 128;
  if (!make_map(&ma, p.a, uint64_t(p.M), cols, kBox) || !make_map(&wa, p.a, uint64_t(p.M), cols, kBM) ||
      !grouped_map(&mb, p.b, rows_b, p.K, 1) || !grouped_map(&wb, p.b, rows_b, p.K, BN / 128) || !scale_map(&sb, p.b_scale, rows_b, words, BN)) {
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
  kernel<<<unsigned(rt * ct < sms ? rt * ct : sms), kThreads, smem, stream>>>(p, ma, mb, wa, wb, sb);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_expert_matmul_fp4(const MatmulFp4Params& p, int sms, const char** error, cudaStream_t stream) {
  // Tiles of 256 columns take 1.3 to 1.7 times as long as those of 128, if their products bound them, so
  // that the rounds of tiles decide: 1024 rows by 64 experts of 2048 by 4096, 351 us in 58 rounds of
  // narrow ones and 218 in 29 of wide ones; 512 rows by 8 of 1040 by 1440, 18.9 in 3 and 21.0 in 2.  With fewer
  // rows the weights' reading does, which narrow tiles share out more evenly (64 rows: 66.8 and 68.7 us).  All
  // of one call alone, behind a flush of L2, experts' rows drawn at random around these.
  const auto rounds = [&](int cols) { return ((2 * p.M / kBM + p.E) * ((p.C + cols - 1) / cols) / 2 + sms - 1) / sms; };
  const bool narrow = p.M <= int64_t(p.E) * 100 || rounds(128) * 5 <= rounds(256) * 8;
  if (p.out_bf16) return narrow ? launch<128, true>(p, sms, error, stream) : launch<256, true>(p, sms, error, stream);
  return narrow ? launch<128, false>(p, sms, error, stream) : launch<256, false>(p, sms, error, stream);
}

}  // namespace moe
