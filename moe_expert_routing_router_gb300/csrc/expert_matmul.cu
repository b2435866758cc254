// The experts' 8-bit matrix products on the fifth-generation tensor cores.
//
// Operands are e4m3 with a fp32 scale for each block of 128 along the
// contraction.  A block's product is formed by four tcgen05.mma (K = 32 each)
// in tensor memory, from zero; the epilogue warps read it back, multiply by the
// block's two scales and add it in fp32 registers, which hold the tile's sum
// over all blocks.  The scales may be any fp32 numbers, and no sum is kept in
// fewer than 32 bits.
//
// One persistent CTA per SM, 20 warps: a TMA producer (one thread), an MMA
// issuer (one thread), a warp that looks at the rows' scales (weight gradient), a spare
// one, and 16 epilogue warps of 32 rows by a quarter of the tile's columns.  Shared memory is a ring of operand stages (one block
// of 128 of both operands, 128-byte swizzled); tensor memory is a ring of block
// products, so that the tensor core forms block b + 1 while the epilogue adds
// block b, and runs ahead into the next tile while a tile is stored.
//
// Every wait is bounded: when one runs out, the CTA records the pipeline's error
// bit, drains its copies and returns.
#include "device_common.cuh"
#include "expert_matmul.h"

#include <cuda.h>
#include <cuda_bf16.h>

#include <atomic>

namespace moe {
namespace {

constexpr int kBM = 128;                      // rows of a tile
constexpr int kBK = 128;                      // block along the contraction: bytes of e4m3, and one scale
constexpr int kBox = 32;                      // rows of one copy of a ragged tile, which copies only those it needs; a whole
                                              // one takes one copy of 128 rows (an issue costs some 30 ns)
constexpr int kEpiWarps = 16, kFirstEpi = 4;
constexpr int kMmThreads = (kFirstEpi + kEpiWarps) * kWarp;
constexpr int kTmemCols = 512;
constexpr int kMaxE = 1024;
constexpr int kOutCols = 32;                  // columns of a tensor copy of results: 128 bytes of fp32
constexpr int kWarpOutBytes = 32 * kOutCols * 4;
constexpr int kGroupM = 16;                   // row tiles of an expert that are taken before the next column tile
constexpr unsigned kFull = 0xffffffffu;

// Error bits of the device's calls: they carry no other state from call to call,
// so calls on any streams, and captured ones, share the word.
__device__ int g_mm_errors;

// Read and cleared in one step, so that a call that finds bits set is always followed by the
// read that tells of them.  As many reads as this may wait at once, each in a place of its own.
constexpr unsigned kReads = 256;
__device__ int g_mm_read[kReads];
__global__ void take_errors_kernel(unsigned place) { g_mm_read[place] = atomicExch(&g_mm_errors, 0); }

// ---- tcgen05 / TMA primitives ------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t* slot) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" :: "r"(smem_addr(slot)), "r"(kTmemCols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(addr), "r"(kTmemCols) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// Arrives on the barrier when the products issued so far have ended.
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(smem_addr(bar)) : "memory");
}

__device__ __forceinline__ void tc_mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}

__device__ __forceinline__ void tma_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
      :: "r"(smem_addr(dst)), "l"(map), "r"(smem_addr(bar)), "r"(x), "r"(y) : "memory");
}

// Shared memory to a box of out [E, R, C]; what lies outside is not written.
__device__ __forceinline__ void tma_store_3d(const void* src, const CUtensorMap* map, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];"
               :: "l"(map), "r"(smem_addr(src)), "r"(x), "r"(y), "r"(z) : "memory");
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               :: "r"(smem_addr(dst)), "l"(src), "r"(bytes), "r"(smem_addr(bar)) : "memory");
}
// Ends a group of stores; a group may be empty.
__device__ __forceinline__ void tma_store_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Until the thread's groups have read their shared memory / have ended.
__device__ __forceinline__ void tma_store_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_store_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void async_proxy_fence() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// One thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
  return ok != 0;
}

// Shared-memory matrix descriptor of a K-major operand in rows of 128 bytes,
// 128-byte swizzle: groups of 8 rows lie 1024 bytes apart.
__device__ __forceinline__ uint64_t smem_desc(const void* p) {
  return uint64_t((smem_addr(p) >> 4) & 0x3fffu) | uint64_t(1) << 16 | uint64_t(1024 >> 4) << 32 | uint64_t(1) << 46 |
         uint64_t(2) << 61;
}

// 16 columns of the warp's 32 rows, asynchronously.
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15"
      "}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr) : "memory");
}
// 16 rows by 32 columns, spread like a matrix product's fragments: for the n-th 8 columns,
// lane l gets columns 2 (l % 4) and the next one of row l / 4 in r[4 n], r[4 n + 1], and of
// row l / 4 + 8 in r[4 n + 2], r[4 n + 3].
__device__ __forceinline__ void tmem_ld_16x32(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15"
      "}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr) : "memory");
}
// Waits for the thread's loads.  The values pass through the statement, so that
// no use of them can be moved before it.
__device__ __forceinline__ void tmem_ld_wait(uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
        "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
      :: "memory");
}

// Lane l of each NP neighbouring lanes holds the NP pieces of row l in v; after
// it, v[r] is piece l of row r.  Rows are then stored NP * 16 bytes at a time
// instead of 16: a store of 32 rows takes a cycle a row.
template <int NP>
__device__ __forceinline__ void turn(uint4* v, int lane) {
#pragma unroll
  for (int s = 1; s < NP; s <<= 1) {
    const bool up = lane & s;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if (i & s) continue;
      uint4 x = up ? v[i] : v[i | s];
      x.x = __shfl_xor_sync(kFull, x.x, s);
      x.y = __shfl_xor_sync(kFull, x.y, s);
      x.z = __shfl_xor_sync(kFull, x.z, s);
      x.w = __shfl_xor_sync(kFull, x.w, s);
      if (up) v[i] = x;
      else v[i | s] = x;
    }
  }
}

// ---- the kernel ----------------------------------------------------------------
// RB: blocks that share a stage, its barriers and its place in tensor memory.
// STORE: the tile leaves through shared memory by tensor copies (a buffer of 4 KB a
// warp), which costs a stage.
template <int BN, int RB, bool STORE>
struct Tile {
  static constexpr int kBlockBytes = (kBM + BN) * kBK;
  static constexpr int kStageBytes = RB * kBlockBytes;
  static constexpr int kOutBytes = STORE ? kEpiWarps * kWarpOutBytes : 0;
  static constexpr int kStages = 196608 / kStageBytes - (STORE ? 1 : 0);   // 192 KB, or 144 KB, of operands
  static constexpr int kBufs = kTmemCols / (BN * RB);          // stages' products in tensor memory
  static constexpr int kCols = BN / 4;                         // columns of one epilogue warp
};

// Blocks whose scales the weight gradient holds in shared memory: its producer copies them
// beside the operands (32,836 rows of 32 experts, 2048 x 2048: 282 -> 228 us, with wider
// copies of the results, against loads by the epilogue's lanes).
constexpr int kScaleSlots = 6;

template <bool WGRAD>
struct alignas(16) Shared {
  // full: a stage's operands have landed; done: its product has been formed (the
  // producer may fill it again, the epilogue may read); tempty: the product has been read;
  // scales: a block's scales have landed
  uint64_t full[8], done[8], tempty[8], drain, scales[kScaleSlots];
  uint32_t tmem;
  int abort;
  int redo;                                                    // a row's scales are not plain
  int block[kMaxE + 1];                                        // weight gradient: column blocks before expert e; product: its first row
  int first[WGRAD ? 1 : kMaxE + 1];                            // product: tiles before expert e
  int count[WGRAD ? 1 : kMaxE];                                // product: its rows
  alignas(16) float scale[WGRAD ? kScaleSlots : 1][kBM + 256]; // weight gradient: a block's scales of rows and columns
};

// Bounded wait that every role uses: false once it, or another role's, ran out.
// Time is counted in SM cycles (at most about two a nanosecond), whose counter is
// read in a few cycles, and only after some waits have failed.
// With a second barrier, both are tested at once: a test takes some 100 cycles.
template <class S>
__device__ __forceinline__ bool mm_wait(S& sh, const MatmulParams& p, uint64_t* bar, uint32_t parity,
                                        uint64_t* bar2 = nullptr, uint32_t parity2 = 0) {
  const auto test = [&]() {
    const bool a = mbar_test(bar, parity), b = bar2 == nullptr || mbar_test(bar2, parity2);
    return a && b;
  };
#pragma unroll 1
  for (int i = 0; i < 32; ++i)
    if (test()) return true;
  const long long t0 = clock64();
  while (!test()) {
    if (*reinterpret_cast<volatile int*>(&sh.abort) != 0) return false;
    if (clock64() - t0 > 2 * (long long)(p.timeout_ns)) {
      *reinterpret_cast<volatile int*>(&sh.abort) = 1;
      atomicOr(&g_mm_errors, kErrPipelineTimeout);
      return false;
    }
  }
  return true;
}

// The rows of expert e: their place and number, whatever the arrays hold, inside [0, M).
__device__ __forceinline__ void expert_rows(const MatmulParams& p, int e, int64_t* start, int64_t* n) {
  if (p.offsets == nullptr) {
    *start = 0;
    *n = p.M;
    return;
  }
  const int64_t lo = min(max(int64_t(p.offsets[e]), int64_t(0)), p.M);
  const int64_t hi = min(max(int64_t(p.offsets[e + 1]), lo), p.M);
  *start = lo;
  *n = p.kept != nullptr ? min(hi - lo, max(int64_t(p.kept[e]), int64_t(0))) : hi - lo;
}

__device__ __forceinline__ int boxes(int rows) { return (rows + kBox - 1) / kBox; }

// A tile of the persistent loop, walked in ascending order by every role.
struct Walk {
  int e = 0;
  int row0 = 0, rows = 0;         // rows of a: the first one and how many are the tile's
  int col0 = 0, cols = 0;         // columns of out within the expert
  int r0 = 0;                     // the tile's first row within the expert's out
  int block0 = 0, blocks = 0;     // blocks along the contraction

  template <int BN, bool WGRAD>
  __device__ __forceinline__ void at(const MatmulParams& p, const Shared<WGRAD>& sh, int tile) {
    const int ct = (p.C + BN - 1) / BN;
    int i = tile, rt = (p.R + kBM - 1) / kBM;                    // of the expert: the tile's place, tiles of rows
    if constexpr (WGRAD) {
      e = tile / (rt * ct);
      i -= e * rt * ct;
    } else {
      for (;;) {                                                 // the expert that has the tile: 32 at a time, by the whole warp
        const int next = e + 1 + int(threadIdx.x % kWarp);
        const unsigned past = __ballot_sync(kFull, next <= p.E && sh.first[next] <= tile);
        e += __popc(past);
        if (past != kFull) break;
      }
      i -= sh.first[e];
      rt = (sh.first[e + 1] - sh.first[e]) / ct;
    }
    // kGroupM row tiles by all column tiles at a time, rows fastest: the CTAs at
    // work share both operands' tiles in L2.
    const int group = i / (kGroupM * ct), in = i - group * kGroupM * ct;
    const int gm = min(kGroupM, rt - group * kGroupM);
    const int m = group * kGroupM + in % gm;
    col0 = in / gm * BN;
    cols = min(BN, p.C - col0);
    r0 = m * kBM;
    if constexpr (WGRAD) {
      row0 = r0;
      rows = min(kBM, p.R - r0);
      block0 = sh.block[e];
      blocks = sh.block[e + 1] - block0;
    } else {
      row0 = sh.block[e] + r0;
      rows = min(kBM, sh.count[e] - r0);
      block0 = 0;
      blocks = (p.K + kBK - 1) / kBK;
    }
  }
};

// ---- scales at the ends of fp32 ---------------------------------------------------
// Scales may be any fp32 numbers.  A block's sum is 0 or between 2^-18 and 2^25 in size: one
// multiplication by a product of scales that is a normal number loses nothing, nor do two in
// turn by scales of which the first lies between 2^-108 and 2^103.  Other rows, whose term can
// be an ordinary number all the same, are computed once more behind the last tile.
// (Decided block by block, with a second way to add one: the weight gradient 218 -> 228 us,
// 512 rows of 64 experts 94 -> 98 us.)  Of 65,536 rows of 64 experts a 64th once more takes
// 5 ms, all of them 16 ms; where scales of 0 have the rows looked at, a fifth of the call.
template <bool WGRAD>
__device__ __forceinline__ bool plain_scale(float s) {           // what is not a number stays one either way
  return !(fabsf(s) < (WGRAD ? 0x1p-108f : 0x1p-126f)) && !(fabsf(s) > (WGRAD ? 0x1p103f : 0x1.fffffep127f));
}

// Of a row and of a column; what a scale of 0 makes of any sum is the same either way.
template <bool WGRAD>
__device__ __forceinline__ bool plain_pair(float sa, float sb) { return plain_scale<WGRAD>(sa * sb) || sa == 0.f || sb == 0.f; }

// Two numbers with the product of r and f, by which a block's sum is multiplied in turn without
// leaving the normal numbers before the whole term does: the same two, or both moved by a
// power of two.  (Digits of f lost below 2^-126 belong to a term below fp32's smallest; an f
// that is cut at 2^101 makes the same infinity.)
__device__ __forceinline__ float2 apart(float r, float f) {
  if (plain_scale<true>(r)) return make_float2(r, f);
  if (fabsf(r) < 1.f) return make_float2(r * 0x1p64f, f * 0x1p-64f);
  const bool cut = fabsf(f) > 0x1p101f && fabsf(f) <= 0x1.fffffep127f;
  return make_float2(r * 0x1p-26f, (cut ? copysignf(0x1p101f, f) : f) * 0x1p26f);
}

// The epilogue's warps and the one that looks at the scales meet.
__device__ __forceinline__ void scales_known() { asm volatile("bar.sync 1, %0;" :: "n"((kEpiWarps + 1) * kWarp) : "memory"); }

// Four e4m3 codes as fp16, which holds them.
__device__ __forceinline__ void codes_f16(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(lo) : "h"(uint16_t(codes)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(hi) : "h"(uint16_t(codes >> 16)));
}
// d [16, 8] += a [16, 16] b [16, 8]: lane l holds columns 2 (l % 4) and the next one of rows
// l / 4 and l / 4 + 8 of d.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A warp's rows of a tile whose scales are not plain, from the operands: 16 such rows at a
// time by all the warp's columns, on fp16 products; half a block's sum and its scales by
// `apart`.  Row `row0` of a and column `col0` of expert e are the first; `to` is out's row of
// row0.  Both operands' codes are taken in the same order, 16 neighbours a lane.  (Single
// products, a column a lane: 132 ms instead of 16.)
template <int CW, bool WGRAD, bool BF16>
__device__ __forceinline__ void redo_rows(const MatmulParams& p, int e, int row0, int rows, int col0, int cols, int block0, int blocks, int64_t to) {
  const int lane = threadIdx.x % kWarp, g = lane / 4, t = lane % 4;
  const int64_t width = WGRAD ? p.blocks * kBK : p.K;
  const int kblocks = (p.K + kBK - 1) / kBK, cblocks = (p.C + kBK - 1) / kBK;
  const int64_t b_row0 = (WGRAD ? 0 : int64_t(e) * p.C) + col0;
  const float* b_scales = WGRAD ? p.b_scale + col0 : p.b_scale + (int64_t(e) * cblocks + col0 / kBK) * kblocks;
  const auto a_scale = [&](int r, int b) { return r < rows ? p.a_scale[int64_t(b) * (WGRAD ? p.R : p.M) + row0 + r] : 0.f; };
  bool redo = false;                                             // row `lane`
#pragma unroll 8
  for (int b = block0; b < block0 + blocks; ++b) redo |= !plain_pair<WGRAD>(a_scale(lane, b), WGRAD ? 1.f : b_scales[b]);
  unsigned which = __ballot_sync(kFull, redo);
  while (which != 0u) {
    int row[2] = {32, 32};                                       // the lane's rows: the g-th and (g + 8)-th, 32 for none
    for (int i = 0; i < 16 && which != 0u; ++i, which &= which - 1u)
      if (i % 8 == g) row[i / 8] = __ffs(which) - 1;
    float sum[CW / 8][4];
#pragma unroll
    for (int n = 0; n < CW / 8; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[n][i] = 0.f;
    for (int h = 2 * block0; h < 2 * (block0 + blocks); ++h) {   // half a block
      const int64_t x = int64_t(h) * (kBK / 2) + t * 16;
      const auto piece = [&](const uint8_t* m, int64_t at, bool there) {
        return there && x < width ? *reinterpret_cast<const uint4*>(m + at * width + x) : make_uint4(0u, 0u, 0u, 0u);
      };
      const uint4 v0 = piece(p.a, int64_t(row0) + row[0], row[0] < rows), v1 = piece(p.a, int64_t(row0) + row[1], row[1] < rows);
      const float sa[2] = {a_scale(row[0], h / 2), a_scale(row[1], h / 2)};
      uint32_t a[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        codes_f16(i == 0 ? v0.x : i == 1 ? v0.y : i == 2 ? v0.z : v0.w, a[i][0], a[i][2]);
        codes_f16(i == 0 ? v1.x : i == 1 ? v1.y : i == 2 ? v1.z : v1.w, a[i][1], a[i][3]);
      }
#pragma unroll
      for (int n = 0; n < CW / 8; ++n) {
        const bool there = n * 8 < cols;                         // cols is a multiple of 16
        const uint4 v = piece(p.b, b_row0 + n * 8 + g, there);
        float dot[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t b0, b1;
          codes_f16(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w, b0, b1);
          mma_f16(dot, a[i][0], a[i][1], a[i][2], a[i][3], b0, b1);
        }
        float2 sb;
        if constexpr (WGRAD) sb = there ? *reinterpret_cast<const float2*>(b_scales + int64_t(h / 2) * p.C + n * 8 + 2 * t) : make_float2(0.f, 0.f);
        else sb.x = sb.y = b_scales[h / 2];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 s = apart(sa[i / 2], i % 2 == 0 ? sb.x : sb.y);
          sum[n][i] = fmaf(dot[i] * s.x, s.y, sum[n][i]);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < CW / 8; ++n)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (row[i] >= rows || n * 8 >= cols) continue;
        const int64_t at = (to + row[i]) * p.C + col0 + n * 8 + 2 * t;
        const float u = sum[n][2 * i], v = sum[n][2 * i + 1];
        if constexpr (BF16) *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(p.out) + at) = __floats2bfloat162_rn(u, v);
        else *reinterpret_cast<float2*>(static_cast<float*>(p.out) + at) = make_float2(u, v);
      }
  }
}

// The warp's parts of the CTA's tiles.  Out of line, once, so that it takes no registers from the loop.
template <int BN, bool WGRAD, bool BF16>
__device__ __noinline__ void redo_tiles(const MatmulParams& p, const Shared<WGRAD>& sh, int n_tiles) {
  constexpr int CW = BN / 4;
  const int warp = threadIdx.x / kWarp, first = warp % 4 * 32;
  Walk w;
  for (int tile = blockIdx.x; tile < n_tiles; tile += gridDim.x) {
    w.at<BN, WGRAD>(p, sh, tile);
    const int col = w.col0 + (warp - kFirstEpi) / 4 * CW;
    if (first < w.rows && col < p.C)
      redo_rows<CW, WGRAD, BF16>(p, w.e, w.row0 + first, min(32, w.rows - first), col, min(CW, p.C - col), w.block0, w.blocks,
                                 (WGRAD ? int64_t(w.e) * p.R : 0) + w.row0 + first);
  }
}

template <int BN, int RB, bool WGRAD, bool BF16>
__global__ void __launch_bounds__(kMmThreads, 1)
expert_matmul_kernel(const __grid_constant__ MatmulParams p, const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                     const __grid_constant__ CUtensorMap whole_a, const __grid_constant__ CUtensorMap whole_b,
                     const __grid_constant__ CUtensorMap map_out) {
  using TL = Tile<BN, RB, WGRAD>;
  extern __shared__ uint8_t s_dyn[];
  __shared__ Shared<WGRAD> sh;
  uint8_t* ring = s_dyn + (1024 - smem_addr(s_dyn) % 1024) % 1024;
  const int warp = threadIdx.x / kWarp, lane = threadIdx.x % kWarp;

  if (warp == 0) {
    if (lane == 0) {
      for (const CUtensorMap* m : {&map_a, &map_b, &whole_a, &whole_b})
        asm volatile("prefetch.tensormap [%0];" :: "l"(m) : "memory");
      for (int i = 0; i < TL::kStages; ++i) {
        mbar_init(&sh.full[i], 1 + p.extra);
        mbar_init(&sh.done[i], 1);
      }
      for (int i = 0; i < TL::kBufs; ++i) mbar_init(&sh.tempty[i], kEpiWarps);
      if constexpr (WGRAD)
        for (int i = 0; i < kScaleSlots; ++i) mbar_init(&sh.scales[i], 1);
      mbar_init(&sh.drain, 1);
      mbar_fence_init();
      // an error that the host has not read yet: write nothing
      sh.redo = 0;
      sh.abort = *static_cast<volatile int*>(&g_mm_errors) != 0;
    }
  } else if (warp == 1) {
    tmem_alloc(&sh.tmem);
    tc_fence_before();
  } else if (warp == 2) {                                        // tiles and blocks before each expert
    const int ct = (p.C + BN - 1) / BN;
    int tiles = 0, blocks = 0;
    float sum = 0.f;                                             // of the tiles, where ranges that overlap pass an int
    for (int e0 = 0; e0 < p.E; e0 += kWarp) {
      int t = 0, b = 0;
      if (e0 + lane < p.E) {
        if constexpr (WGRAD) {
          b = int((max(int64_t(p.kept[e0 + lane]), int64_t(0)) + kBK - 1) / kBK);
        } else {
          int64_t start, n;
          expert_rows(p, e0 + lane, &start, &n);
          sh.block[e0 + lane] = int(start);
          sh.count[e0 + lane] = int(n);
          t = int((n + kBM - 1) / kBM) * ct;
          sum += float(t);
        }
      }
      int ti = t, bi = b;
#pragma unroll
      for (int off = 1; off < kWarp; off <<= 1) {
        const int to = __shfl_up_sync(kFull, ti, off), bo = __shfl_up_sync(kFull, bi, off);
        if (lane >= off) {
          ti += to;
          bi += bo;
        }
      }
      if (e0 + lane < p.E) {
        if constexpr (!WGRAD) sh.first[e0 + lane] = tiles + ti - t;
        else sh.block[e0 + lane] = int(min(int64_t(blocks) + bi - b, p.blocks));   // inside the operands
      }
      tiles += __shfl_sync(kFull, ti, kWarp - 1);
      blocks = int(min(int64_t(blocks) + __shfl_sync(kFull, bi, kWarp - 1), p.blocks));
    }
    if (warp_sum_f(sum) > 2e9f) tiles = 0;                       // such offsets give nothing
    if (lane == 0) {
      if constexpr (!WGRAD) sh.first[p.E] = tiles;
      else sh.block[p.E] = blocks;
    }
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  int n_tiles = 0;
  if (sh.abort == 0) {
    if constexpr (WGRAD) n_tiles = p.E * ((p.R + kBM - 1) / kBM) * ((p.C + BN - 1) / BN);
    else n_tiles = sh.first[p.E];
  }
  __syncthreads();                                               // every thread has seen abort before a role sets it

  // The epilogue's sums want more registers than an even split gives: of the
  // launch's 640 x 96, the first four warps keep 32 a thread and the others take 112.
  static_assert(kFirstEpi * 32 + kEpiWarps * 112 <= (kFirstEpi + kEpiWarps) * 96, "registers of the launch");
  if (warp < kFirstEpi) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
    // Both roles run as whole warps, of which one elected thread issues: their
    // addresses and descriptors then stay in uniform registers.  (With one thread
    // in a branch of its own a block took 430 ns however little it copied.)
    if (warp == 0) {
      // ---- producer: one stage per block ----
      int s = 0, issued = 0, q = 0;
      uint32_t phase = 0;
      bool ok = true;
      Walk w;
      for (int tile = blockIdx.x; tile < n_tiles && ok; tile += gridDim.x) {
        w.at<BN, WGRAD>(p, sh, tile);
        const int na = boxes(w.rows), nb = boxes(w.cols);
        const int b_row = WGRAD ? w.col0 : w.e * p.C + w.col0;
        for (int b = 0; b < w.blocks; b += RB) {
          const int now = RB == 1 ? 1 : min(RB, w.blocks - b);
          ok = __all_sync(kFull, mm_wait(sh, p, &sh.done[s], phase ^ 1u));
          if (!ok) break;
          if (elect_one()) {
            // A block's scales go where those of the block six before were: the stage that is
            // free held the block three before, whose product was formed when the one five
            // before had been read.
            if constexpr (WGRAD) {
              static_assert(kScaleSlots > TL::kStages + TL::kBufs, "scales that are still read");
              const int64_t blk = w.block0 + b;
              mbar_arrive_expect_tx(&sh.scales[q], uint32_t(w.rows + w.cols) * 4u);
              bulk_load(sh.scale[q], p.a_scale + blk * p.R + w.r0, uint32_t(w.rows) * 4u, &sh.scales[q]);
              bulk_load(sh.scale[q] + kBM, p.b_scale + blk * p.C + w.col0, uint32_t(w.cols) * 4u, &sh.scales[q]);
            }
            uint64_t* bar = &sh.full[s];
            mbar_arrive_expect_tx(bar, uint32_t((na + nb) * now * kBox * kBK));
            for (int j = 0; j < now; ++j) {
              uint8_t* sa = ring + s * TL::kStageBytes + j * TL::kBlockBytes;
              uint8_t* sb = sa + kBM * kBK;
              const int x = (w.block0 + b + j) * kBK;
              if (na == kBM / kBox) tma_2d(sa, &whole_a, x, w.row0, bar);
              else for (int i = 0; i < na; ++i) tma_2d(sa + i * kBox * kBK, &map_a, x, w.row0 + i * kBox, bar);
              if (nb == BN / kBox) tma_2d(sb, &whole_b, x, b_row, bar);
              else for (int i = 0; i < nb; ++i) tma_2d(sb + i * kBox * kBK, &map_b, x, b_row + i * kBox, bar);
            }
          }
          __syncwarp();
          ++issued;
          if (++q == kScaleSlots) q = 0;
          if (++s == TL::kStages) {
            s = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) {                                                 // copies in flight land before shared memory goes
        for (int i = 0; i < TL::kStages && i < issued; ++i) {
          const int back = issued - 1 - i;
          mbar_wait(&sh.full[back % TL::kStages], uint32_t(back / TL::kStages) & 1u, p.timeout_ns);
          if constexpr (WGRAD) mbar_wait(&sh.scales[back % kScaleSlots], uint32_t(back / kScaleSlots) & 1u, p.timeout_ns);
        }
      }
    } else if (warp == 1) {
      // ---- MMA issuer ----
      // D fp32, A and B e4m3, both K-major, N = BN, M = 128
      constexpr uint32_t idesc = (1u << 4) | uint32_t(BN / 8) << 17 | uint32_t(kBM / 16) << 24;
      const uint64_t desc0 = smem_desc(ring);
      int s = 0, t = 0;
      uint32_t phase = 0, tphase = 0;
      bool ok = true;
      Walk w;
      for (int tile = blockIdx.x; tile < n_tiles && ok; tile += gridDim.x) {
        w.at<BN, WGRAD>(p, sh, tile);
        for (int b = 0; b < w.blocks; b += RB) {
          ok = __all_sync(kFull, mm_wait(sh, p, &sh.full[s], phase, &sh.tempty[t], tphase ^ 1u));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < RB; ++j) {
              if (j > 0 && b + j >= w.blocks) break;
              const uint64_t da = desc0 + uint64_t((s * TL::kStageBytes + j * TL::kBlockBytes) >> 4), db = da + (kBM * kBK >> 4);
#pragma unroll
              for (int k = 0; k < kBK / 32; ++k)                 // 32 bytes along the row: 2 units of 16
                tc_mma_f8(tmem + (t * RB + j) * BN, da + k * 2, db + k * 2, idesc, k > 0);
            }
            tc_commit(&sh.done[s]);                              // the stage is free, and the product there
          }
          __syncwarp();
          if (++s == TL::kStages) {
            s = 0;
            phase ^= 1u;
          }
          if (++t == TL::kBufs) {
            t = 0;
            tphase ^= 1u;
          }
        }
      }
      if (!ok) {                                                 // products in flight end before tensor memory goes
        if (elect_one()) tc_commit(&sh.drain);
        __syncwarp();
        mbar_wait(&sh.drain, 0, p.timeout_ns);
      }
    } else if (WGRAD && warp == 2) {
      // ---- the scales of the tiles' rows, from global memory: a look at them in the
      // epilogue costs it 227 us instead of 220.  (In the product it is the epilogue's that
      // is free, and this one's that costs: 525 us instead of 515.) ----
      bool plain = true;
      Walk w;
      for (int tile = blockIdx.x; tile < n_tiles; tile += gridDim.x) {
        w.at<BN, WGRAD>(p, sh, tile);
        if (lane * 4 >= w.rows) continue;                        // R is a multiple of 16, the array 16-byte aligned
        const float* s = p.a_scale + int64_t(w.block0) * p.R + w.r0 + lane * 4;
        for (int b = 0; b < w.blocks; ++b, s += p.R) {
          const float4 v = *reinterpret_cast<const float4*>(s);
          plain = plain && plain_pair<true>(v.x, 1.f) && plain_pair<true>(v.y, 1.f) && plain_pair<true>(v.z, 1.f) && plain_pair<true>(v.w, 1.f);
        }
      }
      if (!plain) sh.redo = 1;
      __syncwarp();
      scales_known();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
    // ---- epilogue: rows 32 * quad + lane, kCols columns ----
    constexpr int CW = TL::kCols;
    const int quad = warp % 4, cg = (warp - kFirstEpi) / 4, row = quad * 32 + lane;
    const int kblocks = (p.K + kBK - 1) / kBK, cblocks = (p.C + kBK - 1) / kBK;
    int s = 0, t = 0, q = 0;
    uint32_t phase = 0, qphase = 0;
    bool ok = true;
    Walk w;
    int c0 = 0;                                                  // the warp's first column of out
    bool busy = false, live = false;                             // whether the warp has anything to add, the lane a row
    bool plain = true;                                           // product: all scales that the lane has met
    const float *pa = nullptr, *pb = nullptr;
    float sa[RB], sb[RB];
#pragma unroll
    for (int j = 0; j < RB; ++j) sa[j] = sb[j] = 1.f;
    const auto fetch = [&](int b) {                              // product: the scales of a stage's blocks
#pragma unroll
      for (int j = 0; j < RB; ++j) {
        if (busy && b + j < w.blocks) {
          sa[j] = live ? *pa : 1.f;
          sb[j] = *pb;
        }
        pa += p.M;
        pb += 1;
      }
    };
    const auto begin = [&](int tile) {                           // a tile's place and its first scales
      w.at<BN, WGRAD>(p, sh, tile);
      c0 = w.col0 + cg * CW;
      busy = quad * 32 < w.rows && c0 < p.C;                     // warp-uniform
      live = row < w.rows;
      if constexpr (!WGRAD) {
        pa = p.a_scale + w.row0 + row;
        pb = p.b_scale + (int64_t(w.e) * cblocks + c0 / kBK) * kblocks;
        fetch(0);
      }
    };
    if (!WGRAD && int(blockIdx.x) < n_tiles) begin(blockIdx.x);
    for (int tile = blockIdx.x; tile < n_tiles; tile += gridDim.x) {
      if constexpr (WGRAD) begin(tile);
      float2 acc[CW / 2];
#pragma unroll
      for (int i = 0; i < CW / 2; ++i) acc[i] = make_float2(0.f, 0.f);
      for (int b = 0; b < w.blocks; b += RB) {
        float scale[RB];
        if constexpr (!WGRAD) {
#pragma unroll
          for (int j = 0; j < RB; ++j) {
            scale[j] = sa[j] * sb[j];
            plain = plain && plain_scale<false>(scale[j]);
          }
          // The next scales, in front of the wait (508 us against 535 at 65,536 rows).
          fetch(b + RB);
        }
        ok = __all_sync(kFull, mm_wait(sh, p, &sh.done[s], phase, WGRAD ? &sh.scales[q] : nullptr, qphase));   // one answer for the warp
        if (!ok) break;
        tc_fence_after();
        // The buffer is free as soon as its last columns have been read.
        const auto release = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.tempty[t]);
        };
        if (WGRAD && busy) {
          // Fragments: a lane needs 16 scales of columns and 4 of rows, instead of the 64 of
          // columns that a row a lane takes (219 us against 225 at 32,836 rows).
          const float* f_row = &sh.scale[WGRAD ? q : 0][quad * 32 + lane / 4];
          const float* f_col = &sh.scale[WGRAD ? q : 0][kBM + cg * CW + lane % 4 * 2];
          const uint32_t addr = tmem + t * BN + cg * CW + (uint32_t(quad * 32) << 16);
          const float row_scale[4] = {f_row[0], f_row[8], f_row[16], f_row[24]};   // one behind the last row is not stored
#pragma unroll
          for (int c = 0; c < CW; c += 32) {
            float2 f[4];
#pragma unroll
            for (int n = 0; n < 4; ++n) f[n] = *reinterpret_cast<const float2*>(&f_col[c + 8 * n]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {                        // rows 16 h and following
              uint32_t u[16];
              tmem_ld_16x32(addr + c + (uint32_t(16 * h) << 16), u);
              tmem_ld_wait(u);
              if (c + 32 == CW && h == 1) release();
#pragma unroll
              for (int i = 0; i < 8; ++i) {                      // acc: (columns / 32, rows / 16, columns / 8, rows / 8)
                const float r = row_scale[2 * h + i % 2];
                const float2 x = make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
                float2& a = acc[c / 2 + 8 * h + i];
                a = fma2(mul2(x, make_float2(r, r)), f[i / 2], a);
              }
            }
          }
        } else if (busy) {
#pragma unroll
          for (int j = 0; j < RB; ++j) {
            const bool last = j + 1 == RB || b + j + 1 >= w.blocks;
            const uint32_t addr = tmem + (t * RB + j) * BN + cg * CW + (uint32_t(quad * 32) << 16);
            const float2 s2 = make_float2(scale[j], scale[j]);
#pragma unroll
            for (int c = 0; c < CW; c += 16) {
              uint32_t u[16];
              tmem_ld16(addr + c, u);
              tmem_ld_wait(u);
              if (last && c + 16 == CW) release();
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                const float2 x = make_float2(__uint_as_float(u[i]), __uint_as_float(u[i + 1]));
                const float2 y = make_float2(__uint_as_float(u[i + 2]), __uint_as_float(u[i + 3]));
                acc[(c + i) / 2] = fma2(x, s2, acc[(c + i) / 2]);
                acc[(c + i) / 2 + 1] = fma2(y, s2, acc[(c + i) / 2 + 1]);
              }
            }
            if (last) break;
          }
        } else {
          release();
        }
        if (++s == TL::kStages) {
          s = 0;
          phase ^= 1u;
        }
        if (++t == TL::kBufs) t = 0;
        if (++q == kScaleSlots) {
          q = 0;
          qphase ^= 1u;
        }
      }
      if (!ok) break;
      // The next tile's first scales are on their way while this one is stored.
      const bool store = busy;
      const int to_c0 = c0, to_rows = w.rows, to_row0 = WGRAD ? w.r0 : w.row0, to_e = w.e;
      if (!WGRAD && tile + int(gridDim.x) < n_tiles) begin(tile + gridDim.x);
      if (!store) continue;
      if constexpr (WGRAD) {
        // 32 x 32 values at a time through the warp's part of shared memory, whose
        // 128-byte rows hold their 16-byte pieces in the tensor copy's swizzled order.
        // (Two pieces of 16 rows, so that one is written while the other leaves: 226 us
        // against 219.)
        uint8_t* stage = ring + TL::kStages * TL::kStageBytes + (warp - kFirstEpi) * kWarpOutBytes;
#pragma unroll
        for (int c = 0; c < CW; c += kOutCols) {
          tma_store_read();                                      // the last copy has read it (lane 0 issued it)
          __syncwarp();
#pragma unroll
          for (int i = 0; i < kOutCols / 2; ++i) {               // as acc: rows 16 (i / 8) + 8 (i % 2) + lane / 4
            const int to_row = i / 8 * 16 + i % 2 * 8 + lane / 4, piece = i / 2 % 4 * 2 + lane % 4 / 2;
            *reinterpret_cast<float2*>(stage + to_row * 128 + (piece ^ lane / 4) * 16 + lane % 2 * 8) = acc[c / 2 + i];
          }
          async_proxy_fence();
          __syncwarp();
          if (lane == 0) {
            if (to_c0 + c < p.C) tma_store_3d(stage, &map_out, to_c0 + c, to_row0 + quad * 32, to_e);
            tma_store_commit();
          }
        }
      } else {
        // Pieces of 16 bytes, NP of which are turned among NP lanes at a time.
        constexpr int kPer = BF16 ? 8 : 4, NP = CW / kPer < 8 ? CW / kPer : 8;
#pragma unroll
        for (int h = 0; h < CW; h += NP * kPer) {
          uint4 v[NP];
#pragma unroll
          for (int i = 0; i < NP; ++i) {
            const float2* a = &acc[(h + i * kPer) / 2];
            if constexpr (BF16) {
              uint32_t b2[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const __nv_bfloat162 q = __floats2bfloat162_rn(a[j].x, a[j].y);
                b2[j] = *reinterpret_cast<const uint32_t*>(&q);
              }
              v[i] = make_uint4(b2[0], b2[1], b2[2], b2[3]);
            } else {
              v[i] = make_uint4(__float_as_uint(a[0].x), __float_as_uint(a[0].y), __float_as_uint(a[1].x), __float_as_uint(a[1].y));
            }
          }
          turn<NP>(v, lane);
          const int c = to_c0 + h + lane % NP * kPer;               // C is a multiple of 16: a piece is whole
#pragma unroll
          for (int r = 0; r < NP; ++r) {
            const int to = quad * 32 + lane / NP * NP + r;
            if (to < to_rows && c < p.C)
              *reinterpret_cast<uint4*>(static_cast<char*>(p.out) + (int64_t(to_row0 + to) * p.C + c) * (BF16 ? 2 : 4)) = v[r];
          }
        }
      }
    }
    if constexpr (WGRAD) {
      tma_store_done();                                          // shared memory is read, and the results are there
      scales_known();
      plain = sh.redo == 0;
    }
    __syncwarp();
    if (ok && !__all_sync(kFull, plain)) redo_tiles<BN, WGRAD, BF16>(p, sh, n_tiles);
  }
  __syncwarp();                                                  // the roles' single threads are back
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_free(tmem);
}

// ---- host ------------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      f = nullptr;
    return reinterpret_cast<EncodeFn>(f);
  }();
  return fn;
}

// A row-major [rows, cols] byte matrix read in boxes of `box` rows by 128
// columns; what lies outside reads as zero.
bool make_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint32_t box) {
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols};
  const cuuint32_t boxes[2] = {kBK, box}, ones[2] = {1, 1};
  return encode_fn() != nullptr &&
         encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, boxes, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// fp32 results [E, R, C] written in boxes of 32 rows by 32 columns.
bool make_out_map(CUtensorMap* map, void* base, uint64_t E, uint64_t R, uint64_t C) {
  const cuuint64_t dims[3] = {C, R, E}, strides[2] = {C * 4, R * C * 4};
  const cuuint32_t boxes[3] = {kOutCols, 32, 1}, ones[3] = {1, 1, 1};
  return encode_fn() != nullptr &&
         encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, int RB, bool WGRAD, bool BF16>
cudaError_t launch(const MatmulParams& p, int sms, const char** error, cudaStream_t stream) {
  using TL = Tile<BN, RB, WGRAD>;
  CUtensorMap ma, mb, wa, wb, mo = {};
  const uint64_t cols = WGRAD ? uint64_t(p.blocks) * kBK : uint64_t(p.K);
  const uint64_t rows_a = WGRAD ? uint64_t(p.R) : uint64_t(p.M), rows_b = WGRAD ? uint64_t(p.C) : uint64_t(p.E) * p.C;
  if (!make_map(&ma, p.a, rows_a, cols, kBox) || !make_map(&mb, p.b, rows_b, cols, kBox) ||
      !make_map(&wa, p.a, rows_a, cols, kBM) || !make_map(&wb, p.b, rows_b, cols, BN) ||
      (WGRAD && !make_out_map(&mo, p.out, uint64_t(p.E), uint64_t(p.R), uint64_t(p.C)))) {
    *error = "cuTensorMapEncodeTiled refused an operand";
    return cudaErrorUnknown;
  }
  constexpr size_t smem = size_t(TL::kStages) * TL::kStageBytes + TL::kOutBytes + 1024;
  static_assert(TL::kStages <= 8 && TL::kBufs <= 8 && TL::kBufs >= 2 && sizeof(Shared<WGRAD>) + smem <= 232448, "shared memory of one CTA");
  static_assert(BN % kBox == 0 && TL::kStageBytes % 1024 == 0, "whole boxes, swizzle atoms aligned");
  const auto kernel = expert_matmul_kernel<BN, RB, WGRAD, BF16>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  // At most this many tiles: every expert's last row tile may be ragged.
  const int64_t ct = (p.C + BN - 1) / BN;
  int64_t rt = WGRAD ? int64_t(p.E) * ((p.R + kBM - 1) / kBM) : p.M / kBM + p.E;
  if (!WGRAD && rt > p.M) rt = p.M;
  kernel<<<unsigned(rt * ct < sms ? rt * ct : sms), kMmThreads, smem, stream>>>(p, ma, mb, wa, wb, mo);
  return cudaGetLastError();
}

}  // namespace

cudaError_t expert_matmul_errors(int* bits, cudaStream_t stream) {
  static std::atomic<unsigned> calls{0};
  const unsigned place = calls.fetch_add(1, std::memory_order_relaxed) % kReads;
  take_errors_kernel<<<1, 1, 0, stream>>>(place);
  cudaError_t e = cudaGetLastError();
  void* word = nullptr;
  if (e == cudaSuccess) e = cudaGetSymbolAddress(&word, g_mm_read);
  if (e == cudaSuccess) e = cudaMemcpyAsync(bits, static_cast<int*>(word) + place, sizeof(int), cudaMemcpyDeviceToHost, stream);
  const cudaError_t done = cudaStreamSynchronize(stream);
  return e == cudaSuccess ? done : e;
}

cudaError_t launch_expert_matmul(const MatmulParams& p, int sms, const char** error, cudaStream_t stream) {
  if (p.wgrad) return launch<256, 1, true, false>(p, sms, error, stream);
  // Tiles of 128 columns, two blocks a stage, up to 200 rows an expert: they spread few rows'
  // weights over more SMs (rows x experts, 4096 -> 2048: 87 x 64 109 us against 138, 175 x 64
  // 150 against 158).  Beyond, 256 columns, which halve the reads of the rows (1024 x 64 490
  // against 559), unless the narrow tiles leave the SMs less idle behind the last one: a
  // narrow one takes some 3/5 of a wide one's time, and an expert's last row tile counts
  // half (500 x 4, 1024 -> 1024: 8.5 us against 11.2; 300 x 1, 4096 -> 4096: 14 against 21;
  // but 750 x 8, 1424 -> 1040: 28 against 24, and 600 x 16, 4096 -> 2048: 96 against 93).
  const int64_t row_tiles = (p.M + (p.E > 1 ? 64 * int64_t(p.E) : 0) + kBM - 1) / kBM;
  const auto rounds = [&](int columns) { return (row_tiles * ((p.C + columns - 1) / columns) + sms - 1) / sms; };
  const bool narrow = p.M <= int64_t(p.E) * 200 || rounds(128) * 3 < rounds(256) * 5;
  if (p.out_bf16)
    return narrow ? launch<128, 2, false, true>(p, sms, error, stream) : launch<256, 1, false, true>(p, sms, error, stream);
  return narrow ? launch<128, 2, false, false>(p, sms, error, stream) : launch<256, 1, false, false>(p, sms, error, stream);
}

}  // namespace moe
