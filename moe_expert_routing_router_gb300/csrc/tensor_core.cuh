// What the kernels on the fifth-generation tensor cores share: instructions on tensor
// memory, tensor copies, matrix descriptors, their bounded wait, and the tensor maps of
// operands in rows of 128 bytes.
#pragma once

#include "device_common.cuh"

#include <cuda.h>

namespace moe {
namespace {

constexpr int kTmemCols = 512;                // of an SM: its one CTA takes all
constexpr int kRowBytes = 128;                // of an operand's row in a stage

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

// Bounded wait that every role of a CTA uses: false once it, or another role's, ran out,
// which sets `abort` in shared memory and the pipeline's bit in the device's error word.
// Time is counted in SM cycles (at most about two a nanosecond), whose counter is
// read in a few cycles, and only after some waits have failed.
// With a second barrier, both are tested at once: a test takes some 100 cycles.
__device__ __forceinline__ bool pipeline_wait(int* abort, int* errors, uint64_t timeout_ns, uint64_t* bar, uint32_t parity,
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
    if (*static_cast<volatile int*>(abort) != 0) return false;
    if (clock64() - t0 > 2 * (long long)(timeout_ns)) {
      *static_cast<volatile int*>(abort) = 1;
      atomicOr(errors, kErrPipelineTimeout);
      return false;
    }
  }
  return true;
}

// The rows of expert e: their place and number, whatever the arrays hold, inside [0, M).
template <class P>
__device__ __forceinline__ void expert_rows(const P& p, int e, int64_t* start, int64_t* n) {
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

// ---- host ------------------------------------------------------------------------
using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encode_fn() {
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
// bytes; what lies outside reads as zero.
inline bool make_map(CUtensorMap* map, const void* base, uint64_t rows, uint64_t cols, uint32_t box) {
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols};
  const cuuint32_t boxes[2] = {kRowBytes, box}, ones[2] = {1, 1};
  return encode_fn() != nullptr &&
         encode_fn()(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, boxes, ones,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace moe
