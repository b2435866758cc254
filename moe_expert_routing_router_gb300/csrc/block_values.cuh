// Pieces of rows that a lane holds while its block's maximum is found, and the
// scales and codes of the two block formats (e4m3 by 128, 4 bits by 32): shared by
// the kernels that write or read quantised rows.
#pragma once

#include "device_common.cuh"
#include "quantize.h"

namespace moe {
namespace {

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

// ---- 4-bit blocks of 32 ------------------------------------------------------------
// A scale's code n stands for 2^(n - 127).  max|x| = m * 2^x, 1 <= m < 2, and the largest
// code is 6 = 1.5 * 2^2: the exponent is x - 2, one more where m > 1.5 (the addition
// carries), and at least -126.  127 for a block of zeros, 255 (NaN) where it is not finite.
struct Fp4Scale {
  uint32_t code;
  float inv;
};
__device__ __forceinline__ Fp4Scale fp4_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int n = max(int((b + 0x3fffffu) >> 23) - 2, 1);
  Fp4Scale s = {uint32_t(n), __uint_as_float(uint32_t(254 - n) << 23)};
  if (b == 0u) s = {127u, 1.f};
  if (b >= 0x7f800000u) s = {255u, 0.f};
  return s;
}

// Eight values as codes, the first in the lowest four bits; to nearest, ties to even, at most 6 in size.
__device__ __forceinline__ uint32_t fp4_pack8(float2 a, float2 b, float2 c, float2 d) {
  uint32_t q;
  asm("{\n\t.reg .b8 p, q, r, s;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 p, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 q, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 r, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 s, %8, %7;\n\t"
      "mov.b32 %0, {p, q, r, s};\n\t}"
      : "=r"(q) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y), "f"(d.x), "f"(d.y));
  return q;
}

// Eight codes as fp16, which holds their values.
__device__ __forceinline__ void fp4_unpack8(uint32_t codes, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 p, q, r, s;\n\tmov.b32 {p, q, r, s}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, p;\n\tcvt.rn.f16x2.e2m1x2 %1, q;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, r;\n\tcvt.rn.f16x2.e2m1x2 %3, s;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(codes));
}

// What a scale's code stands for.
__device__ __forceinline__ float fp4_scale_value(uint32_t code) {
  return code == 255u ? __uint_as_float(0x7fc00000u) : code == 0u ? 0x1p-127f : __uint_as_float(code << 23);
}

// The scale codes of the four blocks of 128 values that eight lanes hold, 16 each; `code` is
// that of the lane's own block.  Every lane gets the word.
__device__ __forceinline__ uint32_t fp4_scale_word(uint32_t code, int l) {
  uint32_t w = code << (l / 2 * 8);
  w |= __shfl_xor_sync(kFull, w, 2);
  return w | __shfl_xor_sync(kFull, w, 4);
}

}  // namespace
}  // namespace moe
