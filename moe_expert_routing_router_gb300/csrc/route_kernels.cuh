// Scored, group-limited routing and its gradient.
//
// Scores s = sigmoid(z) or softmax(z); an expert's choice value is s + bias
// (its logit's order without a bias); a group of experts is scored by its
// largest choice value or the sum of its two largest; the k largest choice
// values within the best groups are picked; gates are the picks' scores,
// renormalised over the picks if asked, times a scale.
//
// A row is worked on by 8, 16 or 32 lanes, so that a warp's steps serve up to
// four rows.  A group's experts lie in consecutive lanes and an expert's lane and
// place rise with its index, so that ties go to the lowest lane and place, and a
// group's score is a butterfly over its lanes.
//
// Picks are integers, decided by comparing sums of exponentials.  The fast path
// compares them in fp32 and bounds what its rounding can have changed: where
// two values that decide a pick are nearer than that bound (and not equal
// because their inputs are), the warp ranks them again in double.  That is a row
// in some hundred, so the picks are those of the double-precision definition at
// fp32 cost.
#pragma once

#include "device_common.cuh"
#include "route.h"

#include <cstddef>
#include <type_traits>

namespace moe {
namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / kWarp;

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xff800000u); }
// No choice value: above and below nothing, and passed over by fmaxf.
__device__ __forceinline__ float none() { return __uint_as_float(0x7fc00000u); }

template <class Elem>
__device__ __forceinline__ float load_logit(const void* logits, int64_t at) {
  return __uint_as_float(Elem::bits(static_cast<const typename Elem::Raw*>(logits)[at]));
}

__device__ __forceinline__ float warp_max_f(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, off));
  return x;
}

// The CTAs of a cluster: how many, which one this is, a barrier of all, and the word in
// CTA r's shared memory at the place of this one's `p`.
__device__ __forceinline__ uint32_t cluster_ctas() {
  uint32_t n;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return n;
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t n;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(n));
  return n;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int cluster_load(const int* p, uint32_t r) {
  uint32_t at;
  int v;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(r));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}

// The sigmoid, relative to its own size (no cancellation on either side).
__device__ __forceinline__ float sigmoid_exact(float z) {
  const float t = expf(-fabsf(z));
  return (z >= 0.f ? 1.f : t) / (1.f + t);
}

// Eight neighbouring lanes hold the picks of one row, so that a warp finishes
// four rows at once; reductions over them.
constexpr int kPickLanes = 8;
__device__ __forceinline__ float pick_max(float x) {
#pragma unroll
  for (int off = kPickLanes / 2; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, off));
  return x;
}
__device__ __forceinline__ float pick_value(float x, int j) { return __shfl_sync(kFull, x, j, kPickLanes); }

// The picks' scores up to a common factor of the row, so that renormalised
// gates keep their digits where the scores themselves underflow.
__device__ __forceinline__ float pick_weight(float z, bool live, int softmax) {
  const float m = pick_max(live ? z : neg_inf());
  if (!live || !(z > neg_inf())) return 0.f;                    // masked or not a number: no weight
  if (softmax) return expf(z - m);
  if (m >= 0.f) return sigmoid_exact(z);
  return expf(z - m) / (1.f + expf(z));                         // every pick's sigmoid times exp(-m)
}
// Its share of the row's sum (0 where nothing is left).
__device__ __forceinline__ float pick_share(float w, int k) {
  float sum = 0.f;
  for (int j = 0; j < k; ++j) sum += pick_value(w, j);
  return sum > 0.f ? w / sum : 0.f;
}

// Doubles as integers in the same order (double comparisons share the few units
// that double arithmetic has); what is not a number ranks lowest.
__device__ __forceinline__ long long ordered(double v) {
  const long long b = __double_as_longlong(v + 0.0);
  return v == v ? b ^ (b >> 63 & 0x7fffffffffffffffll) : -0x7fffffffffffffffll - 1;
}
__device__ __forceinline__ double from_ordered(long long k) {
  return __longlong_as_double(k ^ (k >> 63 & 0x7fffffffffffffffll));
}

// A score in double: of one logit, given a softmax row's largest and its sum.
struct DoubleScore {
  int softmax;
  float m;
  double sum;
  __device__ __forceinline__ double operator()(float z) const {
    if (softmax) return exp(double(z) - double(m)) / sum;
    const double t = exp(-fabs(double(z)));                      // never above 1: small scores stay what they are
    return (z >= 0.f ? 1.0 : t) / (1.0 + t);
  }
};
template <class Elem>
__device__ __noinline__ DoubleScore route_double_score(const RouteParams& p, int64_t row, int lane) {
  DoubleScore s = {p.softmax, neg_inf(), 0.0};
  if (!p.softmax) return s;
  constexpr int kAtOnce = 4;                                     // loads in flight
  float z[kAtOnce];
  const auto load = [&](int e0) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      z[i] = e0 + i * kWarp + lane < p.E ? load_logit<Elem>(p.logits, row * p.E + e0 + i * kWarp + lane) : neg_inf();
  };
  for (int e0 = 0; e0 < p.E; e0 += kAtOnce * kWarp) {
    load(e0);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) s.m = fmaxf(s.m, z[i]);
  }
  s.m = warp_max_f(s.m);
  for (int e0 = 0; e0 < p.E; e0 += kAtOnce * kWarp) {
    load(e0);
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (z[i] > neg_inf()) s.sum += exp(double(z[i]) - double(s.m));
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s.sum += __shfl_xor_sync(kFull, s.sum, off);
  return s;
}

// ---------------------------------------------------------------------------
// The row ranked in double: the definition, by all lanes of the warp.  Lane j
// gets pick j.  `bias` and the row are read again (they are in the caches).
// ---------------------------------------------------------------------------
template <class Elem>
__device__ __noinline__ int route_row_double(const RouteParams& p, int64_t row, int lane, DoubleScore score_of) {
  long long c[64];                                               // choice values of the lane's experts
  const int g = lane / p.L, base = g * p.gs + (lane % p.L) * p.chunk;
  const int n = g < p.G ? max(0, min(p.chunk, p.gs - (lane % p.L) * p.chunk)) : 0;
  const long long masked = ordered(double(neg_inf()));
  long long a = masked, b = masked;                              // the two largest of the lane, then of the group
  unsigned long long gone = 0;
  for (int i = 0; i < n; ++i) {
    const float z = load_logit<Elem>(p.logits, row * p.E + base + i);
    long long v = masked, order = masked;
    if (z > neg_inf()) {
      double s = 0.0;
      if (p.bias != nullptr || p.top2) {
        s = score_of(z);
        if (p.bias != nullptr) s += double(p.bias[base + i]);
      }
      v = ordered(s);
      order = p.bias != nullptr ? v : ordered(double(z));
    }
    const long long u = p.top2 ? v : order;
    b = max(b, min(a, u));
    a = max(a, u);
    c[i] = order;
  }
  if (p.G > 1) {
    for (int off = 1; off < p.L; off <<= 1) {
      const long long a2 = __shfl_xor_sync(kFull, a, off), b2 = __shfl_xor_sync(kFull, b, off);
      b = max(min(a, a2), max(b, b2));
      a = max(a, a2);
    }
    const long long score = p.top2 && b > masked ? ordered(from_ordered(a) + from_ordered(b)) : a;
    int rank = 0;
    for (int o = 0; o < p.G; ++o) {
      const long long other = __shfl_sync(kFull, score, o * p.L);
      rank += other > score || (other == score && o < g);
    }
    if (rank >= p.keep) gone = ~0ull;
  }
  int mine = 0;
  for (int j = 0; j < p.k; ++j) {
    long long v = masked;
    int e = 0x7fffffff;
    for (int i = 0; i < n; ++i)
      if (!(gone >> i & 1) && (e == 0x7fffffff || c[i] > v)) {
        v = c[i];
        e = base + i;
      }
    for (int off = 16; off > 0; off >>= 1) {
      const long long v2 = __shfl_xor_sync(kFull, v, off);
      const int e2 = __shfl_xor_sync(kFull, e, off);
      if (e2 != 0x7fffffff && (e == 0x7fffffff || v2 > v || (v2 == v && e2 < e))) {
        v = v2;
        e = e2;
      }
    }
    if (e >= base && e < base + n) gone |= 1ull << (e - base);
    if (lane == j) mine = e;
  }
  return mine;
}

// The choice value of expert e in fp32 (its error within tol / 2), -infinity if masked.
template <class Elem>
__device__ __forceinline__ float route_fast_choice(const RouteParams& p, int64_t row, int e, const DoubleScore& score_of, float inv) {
  const float z = load_logit<Elem>(p.logits, row * p.E + e);
  const float s = score_of.softmax ? ex2_approx((z - score_of.m) * kLog2e) * inv : rcp_approx(1.f + ex2_approx(z * -kLog2e));
  return z > neg_inf() ? s + (p.bias != nullptr ? p.bias[e] : 0.f) : neg_inf();
}

// The experts of the lanes' groups whose choice values reach the lane's bound: how many,
// and in `list` (32 ints of shared memory) up to 32 of them.
template <class Elem>
__device__ __forceinline__ int route_candidates(const RouteParams& p, int64_t row, int lane, float reach, bool taken, int* list,
                                                const DoubleScore& score_of, float inv) {
  const int g = lane / p.L, base = g * p.gs + (lane % p.L) * p.chunk;
  const int n = g < p.G && taken ? max(0, min(p.chunk, p.gs - (lane % p.L) * p.chunk)) : 0;
  int total = 0;
  for (int i = 0; i < p.chunk; ++i) {
    const float v = i < n ? route_fast_choice<Elem>(p, row, base + i, score_of, inv) : neg_inf();
    const bool in = v > neg_inf() && !(v < reach);               // a bound of -infinity: every expert that is not masked
    const unsigned m = __ballot_sync(kFull, in);
    const int at = total + __popc(m & ((1u << lane) - 1u));
    if (in && at < kWarp) list[at] = base + i;
    total += __popc(m);
  }
  __syncwarp();
  return total;
}

// ---------------------------------------------------------------------------
// Whether the row's best groups in double are those that fp32 has taken
// (`kept`: bit g << tshift for group g).  Only the experts that can be among a
// group's two largest are evaluated, one a lane; false where there are more than
// 32 of them.  `list`: 32 ints of shared memory.
// ---------------------------------------------------------------------------
template <class Elem>
__device__ __noinline__ bool route_groups_hold(const RouteParams& p, int64_t row, int lane, float tol, unsigned kept, int* list, DoubleScore score_of) {
  const float inv = float(1.0 / score_of.sum);                   // softmax
  const int g = lane / p.L, base = g * p.gs + (lane % p.L) * p.chunk;
  const int n = g < p.G ? max(0, min(p.chunk, p.gs - (lane % p.L) * p.chunk)) : 0;
  float a = neg_inf(), b = neg_inf();
  for (int i = 0; i < n; ++i) {
    const float v = route_fast_choice<Elem>(p, row, base + i, score_of, inv);
    b = fmaxf(b, fminf(a, v));
    a = fmaxf(a, v);
  }
  for (int off = 1; off < p.L; off <<= 1) {
    const float a2 = __shfl_xor_sync(kFull, a, off), b2 = __shfl_xor_sync(kFull, b, off);
    b = fmaxf(fminf(a, a2), fmaxf(b, b2));
    a = fmaxf(a, a2);
  }
  const float last = p.top2 ? b : a, reach = last - (tol + 2.4e-7f * fabsf(last));
  const int total = route_candidates<Elem>(p, row, lane, reach, true, list, score_of, inv);
  if (total > kWarp) return false;
  const long long masked = ordered(double(neg_inf()));
  const int e = lane < total ? list[lane] : 0, of = lane < total ? e / p.gs : -1;
  long long v = masked;
  if (lane < total)
    v = ordered(score_of(load_logit<Elem>(p.logits, row * p.E + e)) + (p.bias != nullptr ? double(p.bias[e]) : 0.0));
  long long a2 = masked, b2 = masked;                            // of group `lane`
  for (int o = 0; o < total; ++o) {
    const long long w = __shfl_sync(kFull, v, o);
    if (__shfl_sync(kFull, of, o) == lane) {
      b2 = max(b2, min(a2, w));
      a2 = max(a2, w);
    }
  }
  const long long score = p.top2 && b2 > masked ? ordered(from_ordered(a2) + from_ordered(b2)) : a2;
  int rank = 0;
  for (int o = 0; o < p.G; ++o) {
    const long long other = __shfl_sync(kFull, score, o);
    rank += other > score || (other == score && o < lane);
  }
  return __all_sync(kFull, lane >= p.G || (rank < p.keep) == ((kept >> ((lane << p.tshift) & 31) & 1u) != 0u));
}

// ---------------------------------------------------------------------------
// The picks of a row where values that decide them are next to one another
// (`close`), or where its groups' scores are (`unsure`).  Lane j holds the j-th
// largest choice value and its expert, the k picks and two more.  (A whole row in
// double takes some 40 us, its candidates a few: 2048 x 384 softmax with a bias 57 us
// with the whole rows, 22 with the candidates.)
// ---------------------------------------------------------------------------
template <class Elem>
__device__ __noinline__ int route_settle(const RouteParams& p, int64_t row, int lane, float c, int ce, int rounds, float tol,
                                         bool close, bool unsure, unsigned kept, int* list) {
  const DoubleScore score_of = route_double_score<Elem>(p, row, lane);
  if (unsure && !route_groups_hold<Elem>(p, row, lane, tol, kept, list, score_of)) return route_row_double<Elem>(p, row, lane, score_of);
  if (!close) return ce;
  const bool there = lane < rounds && c == c;
  const float zc = there ? load_logit<Elem>(p.logits, row * p.E + ce) : neg_inf();
  const float bc = there && p.bias != nullptr ? p.bias[ce] : 0.f;
  const float c_up = __shfl_up_sync(kFull, c, 1), z_up = __shfl_up_sync(kFull, zc, 1), b_up = __shfl_up_sync(kFull, bc, 1);
  // sure all the same where the inputs are equal; but behind the last one that is held there
  // can be more
  const bool open = lane >= 1 && lane <= p.k && there && c_up - c <= tol + 2.4e-7f * fabsf(c_up) &&
                    !(zc == z_up && bc == b_up);
  const float last = __shfl_sync(kFull, c, p.k - 1);
  const bool beyond = lane == p.k + 1 && there && last - c <= tol + 2.4e-7f * fabsf(last);
  const bool any_open = __any_sync(kFull, open), any_beyond = __any_sync(kFull, beyond);
  if (any_beyond) {
    const bool taken = p.keep >= p.G || (kept >> ((lane / p.L << p.tshift) & 31) & 1u) != 0u;
    const int total = route_candidates<Elem>(p, row, lane, last - (tol + 2.4e-7f * fabsf(last)), taken, list, score_of,
                                             float(1.0 / score_of.sum));
    if (total > kWarp) return route_row_double<Elem>(p, row, lane, score_of);
    const int e = lane < total ? list[lane] : 0x7fffffff;
    const long long d = lane < total ? ordered(score_of(load_logit<Elem>(p.logits, row * p.E + e)) + double(p.bias[e])) : 0;
    int rank = 0;
    for (int o = 0; o < total; ++o) {
      const long long od = __shfl_sync(kFull, d, o);
      const int oe = __shfl_sync(kFull, e, o);
      rank += od > d || (od == d && oe < e);
    }
    int to = ce;
    for (int o = 0; o < total; ++o) {
      const int orank = __shfl_sync(kFull, rank, o), oe = __shfl_sync(kFull, e, o);
      if (orank == lane) to = oe;
    }
    return to;
  }
  if (!any_open) return ce;
  // The k + 1 largest are known as a set: one double-precision score a lane orders them.
  const bool in = there && lane <= p.k;
  const long long d = ordered(in && zc > neg_inf() ? score_of(zc) + double(bc) : double(neg_inf()));
  int rank = 0;
  for (int o = 0; o <= p.k; ++o) {
    const long long od = __shfl_sync(kFull, d, o);
    const int oe = __shfl_sync(kFull, ce, o);
    rank += __shfl_sync(kFull, int(in), o) != 0 && (od > d || (od == d && oe < ce));
  }
  int to = ce;
  for (int o = 0; o <= p.k; ++o) {
    const int orank = __shfl_sync(kFull, in ? rank : kWarp, o), oe = __shfl_sync(kFull, ce, o);
    if (orank == lane) to = oe;
  }
  return to;
}

// ---------------------------------------------------------------------------
// Forward.
//   LPR   lanes of a row; NV: experts of a lane, at least `tchunk`
//   VB    bytes per load, 16 or the element's size; 16 only with FULL: every lane has
//         NV experts or none, and rows, groups and the array are aligned
//   MODE  0: the order of the logits decides everything and gates need no sum over the
//         row; 1: sigmoid scores; 2: softmax scores
//
// Selection: the k largest of the maxima of eight experts each bound the k-th
// choice value from below; the few experts that reach the bound (lowered by what
// rounding can have done, where there is a bias) are gathered in expert order and
// ranked by counting.  Should more than 32 reach it (long ties, masked rows), the
// row's lanes take the maximum again and again instead.  The rows that hang on
// rounding are settled behind a warp's four rows, and then the gates of all of
// them are computed, a pick a lane.
// Instructions bound it.  For a row of 256 in 8 groups: 1145 with a warp a row whose
// lanes sort their experts, 728 with a warp a row and this selection, 436 with 8 lanes
// a row: 131,072 rows of bf16 in 82 us (0.9 TB/s), where the bytes alone would take 11.
// Experts that do not fill their lanes are loaded one at a time and computed as if they
// did: 131,072 rows of 160 in 8 groups 102 us, of 96 in 4 groups 99, of 384 without groups
// 138 (256 without groups: 69).
// ---------------------------------------------------------------------------
constexpr int kMaxRounds = 10;                                   // 8 picks and two more
constexpr int kMaxPer = kWarp / kPickLanes;                      // rows a warp finishes at once
constexpr int kCand = 32;                                        // candidates of a row

template <int LPR>
__device__ __forceinline__ float row_max(float x) {
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, off));
  return x;
}
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1) x += __shfl_xor_sync(kFull, x, off);
  return x;
}

// CTAs of an SM, which hide the loads: as many as the registers of a lane's experts leave
// room for.  (The next pass's loads issued beside this one's work cost more in registers
// than they hid: 131,072 x 256 bf16 89 us, with 2 CTAs; 79 with 3 and no such loads, 82
// with 4; fp32 93 with 2, slower with 3; 131,072 x 128 fp32 94 with 3, 87 with 4.)
template <int NV, int SIZE>
constexpr int kRouteCtas = NV <= 16 ? 4 : NV > 32 ? 1 : SIZE == 2 ? 3 : 2;

template <class Elem, int LPR, int NV, int VB, bool FULL, int MODE>
__global__ void __launch_bounds__(kRouteThreads, kRouteCtas<NV, sizeof(typename Elem::Raw)>)
route_fwd_kernel(const __grid_constant__ RouteParams p, const int per) {
  using Raw = typename Elem::Raw;
  constexpr int R = kWarp / LPR;                                 // rows of a pass
  constexpr int kPer = VB / int(sizeof(Raw));                    // elements per load
  constexpr int kMaxima = (NV + 7) / 8;
  constexpr bool kSpread = NV <= 32;                             // values go through shared memory to be picked by place
  using Mask = typename std::conditional<NV <= 32, uint32_t, unsigned long long>::type;
  __shared__ __align__(16) float s_val[kRouteWarps][kSpread ? NV * kWarp : 4];
  __shared__ __align__(16) float s_cv[kRouteWarps][R][kCand];    // candidates, in expert order
  __shared__ int s_ce[kRouteWarps][R][kCand];
  __shared__ float2 s_ranked[kRouteWarps][kMaxPer][kMaxRounds];  // value and expert (as bits), largest first
  __shared__ unsigned s_kept[kRouteWarps][kMaxPer];              // lanes of the groups taken
  extern __shared__ __align__(16) float s_bias[];                // in lane order, NV (rounded up to 4) a lane; then
  int* s_hist = reinterpret_cast<int*>(s_bias + LPR * ((NV + 3) / 4 * 4));   // the counts [E]
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  const int li = lane % LPR, rr = lane / LPR;
  const int g = li >> p.tshift, sub = li & ((1 << p.tshift) - 1);
  const int base = g * p.gs + sub * p.tchunk;
  const int n = g < p.G ? max(0, min(p.tchunk, p.gs - sub * p.tchunk)) : 0;
  const bool has_bias = p.bias != nullptr;
  const bool grouped = p.keep < p.G;
  const int rounds = has_bias ? p.k + 2 : p.k;
  for (int e = threadIdx.x; e < p.E; e += kRouteThreads) s_hist[e] = 0;
  if (MODE != 0 && warp < NV / 4 && rr == 0)                     // [i / 4][li][i % 4]: a lane reads four at a time
    for (int i4 = warp; i4 < (NV + 3) / 4; i4 += kRouteWarps)
#pragma unroll
      for (int j = 0; j < 4; ++j) s_bias[(i4 * LPR + li) * 4 + j] = has_bias && i4 * 4 + j < n ? p.bias[base + i4 * 4 + j] : 0.f;
  __syncthreads();

  Raw raw[NV];
  const auto fetch = [&](int64_t row) {
    const Raw* src = static_cast<const Raw*>(p.logits) + row * p.E + base;
#pragma unroll
    for (int v = 0; v < NV / kPer; ++v) {
      alignas(16) Raw part[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) part[i] = Elem::kNegInf;
      if (row < p.T && (FULL ? n > 0 : v * kPer < n)) {
        if constexpr (VB == 16) *reinterpret_cast<uint4*>(part) = *reinterpret_cast<const uint4*>(src + v * kPer);
        else if constexpr (VB == 4) *reinterpret_cast<uint32_t*>(part) = *reinterpret_cast<const uint32_t*>(src + v * kPer);
        else part[0] = src[v];
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) raw[v * kPer + i] = part[i];
    }
  };
  const auto logit = [&](int i) {
    const float x = __uint_as_float(Elem::bits(raw[i]));
    return x == x ? x : neg_inf();                               // not a number: masked
  };

  const int64_t stride = int64_t(gridDim.x) * kRouteWarps * per;
  const int64_t first0 = (int64_t(blockIdx.x) * kRouteWarps + warp) * per;
  for (int64_t first = first0; first < p.T; first += stride) {
    float my_max = 0.f, my_sum = 1.f, my_tol = 0.f;              // of row first + lane / 8
    unsigned close_rows = 0u, unsure_rows = 0u;
    const int rows = int(min(int64_t(per), p.T - first));
    for (int r0 = 0; r0 < rows; r0 += R) {
      fetch(first + r0 + rr);

      // Choice values in fp32.  Their error is within tol / 2.
      float c[NV], tol = 0.f;
      if constexpr (MODE == 2) {
        float m = logit(0);
#pragma unroll
        for (int i = 1; i < NV; ++i) m = fmaxf(m, logit(i));
        const float top = row_max<LPR>(m);
        m = top > neg_inf() ? top : 0.f;
        float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          c[i] = ex2_approx((logit(i) - m) * kLog2e);
          part[i % 4] += c[i];
        }
        const float sum = row_sum<LPR>((part[0] + part[1]) + (part[2] + part[3]));
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) c[i] *= inv;
        // In units of the row's largest score, 1 / sum: a score's rounded argument moves
        // it by 3 * 2^-24 x e^-x <= 0.7e-7, ex2.approx by 2^-22 of itself and of the
        // sum, the sum's NV / 4 + 7 additions by 2^-24 each, the quotient by 2^-23.
        // The sum's arguments move it too, by 3 * 2^-24 times the mean distance of the row's
        // logits from the largest, which for E experts is below t - 1, (t - 1) e^t = E - 1:
        // 8e-7 for 1024.  That is within tol: the sum's error scales all scores of the row
        // alike, so a comparison meets it once, and tol counts it for either side; against
        // scores from an exact sum (settling a row) it meets one side only.
        tol = (2.f * 6.7e-7f + (NV / 4 + 7) * 2.f * 6e-8f) * inv;
        const int from = (lane / kPickLanes - r0) * LPR;         // the row whose pick the lane will hold
        const bool mine = lane / kPickLanes >= r0 && lane / kPickLanes < r0 + R;
        const float t = __shfl_sync(kFull, top, from & 31), u = __shfl_sync(kFull, sum, from & 31), v = __shfl_sync(kFull, tol, from & 31);
        if (mine) {
          my_max = t;
          my_sum = u;
          my_tol = v;
        }
      } else if constexpr (MODE == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) c[i] = rcp_approx(1.f + ex2_approx(logit(i) * -kLog2e));
        // e = exp(-z) is off by 2^-22 (ex2.approx) + 1.5 |z| 2^-24 (its rounded argument and
        // log2 e) of itself, which moves s by s (1 - s) of that, at most 0.7e-7; 1 + e is
        // rounded (2^-24 of s), rcp.approx is off by 2^-23 of s: 2.6e-7 covers them
        tol = my_tol = 5.2e-7f;
      }
      if constexpr (MODE != 0) {
#pragma unroll
        for (int i = 0; i < NV; i += 4) {
          const float4 b = *reinterpret_cast<const float4*>(&s_bias[(i / 4 * LPR + li) * 4]);
          const float bi[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (i + j < NV) c[i + j] = logit(i + j) > neg_inf() && (FULL || i + j < n) ? c[i + j] + bi[j] : neg_inf();
        }
      }

      bool open = g < p.G;                                       // whether the lane's group is a choice
      float score = neg_inf(), size = 0.f;                       // of the group; the sizes of the values it is made of
      if (grouped && MODE != 0 && p.top2) {
        float a = neg_inf(), b = neg_inf();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          b = fmaxf(b, fminf(a, c[i]));
          a = fmaxf(a, c[i]);
        }
        for (int off = 1 << p.tshift >> 1; off > 0; off >>= 1) {
          const float a2 = __shfl_xor_sync(kFull, a, off), b2 = __shfl_xor_sync(kFull, b, off);
          b = fmaxf(fminf(a, a2), fmaxf(b, b2));
          a = fmaxf(a, a2);
        }
        score = b > neg_inf() ? a + b : a;
        size = a > neg_inf() ? fabsf(a) + (b > neg_inf() ? fabsf(b) : 0.f) : 0.f;
      }
      if (MODE == 0 || !has_bias) {                              // without a bias the logits' order is the scores'
#pragma unroll
        for (int i = 0; i < NV; ++i) c[i] = logit(i);
      }
      if constexpr (!FULL) {
#pragma unroll
        for (int i = 0; i < NV; ++i) c[i] = i < n ? c[i] : none();
      }

      float best[kMaxima];                                       // the maxima of eight
#pragma unroll
      for (int j = 0; j < kMaxima; ++j) {
        best[j] = c[8 * j];
#pragma unroll
        for (int i = 8 * j + 1; i < 8 * j + 8 && i < NV; ++i) best[j] = fmaxf(best[j], c[i]);
      }
      bool hangs = false;                                        // whether the choice of groups hangs on rounding
      if (grouped) {
        if (MODE == 0 || !p.top2) {
          score = best[0];
#pragma unroll
          for (int j = 1; j < kMaxima; ++j) score = fmaxf(score, best[j]);
          for (int off = 1 << p.tshift >> 1; off > 0; off >>= 1) score = fmaxf(score, __shfl_xor_sync(kFull, score, off));
        }
        if (!open) score = none();
        // The groups above this one; of equal ones the lower index is above.
        int rank = 0;
        for (int o = 1 << p.tshift; o < LPR; o += 1 << p.tshift) {
          const float other = __shfl_xor_sync(kFull, score, o);
          rank += other > score || (other == score && (li ^ o) < li);
        }
        const bool kept = open && rank < p.keep;
        if (MODE != 0 && (has_bias || p.top2)) {
          // A score is the true one within tol / 2 for each of its values and two roundings of
          // 2^-24 of their sizes: where the bias was added, and where the two were, which can
          // be far larger than their sum.  (The lines below round outwards.)  A masked group's
          // is exact; where the sizes pass fp32 nothing is known.
          if (!p.top2) size = score > neg_inf() ? fabsf(score) : 0.f;
          const float e = 1.2e-7f * size;
          const bool known = e < __uint_as_float(0x7f800000u);
          const float least = known ? __fsub_rd(score, e) : neg_inf(), most = known ? __fadd_ru(score, e) : -neg_inf();
          const float lo = -row_max<LPR>(kept ? -least : none()), hi = row_max<LPR>(kept ? none() : most);
          hangs = __fsub_rd(lo, hi) <= (p.top2 ? 2.f * tol : tol);
        }
        open = kept;
        const unsigned lanes = __ballot_sync(kFull, kept);
        if (li == 0) s_kept[warp][r0 + rr] = lanes >> (rr * LPR);
      }

      // The bound.
      float reach = none();
#pragma unroll
      for (int j = 0; j < kMaxima; ++j) best[j] = open ? best[j] : none();
      for (int j = 0; j < p.k; ++j) {
        float m = best[0];
#pragma unroll
        for (int i = 1; i < kMaxima; ++i) m = fmaxf(m, best[i]);
        reach = row_max<LPR>(m);
#pragma unroll
        for (int i = 0; i < kMaxima; ++i) best[i] = best[i] == reach ? none() : best[i];
      }
      reach = reach == reach ? reach : neg_inf();                // fewer maxima than picks: everything
      if (MODE != 0 && has_bias) reach -= tol + 2.4e-7f * fabsf(reach);
      Mask mask = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) mask |= c[i] >= reach ? Mask(1) << i : Mask(0);
      if (!open) mask = 0;
      const int count = NV <= 32 ? __popc(uint32_t(mask)) : __popcll((unsigned long long)mask);
      int before = count;
#pragma unroll
      for (int off = 1; off < LPR; off <<= 1) {
        const int o = __shfl_up_sync(kFull, before, off, LPR);
        if (li >= off) before += o;
      }
      const int total = __shfl_sync(kFull, before, LPR - 1, LPR);
      float2* ranked = s_ranked[warp][r0 + rr];
      const bool fits = total <= kCand;
      if (fits) {
        int at = before - count;
        if constexpr (kSpread) {
          float* val = &s_val[warp][lane * 4];
          if (count > 0) {
#pragma unroll
            for (int i = 0; i < NV; i += 4)
              *reinterpret_cast<float4*>(val + i * kWarp) =
                  make_float4(c[i], i + 1 < NV ? c[i + 1 < NV ? i + 1 : i] : 0.f, i + 2 < NV ? c[i + 2 < NV ? i + 2 : i] : 0.f, i + 3 < NV ? c[i + 3 < NV ? i + 3 : i] : 0.f);
            while (mask != 0) {                                  // the lane's own values: no other lane's writes are read
              const int i = __ffs(int(mask)) - 1;
              mask &= mask - 1;
              s_cv[warp][rr][at] = val[(i & ~3) * kWarp + (i & 3)];
              s_ce[warp][rr][at] = base + i;
              ++at;
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (mask >> i & 1) {
              s_cv[warp][rr][at] = c[i];
              s_ce[warp][rr][at] = base + i;
              ++at;
            }
        }
        for (int q = li; q < kCand; q += LPR)
          if (q >= total) s_cv[warp][rr][q] = none();
        for (int j = li; j < rounds; j += LPR)
          if (j >= total) ranked[j] = make_float2(none(), 0.f);
      }
      __syncwarp();
      if (fits) {
        for (int q = li; q < total; q += LPR) {
          const float mine = s_cv[warp][rr][q];
          int rank = 0;
          for (int o = 0; o < total; o += 4) {
            const float4 v = *reinterpret_cast<const float4*>(&s_cv[warp][rr][o]);
            rank += v.x > mine || (v.x == mine && o < q);
            rank += v.y > mine || (v.y == mine && o + 1 < q);
            rank += v.z > mine || (v.z == mine && o + 2 < q);
            rank += v.w > mine || (v.w == mine && o + 3 < q);
          }
          if (rank < rounds) ranked[rank] = make_float2(mine, __int_as_float(s_ce[warp][rr][q]));
        }
      }
      if (!__all_sync(kFull, fits)) {
        for (int j = 0; j < rounds; ++j) {
          float m = none();
          if (open) {
#pragma unroll
            for (int i = 0; i < NV; ++i) m = fmaxf(m, c[i]);
          }
          const float top = row_max<LPR>(m);
          const unsigned have = __ballot_sync(kFull, open && m == top) >> (rr * LPR) & (LPR == 32 ? kFull : (1u << (LPR & 31)) - 1u);
          if (have != 0u ? li == __ffs(have) - 1 : li == 0) {    // the lowest lane that has it, or none is left
            bool found = have == 0u;
            if (!fits && found) ranked[j] = make_float2(none(), 0.f);
#pragma unroll
            for (int i = 0; i < NV; ++i)
              if (!found && c[i] == top) {
                found = true;
                if (!fits) ranked[j] = make_float2(top, __int_as_float(base + i));
                c[i] = none();
              }
          }
        }
      }
      __syncwarp();
      if (MODE != 0 && has_bias) {
        const float v = li < p.k ? ranked[li].x : none(), next = li < p.k ? ranked[li + 1].x : none();
        const unsigned close = __ballot_sync(kFull, v - next <= tol + 2.4e-7f * fabsf(v));
#pragma unroll
        for (int q = 0; q < R; ++q)
          if (close >> (q * LPR) & (LPR == 32 ? kFull : (1u << (LPR & 31)) - 1u)) close_rows |= 1u << (r0 + q);
      }
      if (MODE != 0 && grouped && (has_bias || p.top2)) {
        const unsigned unsure = __ballot_sync(kFull, hangs);
#pragma unroll
        for (int q = 0; q < R; ++q)
          if (unsure >> (q * LPR) & 1u) unsure_rows |= 1u << (r0 + q);
      }
    }
    const unsigned real = (1u << rows) - 1u;
    if (MODE != 0 && ((close_rows | unsure_rows) & real) != 0u) {
      for (unsigned left = (close_rows | unsure_rows) & real; left != 0u; left &= left - 1u) {
        const int r = __ffs(left) - 1;
        const float2 v = lane < rounds ? s_ranked[warp][r][lane] : make_float2(none(), 0.f);
        const int e = route_settle<Elem>(p, first + r, lane, v.x, __float_as_int(v.y), rounds, __shfl_sync(kFull, my_tol, r * kPickLanes),
                                         close_rows >> r & 1, unsure_rows >> r & 1, s_kept[warp][r], &s_ce[warp][0][0]);
        if (lane < p.k) s_ranked[warp][r][lane].y = __int_as_float(e);
        __syncwarp();
      }
    }

    const int64_t row = first + lane / kPickLanes;
    const bool pick = lane / kPickLanes < rows && lane % kPickLanes < p.k;
    const int my_e = pick ? __float_as_int(s_ranked[warp][lane / kPickLanes][lane % kPickLanes].y) : 0;
    __syncwarp();                                                // read before the next rows' are written
    const float zp = pick ? load_logit<Elem>(p.logits, row * p.E + my_e) : neg_inf();
    float w;
    if (p.renorm) {
      w = pick_share(pick_weight(zp, pick, p.softmax), p.k);
    } else if (p.softmax) {
      w = my_sum > 0.f && zp > neg_inf() ? expf(zp - my_max) / my_sum : 0.f;
    } else {
      w = zp > neg_inf() ? sigmoid_exact(zp) : 0.f;
    }
    if (pick) {
      const int64_t at = row * p.k + lane % kPickLanes;
      p.idx[at] = my_e;
      p.gate[at] = p.scale * w;
      atomicAdd(&s_hist[my_e], 1);
    }
  }
  __syncthreads();
  const uint32_t ctas = cluster_ctas();
  if (gridDim.x > ctas) {
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads)
      if (s_hist[e] != 0) atomicAdd(&p.counts[e], s_hist[e]);   // integers: any order gives the same sum
    return;
  }
  // One cluster has all rows: its CTAs finish the experts between them.
  if (ctas > 1) cluster_barrier();
  for (int e = cluster_rank() * kRouteThreads + threadIdx.x; e < p.E; e += ctas * kRouteThreads) {
    int cnt = 0;
    for (uint32_t r = 0; r < ctas; ++r) cnt += cluster_load(&s_hist[e], r);
    p.counts[e] = cnt;
    if (p.bias_out != nullptr) {
      const int64_t over = p.T * p.k - int64_t(cnt) * p.E;
      const float b = has_bias ? p.bias[e] : 0.f;
      p.bias_out[e] = over > 0 ? b + p.bias_gamma : over < 0 ? b - p.bias_gamma : b;
    }
  }
  if (ctas > 1) cluster_barrier();                               // its counts have been read
}

// bias + gamma * sign(T*k/E - count), after all counts are in.
__global__ void __launch_bounds__(256) route_bias_kernel(const RouteParams p) {
  const int e = blockIdx.x * blockDim.x + threadIdx.x;
  if (e >= p.E) return;
  const int64_t over = p.T * p.k - int64_t(p.counts[e]) * p.E;
  const float b = p.bias != nullptr ? p.bias[e] : 0.f;
  p.bias_out[e] = over > 0 ? b + p.bias_gamma : over < 0 ? b - p.bias_gamma : b;
}

// Four rows a warp share the work on the picks; where a pass has fewer, only from 64 rows
// an SM on (1024 experts, a row a pass: 2048 rows 24.7 us with one row a warp and 32.8 with
// four, 8192 rows 39.7 and 38.8, 32,768 rows 112 and 99).
int rows_per_warp(int64_t T, int sms) { return T >= int64_t(sms) * 64 ? 4 : 1; }
// CTAs of a cluster.  One CTA alone, and one cluster, write counts and bias without a second
// and third launch; each takes what it has in one pass (256 experts, 32 rows a CTA, with a
// bias; CTA, cluster, more CTAs: 32 rows 6.6, 7.7 and 11.5 us; 64 rows 10.7, 7.6 and 11.2;
// 256 rows -, 8.9 and 13.0; 512 rows, two passes, 12.8 and 12.9; 768 rows 16.3 and 12.3).
constexpr int kCluster = 8;

template <class Elem, int LPR, int NV, int VB, bool FULL, int MODE>
cudaError_t fwd_launch(const RouteParams& p, int sms, cudaStream_t stream) {
  const size_t counts = size_t(p.E) * sizeof(int), smem = counts + size_t(LPR) * ((NV + 3) / 4 * 4) * sizeof(float);
  constexpr int R = kWarp / LPR;
  if (p.T <= kRouteWarps * R) {
    route_fwd_kernel<Elem, LPR, NV, VB, FULL, MODE><<<1, kRouteThreads, smem, stream>>>(p, R);
    return cudaGetLastError();
  }
  if (p.T <= kCluster * kRouteWarps * R) {
    cudaLaunchAttribute cluster = {};
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = kCluster;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kRouteThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = &cluster;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, route_fwd_kernel<Elem, LPR, NV, VB, FULL, MODE>, p, R);
  }
  cudaError_t e = cudaMemsetAsync(p.counts, 0, counts, stream);
  if (e != cudaSuccess) return e;
  const int per = rows_per_warp(p.T, sms) > R ? rows_per_warp(p.T, sms) : R;
  const int64_t rows = int64_t(kRouteWarps) * per, want = (p.T + rows - 1) / rows;
  const int64_t most = int64_t(sms) * 8;
  route_fwd_kernel<Elem, LPR, NV, VB, FULL, MODE><<<int(want < most ? want : most), kRouteThreads, smem, stream>>>(p, per);
  if ((e = cudaGetLastError()) != cudaSuccess || p.bias_out == nullptr) return e;
  route_bias_kernel<<<(p.E + 255) / 256, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

template <class Elem, int LPR, int NV, int MODE>
cudaError_t fwd_width(const RouteParams& p, int sms, cudaStream_t stream) {
  constexpr int kSize = int(sizeof(typename Elem::Raw)), VB = 16;
  static_assert(NV * kSize % VB == 0, "a lane's experts are whole loads");
  // Loads of 16 bytes: every lane has NV experts or none, and rows, groups and the array are aligned.
  const bool full = p.tchunk == NV && p.gs == (p.tchunk << p.tshift);
  if (full && int64_t(p.E) * kSize % VB == 0 && reinterpret_cast<uintptr_t>(p.logits) % VB == 0)
    return fwd_launch<Elem, LPR, NV, VB, true, MODE>(p, sms, stream);
  return fwd_launch<Elem, LPR, NV, kSize, false, MODE>(p, sms, stream);
}

template <class Elem, int LPR, int MODE>
cudaError_t fwd_lanes(const RouteParams& p, int sms, cudaStream_t stream) {
  if (p.tchunk <= 8) return fwd_width<Elem, LPR, 8, MODE>(p, sms, stream);
  if (p.tchunk <= 16) return fwd_width<Elem, LPR, 16, MODE>(p, sms, stream);
  return fwd_width<Elem, LPR, 32, MODE>(p, sms, stream);
}

// The fewest lanes of a row that hold its groups apart with at most 32 experts a
// lane: steps across lanes then serve the most rows.
template <class Elem, int MODE>
cudaError_t fwd_mode(RouteParams p, int sms, cudaStream_t stream) {
  int groups = 1;                                                // rounded up to a power of two
  while (groups < p.G) groups *= 2;
  int lpr = groups < 8 ? 8 : groups;
  while (lpr < kWarp && (p.gs + lpr / groups - 1) / (lpr / groups) > 32) lpr *= 2;
  p.tshift = 0;
  while (groups << (p.tshift + 1) <= lpr) ++p.tshift;
  p.tchunk = (p.gs + (1 << p.tshift) - 1) >> p.tshift;
  if (lpr == 8) return fwd_lanes<Elem, 8, MODE>(p, sms, stream);
  if (lpr == 16) return fwd_lanes<Elem, 16, MODE>(p, sms, stream);
  if (p.tchunk <= 32) return fwd_lanes<Elem, 32, MODE>(p, sms, stream);
  return fwd_launch<Elem, 32, 64, int(sizeof(typename Elem::Raw)), false, MODE>(p, sms, stream);
}

template <class Elem>
cudaError_t fwd_elem(const RouteParams& p, int sms, cudaStream_t stream) {
  const bool grouped = p.keep < p.G;
  if (p.softmax && (p.bias != nullptr || (p.top2 && grouped) || !p.renorm)) return fwd_mode<Elem, 2>(p, sms, stream);
  if (!p.softmax && (p.bias != nullptr || (p.top2 && grouped))) return fwd_mode<Elem, 1>(p, sms, stream);
  return fwd_mode<Elem, 0>(p, sms, stream);
}

// ---------------------------------------------------------------------------
// Backward.  The picks are held constant, so with sigmoid scores or
// renormalised softmax gates only the picked logits have a gradient: the row
// of zeros is what is written, and only the picked logits are read.  Softmax
// scores taken as they are reach every logit.  Lane j < k holds pick j; picks
// that name one expert twice add up; an index outside [0, E) contributes
// nothing.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float sum_same(float v, int e, int k) {
  float total = 0.f;
  for (int j = 0; j < k; ++j) {
    const float o = pick_value(v, j);
    if (__shfl_sync(kFull, e, j, kPickLanes) == e) total += o;
  }
  return total;
}

// Four rows a warp, lane 8 r + j with pick j of row r.  (One row a warp is no faster even
// for few rows: 4096 x 256 3.7 us against 3.0, 65,536 30 us against 15.)
template <class Elem, bool VEC>
__global__ void __launch_bounds__(kRouteThreads) route_bwd_picks_kernel(const RouteBwdParams p) {
  constexpr int per = kMaxPer;
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  const int j = lane % kPickLanes;
  const int64_t stride = int64_t(gridDim.x) * kRouteWarps * per;
  for (int64_t first = (int64_t(blockIdx.x) * kRouteWarps + warp) * per; first < p.T; first += stride) {
    const int64_t row = first + lane / kPickLanes;
    const bool there = row < p.T && j < p.k;
    const int e = there ? p.idx[row * p.k + j] : -1;
    const bool live = e >= 0 && e < p.E;
    const float dg = live ? p.scale * p.dgate[row * p.k + j] : 0.f;
    const float z = live ? load_logit<Elem>(p.logits, row * p.E + e) : neg_inf();
    float* out = p.dlogits + first * p.E;
    const int64_t rows = p.T - first < per ? p.T - first : per;
    if constexpr (VEC) {
      for (int i = lane; i < int(rows) * p.E / 4; i += kWarp) reinterpret_cast<float4*>(out)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
      for (int i = lane; i < int(rows) * p.E; i += kWarp) out[i] = 0.f;
    }
    float v;
    if (p.renorm) {
      const float w = pick_share(pick_weight(z, live, p.softmax), p.k);
      float d = 0.f;                                     // dg - sum_i w_i dg_i, as a sum of differences
      for (int i = 0; i < p.k; ++i) d += pick_value(w, i) * (dg - pick_value(dg, i));
      v = w * d;
      if (!p.softmax && w > 0.f) v *= sigmoid_exact(-z); // 1 - sigmoid(z)
    } else {
      v = live && z > neg_inf() ? dg * sigmoid_exact(z) * sigmoid_exact(-z) : 0.f;
    }
    v = sum_same(v, e, p.k);
    __syncwarp();                                        // the zeros lie before the picks' values
    if (live) p.dlogits[row * p.E + e] = v;
  }
}

// CTAs of an SM: the loads' latency is hidden by other rows.
template <int NV>
constexpr int kBwdCtas = NV <= 4 ? 8 : NV <= 8 ? 6 : NV <= 12 ? 5 : 4;

template <class Elem, int NV>
__global__ void __launch_bounds__(kRouteThreads, kBwdCtas<NV>) route_bwd_softmax_kernel(const RouteBwdParams p) {
  __shared__ float4 s_pick[kRouteWarps][kPickLanes];     // a row's picks: expert (as bits), dgate, score times dgate
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  const int64_t stride = int64_t(gridDim.x) * kRouteWarps;
  for (int64_t row = int64_t(blockIdx.x) * kRouteWarps + warp; row < p.T; row += stride) {
    float z[NV], m = neg_inf(), sum = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * kWarp + lane;
      z[i] = c < p.E ? load_logit<Elem>(p.logits, row * p.E + c) : neg_inf();
      if (!(z[i] == z[i])) z[i] = neg_inf();             // not a number: masked
      m = fmaxf(m, z[i]);
    }
    m = warp_max_f(m);
    const float shift = m > neg_inf() ? m : 0.f;
    const int e = lane < p.k ? p.idx[row * p.k + lane] : -1;
    const bool live = e >= 0 && e < p.E;
    const float dg = live ? p.scale * p.dgate[row * p.k + lane] : 0.f;
    const float zp = live ? load_logit<Elem>(p.logits, row * p.E + e) : neg_inf();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      z[i] = ex2_approx((z[i] - shift) * kLog2e);
      sum += z[i];
    }
    sum = warp_sum_f(sum);
    const float own = zp > neg_inf() ? ex2_approx((zp - shift) * kLog2e) : 0.f;
    // dg_i - sum_j p_j dg_j at a pick, as dg_i times the share of all other experts less the
    // other picks' p_j dg_j: next to an expert that has nearly all of the row the rest is
    // small, and its digits count.  So it is summed apart there.
    float outside = sum - own;
    const unsigned most = __ballot_sync(kFull, own > 0.5f * sum);
    if (most != 0u) {
      const int o = __shfl_sync(kFull, e, __ffs(most) - 1), at = o % kWarp == lane ? o / kWarp : -1;
      float rest = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i != at) rest += z[i];
      rest = warp_sum_f(rest);
      if (e == o) outside = rest;
    }
    if (lane < kPickLanes) s_pick[warp][lane] = make_float4(__int_as_float(e), dg, own * dg, 0.f);
    __syncwarp();
    float dge = 0.f, S = 0.f, others = 0.f;              // the lanes from 8 on have no pick
    for (int j = 0; j < p.k; ++j) {
      const float4 o = s_pick[warp][j];
      const bool same = __float_as_int(o.x) == e;
      S += o.z;
      if (same) dge += o.y;
      if (!same) others += o.z;
    }
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const float v = own * inv * ((dge * outside - others) * inv);
    S *= inv;
    float* out = p.dlogits + row * p.E;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = i * kWarp + lane;
      if (c < p.E) out[c] = -(z[i] * inv) * S;
    }
    __syncwarp();
    if (live) out[e] = v;
  }
}

template <class Elem, int NV>
cudaError_t bwd_softmax(const RouteBwdParams& p, int sms, cudaStream_t stream) {
  const int64_t want = (p.T + kRouteWarps - 1) / kRouteWarps, most = int64_t(sms) * kBwdCtas<NV>;   // all at once
  route_bwd_softmax_kernel<Elem, NV><<<int(want < most ? want : most), kRouteThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <class Elem>
cudaError_t bwd_elem(const RouteBwdParams& p, int sms, cudaStream_t stream) {
  if (p.softmax && !p.renorm) {
    if (p.E <= 4 * kWarp) return bwd_softmax<Elem, 4>(p, sms, stream);
    if (p.E <= 8 * kWarp) return bwd_softmax<Elem, 8>(p, sms, stream);
    if (p.E <= 12 * kWarp) return bwd_softmax<Elem, 12>(p, sms, stream);
    return bwd_softmax<Elem, 32>(p, sms, stream);
  }
  const int64_t rows = int64_t(kRouteWarps) * kMaxPer, want = (p.T + rows - 1) / rows;
  const int64_t most = int64_t(sms) * 8;
  const int grid = int(want < most ? want : most);
  if (p.E % 4 == 0 && reinterpret_cast<uintptr_t>(p.dlogits) % 16 == 0)
    route_bwd_picks_kernel<Elem, true><<<grid, kRouteThreads, 0, stream>>>(p);
  else
    route_bwd_picks_kernel<Elem, false><<<grid, kRouteThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace
}  // namespace moe
