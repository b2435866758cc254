// Scored, group-limited routing and its gradient.
//
// Scores s = sigmoid(z) or softmax(z); an expert's choice value is s + bias
// (its logit's order without a bias); a group of experts is scored by its
// largest choice value or the sum of its two largest; the k largest choice
// values within the best groups are picked; gates are the picks' scores,
// renormalised over the picks if asked, times a scale.
//
// One warp works on one row.  A group's experts lie in L consecutive lanes
// (L the largest power of two with G * L <= 32), `chunk` consecutive experts
// in each, so that the lane order is the expert order (ties go to the lowest
// lane) and a group's score is a butterfly over its lanes.
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

namespace moe {
namespace {

constexpr int kRouteThreads = 256;
constexpr int kRouteWarps = kRouteThreads / kWarp;
// Rows that one CTA takes alone, in one launch that also writes the counts and
// the bias.  Beyond them, more CTAs and a cleared counter array in front.
constexpr int kRouteOneCtaRows = 32;
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ float neg_inf() { return __uint_as_float(0xff800000u); }

// Order-preserving key of a float that is not NaN; 0 is below every key.
__device__ __forceinline__ uint32_t float_key(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ (uint32_t(int(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_float(uint32_t k) {
  return __uint_as_float(k ^ ((k & 0x80000000u) ? 0x80000000u : 0xffffffffu));
}

template <class Elem>
__device__ __forceinline__ float load_logit(const void* logits, int64_t at) {
  return __uint_as_float(Elem::bits(static_cast<const typename Elem::Raw*>(logits)[at]));
}

__device__ __forceinline__ float warp_max_f(float x) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, off));
  return x;
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

// ---------------------------------------------------------------------------
// The row ranked in double: the definition, by all lanes of the warp.  Lane j
// gets pick j.  `bias` and the row are read again (they are in the caches).
// ---------------------------------------------------------------------------
template <class Elem>
__device__ __noinline__ int route_row_double(const RouteParams& p, int64_t row, int lane) {
  double c[64];                                                  // choice values of the lane's experts
  const int g = lane / p.L, base = g * p.gs + (lane % p.L) * p.chunk;
  const int n = g < p.G ? max(0, min(p.chunk, p.gs - (lane % p.L) * p.chunk)) : 0;
  const double ninf = double(neg_inf());
  float m = neg_inf();
  for (int i = 0; i < n; ++i) m = fmaxf(m, load_logit<Elem>(p.logits, row * p.E + base + i));
  m = warp_max_f(m);
  double sum = 0.0;
  for (int i = 0; i < n; ++i) {
    const float z = load_logit<Elem>(p.logits, row * p.E + base + i);
    double s = 0.0;
    if (z > neg_inf()) s = p.softmax ? exp(double(z) - double(m)) : 1.0 / (1.0 + exp(-double(z)));
    c[i] = s;
    sum += s;
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(kFull, sum, off);
  double a = ninf, b = ninf;                                     // the two largest of the lane, then of the group
  unsigned long long gone = 0;
  for (int i = 0; i < n; ++i) {
    const float z = load_logit<Elem>(p.logits, row * p.E + base + i);
    double v = p.softmax ? c[i] / sum : c[i];
    if (p.bias != nullptr) v += double(p.bias[base + i]);
    if (!(z > neg_inf())) v = ninf;
    const double order = p.bias != nullptr || !(z > neg_inf()) ? v : double(z);
    const double u = p.top2 ? v : order;
    if (u > a) {
      b = a;
      a = u;
    } else if (u > b) {
      b = u;
    }
    c[i] = order;
  }
  if (p.G > 1) {
    for (int off = 1; off < p.L; off <<= 1) {
      const double a2 = __shfl_xor_sync(kFull, a, off), b2 = __shfl_xor_sync(kFull, b, off);
      b = fmax(fmin(a, a2), fmax(b, b2));
      a = fmax(a, a2);
    }
    const double score = p.top2 && b > ninf ? a + b : a;
    int rank = 0;
    for (int o = 0; o < p.G; ++o) {
      const double other = __shfl_sync(kFull, score, o * p.L);
      rank += other > score || (other == score && o < g);
    }
    if (rank >= p.keep) gone = ~0ull;
  }
  int mine = 0;
  for (int j = 0; j < p.k; ++j) {
    double v = ninf;
    int e = 0x7fffffff;
    for (int i = 0; i < n; ++i)
      if (!(gone >> i & 1) && (e == 0x7fffffff || c[i] > v)) {
        v = c[i];
        e = base + i;
      }
    for (int off = 16; off > 0; off >>= 1) {
      const double v2 = __shfl_xor_sync(kFull, v, off);
      const int e2 = __shfl_xor_sync(kFull, e, off);
      const bool take = e == 0x7fffffff ? e2 != 0x7fffffff : e2 != 0x7fffffff && (v2 > v || (v2 == v && e2 < e));
      if (take) {
        v = v2;
        e = e2;
      }
    }
    if (e >= base && e < base + n) gone |= 1ull << (e - base);
    if (lane == j) mine = e;
  }
  return mine;
}

// ---------------------------------------------------------------------------
// The picks of a row where values that decide them are next to one another
// (`close`), or where its groups' scores are (`unsure`).  Lane j holds the j-th
// largest key and its expert, the k picks and two more.
// ---------------------------------------------------------------------------
template <class Elem>
__device__ __noinline__ int route_settle(const RouteParams& p, int64_t row, int lane, uint32_t ck, int ce, int rounds,
                                         float tol, bool close, bool unsure) {
  const bool there = lane < rounds && ck != 0u;
  const float zc = there ? load_logit<Elem>(p.logits, row * p.E + ce) : neg_inf();
  const float bc = there && p.bias != nullptr ? p.bias[ce] : 0.f, c = key_float(ck);
  const float c_up = __shfl_up_sync(kFull, c, 1), z_up = __shfl_up_sync(kFull, zc, 1), b_up = __shfl_up_sync(kFull, bc, 1);
  // sure all the same where the inputs are equal
  const bool open = close && lane >= 1 && lane <= p.k && there && c_up - c <= tol + 2.4e-7f * fabsf(c_up) &&
                    !(zc == z_up && bc == b_up);
  const float last = __shfl_sync(kFull, c, p.k - 1);
  const bool beyond = lane == p.k + 1 && there && last - c <= tol + 2.4e-7f * fabsf(last);
  const bool any_open = __any_sync(kFull, open), any_beyond = __any_sync(kFull, beyond);
  if (unsure || (any_open && (any_beyond || p.softmax))) return route_row_double<Elem>(p, row, lane);
  if (!any_open) return ce;
  // The k + 1 largest are known as a set: one double-precision sigmoid a lane orders them.
  const bool in = there && lane <= p.k;
  const double d = in && zc > neg_inf() ? 1.0 / (1.0 + exp(-double(zc))) + double(bc) : double(neg_inf());
  int rank = 0;
  for (int o = 0; o <= p.k; ++o) {
    const double od = __shfl_sync(kFull, d, o);
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
//   NV    experts per lane, at least `chunk`
//   VB    bytes per load; above the element's size only where every lane's NV
//         experts are there and aligned (FULL: no lane has fewer)
//   MODE  0: the order of the logits decides everything and gates need no sum over the
//         row; 1: sigmoid scores; 2: softmax scores
//
// Selection: the k largest of the lanes' maxima bound the k-th choice value from
// below (a warp reduction and two instructions each); the few experts that reach
// the bound are gathered, one a lane in expert order, and ranked by counting.
// With a bias two more than the k picks are ranked, to see what hangs on
// rounding.  Should more than 32 experts reach the bound (whole groups in single
// lanes, long ties), the warp takes the maximum again and again instead.  A warp
// selects for `per` rows one after another, each loaded while the one before is
// worked on; the rows that hang on rounding are settled behind them, and then
// the gates of all of them are computed, a pick a lane.
// The instructions bound it: sorting a lane's experts and popping them one by one
// took 1145 a row of 256.
// ---------------------------------------------------------------------------
constexpr int kMaxRounds = 10;                                   // 8 picks and two more
constexpr int kMaxPer = kWarp / kPickLanes;                      // rows a warp finishes at once

template <class Elem, int NV, int VB, bool FULL, int MODE>
__global__ void __launch_bounds__(kRouteThreads, NV <= 8 ? 4 : NV <= 16 ? 3 : NV <= 32 ? 2 : 1)
route_fwd_kernel(const __grid_constant__ RouteParams p, const int per) {
  using Raw = typename Elem::Raw;
  constexpr int kPer = VB / int(sizeof(Raw));                    // elements per load
  constexpr bool kAhead = NV * int(sizeof(Raw)) <= 64;           // whether the next row fits beside this one
  __shared__ __align__(16) uint2 s_cand[kRouteWarps][kWarp];     // key and expert of the candidates, in expert order
  __shared__ uint2 s_ranked[kRouteWarps][kMaxPer][kMaxRounds];   // largest first
  extern __shared__ int s_hist[];                                // [E]
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  for (int e = threadIdx.x; e < p.E; e += kRouteThreads) s_hist[e] = 0;
  __syncthreads();

  const int g = lane >> p.lshift, sub = lane & (p.L - 1);
  const int base = g * p.gs + sub * p.chunk;
  const int n = g < p.G ? max(0, min(p.chunk, p.gs - sub * p.chunk)) : 0;
  const bool has_bias = p.bias != nullptr;
  const bool grouped = p.keep < p.G;
  const int rounds = has_bias ? p.k + 2 : p.k;
  float bv[NV];
  const auto fetch_bias = [&]() {
#pragma unroll
    for (int i = 0; i < NV; ++i) bv[i] = has_bias && i < n ? p.bias[base + i] : 0.f;
  };
  fetch_bias();

  Raw raw[NV];
  const auto fetch = [&](int64_t row) {
    const Raw* src = static_cast<const Raw*>(p.logits) + row * p.E + base;
#pragma unroll
    for (int v = 0; v < NV / kPer; ++v) {
      alignas(16) Raw part[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) part[i] = Elem::kNegInf;
      if (FULL ? n > 0 : v * kPer < n) {
        if constexpr (VB == 16) *reinterpret_cast<uint4*>(part) = *reinterpret_cast<const uint4*>(src + v * kPer);
        else if constexpr (VB == 8) *reinterpret_cast<uint2*>(part) = *reinterpret_cast<const uint2*>(src + v * kPer);
        else if constexpr (VB == 4) *reinterpret_cast<uint32_t*>(part) = *reinterpret_cast<const uint32_t*>(src + v * kPer);
        else part[0] = src[v];
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) raw[v * kPer + i] = part[i];
    }
  };

  const int64_t stride = int64_t(gridDim.x) * kRouteWarps * per;
  const int64_t first0 = (int64_t(blockIdx.x) * kRouteWarps + warp) * per;
  if (kAhead && first0 < p.T) fetch(first0);
  for (int64_t first = first0; first < p.T; first += stride) {
    float my_max = 0.f, my_sum = 1.f, my_tol = 0.f;              // of row first + lane / 8
    unsigned close_rows = 0u, unsure_rows = 0u;
    const int rows = int(min(int64_t(per), p.T - first));
    for (int r = 0; r < rows; ++r) {
      const int64_t row = first + r;
      if constexpr (!kAhead) fetch(row);
      float z[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float x = __uint_as_float(Elem::bits(raw[i]));
        z[i] = x == x ? x : neg_inf();                           // not a number: never preferred
      }
      if constexpr (kAhead) {
        const int64_t then = r + 1 < rows ? row + 1 : first + stride;
        if (then < p.T) fetch(then);
      }

      // Choice values in fp32.  Their error is within tol / 2.
      float s[NV], tol = 0.f;
      if constexpr (MODE == 2) {
        float m = z[0];
#pragma unroll
        for (int i = 1; i < NV; ++i) m = fmaxf(m, z[i]);
        const float row_max = warp_max_f(m);
        m = row_max > neg_inf() ? row_max : 0.f;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          s[i] = ex2_approx((z[i] - m) * kLog2e);
          sum += s[i];
        }
        sum = warp_sum_f(sum);
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] *= inv;
        // x e^-x <= 0.37: the rounded argument moves a score by 2^-23 * 0.37 * 1.45 of
        // the row's largest, ex2.approx by 2^-22 of itself, the sum of at most 64
        // values a lane and 5 steps by 69 * 2^-24 of itself: 5e-6 covers them
        tol = 1e-5f * inv;
        if (lane / kPickLanes == r) {
          my_max = row_max;
          my_sum = sum;
          my_tol = tol;
        }
      } else if constexpr (MODE == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] = rcp_approx(1.f + ex2_approx(z[i] * -kLog2e));
        // e = exp(-z) is off by 2^-22 + 2^-24 * 1.45 |z| of itself; s moves by
        // s (1 - s) of that, below 2^-23, and rcp.approx and 1 + e by 2^-22 of s: 6e-7 covers them
        tol = my_tol = 1.2e-6f;
      }
      if constexpr (MODE != 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] = z[i] > neg_inf() ? s[i] + bv[i] : neg_inf();
      }
      uint32_t key[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const float v = MODE != 0 && has_bias ? s[i] : z[i];
        key[i] = FULL || i < n ? float_key(v + 0.f) : 0u;
      }

      bool open = g < p.G;                                       // whether the lane's group is a choice
      if (grouped) {
        uint32_t gkey;
        float gtol = tol;
        if (MODE != 0 && p.top2) {
          float a = neg_inf(), b = neg_inf();
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const float v = FULL || i < n ? s[i] : neg_inf();
            b = fmaxf(b, fminf(a, v));
            a = fmaxf(a, v);
          }
          for (int off = 1; off < p.L; off <<= 1) {
            const float a2 = __shfl_xor_sync(kFull, a, off), b2 = __shfl_xor_sync(kFull, b, off);
            b = fmaxf(fminf(a, a2), fmaxf(b, b2));
            a = fmaxf(a, a2);
          }
          gkey = float_key((b > neg_inf() ? a + b : a) + 0.f);
          gtol = 2.f * tol;
        } else {
          gkey = key[0];
#pragma unroll
          for (int i = 1; i < NV; ++i) gkey = max(gkey, key[i]);
          for (int off = 1; off < p.L; off <<= 1) gkey = max(gkey, __shfl_xor_sync(kFull, gkey, off));
        }
        if (!open) gkey = 0u;
        // The best group, `keep` times; groups that tie go by lane, the lower first.
        open = false;
        uint32_t worst = 0u;
        for (int j = 0; j < p.keep; ++j) {
          worst = __reduce_max_sync(kFull, gkey);
          const int at = __ffs(__ballot_sync(kFull, gkey == worst)) - 1;
          if (g == at >> p.lshift) {
            open = true;
            gkey = 0u;
          }
        }
        if (MODE != 0 && (has_bias || p.top2)) {
          const float lo = key_float(worst), hi = key_float(__reduce_max_sync(kFull, gkey));
          if (lo - hi <= gtol + 4.8e-7f * fabsf(lo)) unsure_rows |= 1u << r;   // + the sums' own roundings
        }
      }

      uint32_t best = 0u;
      if (open) {
#pragma unroll
        for (int i = 0; i < NV; ++i) best = max(best, key[i]);
      }
      uint32_t rest = best, reach = 0u;
#pragma unroll
      for (int j = 0; j < kMaxRounds; ++j) {
        if (j >= rounds) break;
        reach = __reduce_max_sync(kFull, rest);
        rest = rest == reach ? 0u : rest;
      }
      reach = open ? max(reach, 1u) : 0xffffffffu;               // 0: places without an expert; the last: above every number
      int count = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) count += key[i] >= reach;
      int before = count;
#pragma unroll
      for (int off = 1; off < kWarp; off <<= 1) {
        const int o = __shfl_up_sync(kFull, before, off);
        if (lane >= off) before += o;
      }
      const int total = __shfl_sync(kFull, before, kWarp - 1);
      uint2* ranked = s_ranked[warp][r];
      if (total <= kWarp) {
        uint2* at = &s_cand[warp][before - count];
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (key[i] >= reach) *at++ = make_uint2(key[i], uint32_t(base + i));
        if (lane >= total) s_cand[warp][lane] = make_uint2(0u, 0u);
        __syncwarp();
        const uint2 mine = s_cand[warp][lane];
        int rank = 0;
        for (int o = 0; o < total; o += 4) {
          const uint4 two = *reinterpret_cast<const uint4*>(&s_cand[warp][o]), more = *reinterpret_cast<const uint4*>(&s_cand[warp][o + 2]);
          rank += two.x > mine.x;
          rank += two.z > mine.x;
          rank += more.x > mine.x;
          rank += more.z > mine.x;
        }
        rank += __popc(__match_any_sync(kFull, mine.x) & ((1u << lane) - 1u));
        if (rank < rounds) ranked[rank] = mine;                  // the empty ones come last
      } else {
        for (int j = 0; j < rounds; ++j) {
          const uint32_t top = __reduce_max_sync(kFull, best);
          const int from = __ffs(__ballot_sync(kFull, best == top)) - 1;
          if (lane == from) {
            bool found = false;
            best = 0u;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
              if (!found && key[i] == top) {
                found = true;
                ranked[j] = make_uint2(top, uint32_t(base + i));
                key[i] = 0u;
              }
              best = max(best, key[i]);
            }
          }
        }
      }
      __syncwarp();
      if (MODE != 0 && has_bias) {
        const uint32_t ck = lane < rounds ? ranked[lane].x : 0u;
        const float c = key_float(ck), c_up = __shfl_up_sync(kFull, c, 1);
        if (__any_sync(kFull, lane >= 1 && lane <= p.k && ck != 0u && c_up - c <= tol + 2.4e-7f * fabsf(c_up))) close_rows |= 1u << r;
      }
    }
    if (MODE != 0 && (close_rows | unsure_rows) != 0u) {
      for (unsigned left = close_rows | unsure_rows; left != 0u; left &= left - 1u) {
        const int r = __ffs(left) - 1;
        const uint2 c = lane < rounds ? s_ranked[warp][r][lane] : make_uint2(0u, 0u);
        const int e = route_settle<Elem>(p, first + r, lane, c.x, int(c.y), rounds, __shfl_sync(kFull, my_tol, r * kPickLanes),
                                         close_rows >> r & 1, unsure_rows >> r & 1);
        if (lane < p.k) s_ranked[warp][r][lane].y = uint32_t(e);
        __syncwarp();
      }
      // Read again, so that nothing of a row's size is kept across the calls.
      fetch_bias();
      if (kAhead && first + stride < p.T) fetch(first + stride);
    }

    const int64_t row = first + lane / kPickLanes;
    const bool pick = lane / kPickLanes < rows && lane % kPickLanes < p.k;
    const int my_e = pick ? int(s_ranked[warp][lane / kPickLanes][lane % kPickLanes].y) : 0;
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
  if (gridDim.x > 1) {
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads)
      if (s_hist[e] != 0) atomicAdd(&p.counts[e], s_hist[e]);   // integers: any order gives the same sum
    return;
  }
  for (int e = threadIdx.x; e < p.E; e += kRouteThreads) {
    const int cnt = s_hist[e];
    p.counts[e] = cnt;
    if (p.bias_out != nullptr) {
      const int64_t over = p.T * p.k - int64_t(cnt) * p.E;
      const float b = has_bias ? p.bias[e] : 0.f;
      p.bias_out[e] = over > 0 ? b + p.bias_gamma : over < 0 ? b - p.bias_gamma : b;
    }
  }
}

// bias + gamma * sign(T*k/E - count), after all counts are in.
__global__ void __launch_bounds__(256) route_bias_kernel(const RouteParams p) {
  const int e = blockIdx.x * blockDim.x + threadIdx.x;
  if (e >= p.E) return;
  const int64_t over = p.T * p.k - int64_t(p.counts[e]) * p.E;
  const float b = p.bias != nullptr ? p.bias[e] : 0.f;
  p.bias_out[e] = over > 0 ? b + p.bias_gamma : over < 0 ? b - p.bias_gamma : b;
}

// Four rows a warp share the work on the picks; one row where that leaves fewer than
// 16 warps an SM.
int rows_per_warp(int64_t T, int sms) { return T >= int64_t(sms) * 64 ? 4 : 1; }

template <class Elem, int NV, int VB, bool FULL, int MODE>
cudaError_t fwd_launch(const RouteParams& p, int sms, cudaStream_t stream) {
  const size_t smem = size_t(p.E) * sizeof(int);
  if (p.T <= kRouteOneCtaRows) {
    route_fwd_kernel<Elem, NV, VB, FULL, MODE><<<1, kRouteThreads, smem, stream>>>(p, 1);
    return cudaGetLastError();
  }
  cudaError_t e = cudaMemsetAsync(p.counts, 0, smem, stream);
  if (e != cudaSuccess) return e;
  const int per = rows_per_warp(p.T, sms);
  const int64_t rows = int64_t(kRouteWarps) * per, want = (p.T + rows - 1) / rows;
  const int64_t most = int64_t(sms) * 8;
  route_fwd_kernel<Elem, NV, VB, FULL, MODE><<<int(want < most ? want : most), kRouteThreads, smem, stream>>>(p, per);
  if ((e = cudaGetLastError()) != cudaSuccess || p.bias_out == nullptr) return e;
  route_bias_kernel<<<(p.E + 255) / 256, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

template <class Elem, int NV, int MODE>
cudaError_t fwd_width(const RouteParams& p, int sms, cudaStream_t stream) {
  constexpr int kSize = int(sizeof(typename Elem::Raw)), kRow = NV * kSize;
  constexpr int VB = kRow % 16 == 0 ? 16 : kRow % 8 == 0 ? 8 : 4;
  // Loads of VB bytes: every lane has NV experts, and rows, groups and the array are aligned.
  const bool full = p.chunk == NV && p.gs == p.L * p.chunk;
  if (full && int64_t(p.E) * kSize % VB == 0 && reinterpret_cast<uintptr_t>(p.logits) % VB == 0)
    return fwd_launch<Elem, NV, VB, true, MODE>(p, sms, stream);
  return fwd_launch<Elem, NV, kSize, false, MODE>(p, sms, stream);
}

template <class Elem, int MODE>
cudaError_t fwd_mode(const RouteParams& p, int sms, cudaStream_t stream) {
  if (p.chunk <= 2) return fwd_width<Elem, 2, MODE>(p, sms, stream);
  if (p.chunk <= 4) return fwd_width<Elem, 4, MODE>(p, sms, stream);
  if (p.chunk <= 8) return fwd_width<Elem, 8, MODE>(p, sms, stream);
  if (p.chunk <= 12) return fwd_width<Elem, 12, MODE>(p, sms, stream);
  if (p.chunk <= 16) return fwd_width<Elem, 16, MODE>(p, sms, stream);
  if (p.chunk <= 32) return fwd_width<Elem, 32, MODE>(p, sms, stream);
  return fwd_launch<Elem, 64, int(sizeof(typename Elem::Raw)), false, MODE>(p, sms, stream);
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

// `per` rows a warp, lane 8 r + j with pick j of row r.
template <class Elem, bool VEC>
__global__ void __launch_bounds__(kRouteThreads) route_bwd_picks_kernel(const RouteBwdParams p, const int per) {
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  const int j = lane % kPickLanes;
  const int64_t stride = int64_t(gridDim.x) * kRouteWarps * per;
  for (int64_t first = (int64_t(blockIdx.x) * kRouteWarps + warp) * per; first < p.T; first += stride) {
    const int64_t row = first + lane / kPickLanes;
    const bool there = lane / kPickLanes < per && row < p.T && j < p.k;
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

template <class Elem, int NV>
__global__ void __launch_bounds__(kRouteThreads) route_bwd_softmax_kernel(const RouteBwdParams p) {
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
    const float inv = sum > 0.f ? 1.f / sum : 0.f;
    const float pp = zp > neg_inf() ? ex2_approx((zp - shift) * kLog2e) * inv : 0.f;
    float S = 0.f;                                       // sum_j p_j dg_j over the picks
    for (int j = 0; j < p.k; ++j) S += __shfl_sync(kFull, pp, j) * __shfl_sync(kFull, dg, j);
    const float v = pp * (sum_same(dg, e, p.k) - S);     // the lanes from 8 on have no pick
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

template <class Elem>
cudaError_t bwd_elem(const RouteBwdParams& p, int sms, cudaStream_t stream) {
  const bool picks = !p.softmax || p.renorm;
  const int per = picks ? rows_per_warp(p.T, sms) : 1;
  const int64_t rows = int64_t(kRouteWarps) * per, want = (p.T + rows - 1) / rows;
  const int64_t most = int64_t(sms) * 8;
  const int grid = int(want < most ? want : most);
  if (picks) {
    if (p.E % 4 == 0 && reinterpret_cast<uintptr_t>(p.dlogits) % 16 == 0)
      route_bwd_picks_kernel<Elem, true><<<grid, kRouteThreads, 0, stream>>>(p, per);
    else
      route_bwd_picks_kernel<Elem, false><<<grid, kRouteThreads, 0, stream>>>(p, per);
  } else if (p.E <= 4 * kWarp) {
    route_bwd_softmax_kernel<Elem, 4><<<grid, kRouteThreads, 0, stream>>>(p);
  } else if (p.E <= 8 * kWarp) {
    route_bwd_softmax_kernel<Elem, 8><<<grid, kRouteThreads, 0, stream>>>(p);
  } else if (p.E <= 12 * kWarp) {
    route_bwd_softmax_kernel<Elem, 12><<<grid, kRouteThreads, 0, stream>>>(p);
  } else {
    route_bwd_softmax_kernel<Elem, 32><<<grid, kRouteThreads, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace
}  // namespace moe
