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

// Descending order of NV keys: Batcher's merge exchange, unrolled.
template <int NV>
__device__ __forceinline__ void sort_keys(unsigned long long (&v)[NV]) {
  constexpr int N = NV <= 4 ? 4 : NV <= 8 ? 8 : NV <= 16 ? 16 : NV <= 32 ? 32 : 64;
#pragma unroll
  for (int p = 1; p < N; p *= 2) {
#pragma unroll
    for (int q = p; q >= 1; q /= 2) {
#pragma unroll
      for (int a = 0; a < NV; ++a) {
        const int b = a + q;
        // pairs a, a + q whose distance from q % p falls into even runs of q, inside one block of 2p
        if (b < NV && a >= q % p && (a - q % p) / q % 2 == 0 && a / (2 * p) == b / (2 * p)) {
          const unsigned long long x = v[a], y = v[b];
          const bool swap = x < y;
          v[a] = swap ? y : x;
          v[b] = swap ? x : y;
        }
      }
    }
  }
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
// Forward.  NV: experts per lane, at least `chunk`; VB: bytes per load.
//
// A lane sorts its experts' keys (value above the inverted place, so that ties
// stand in expert order) into shared memory; a pick is then the largest head of
// the 32 lists (one warp reduction, the lowest lane that has it), whose lane
// goes on to its next entry.  With a bias two more than the k picks are taken,
// to see what hangs on rounding.  A warp selects for `per` rows one after another and then
// computes the gates of all of them, a pick a lane.
// ---------------------------------------------------------------------------
constexpr int kMaxRounds = 10;                                   // 8 picks and two more

template <class Elem, int NV, int VB>
__global__ void __launch_bounds__(kRouteThreads) route_fwd_kernel(const __grid_constant__ RouteParams p, const int per) {
  using Raw = typename Elem::Raw;
  constexpr int kPer = VB / int(sizeof(Raw));                    // elements per load
  constexpr int kList = NV < kMaxRounds ? NV : kMaxRounds;
  __shared__ unsigned long long s_list[kRouteWarps][kList][kWarp];
  extern __shared__ int s_hist[];                                // [E]
  const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
  for (int e = threadIdx.x; e < p.E; e += kRouteThreads) s_hist[e] = 0;
  __syncthreads();

  const int g = lane / p.L, sub = lane % p.L;
  const int base = g * p.gs + sub * p.chunk;
  const int n = g < p.G ? max(0, min(p.chunk, p.gs - sub * p.chunk)) : 0;
  const bool has_bias = p.bias != nullptr;
  const bool grouped = p.keep < p.G;
  const bool all_scores = has_bias || (p.top2 && grouped) || (p.softmax && !p.renorm);
  const int rounds = has_bias ? p.k + 2 : p.k;
  float bv[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) bv[i] = has_bias && i < n ? p.bias[base + i] : 0.f;

  const int64_t stride = int64_t(gridDim.x) * kRouteWarps * per;
  for (int64_t first = (int64_t(blockIdx.x) * kRouteWarps + warp) * per; first < p.T; first += stride) {
    int my_e = 0;                                                // lane 8 r + j: pick j of row first + r
    float my_max = 0.f, my_sum = 1.f;                            // and that row's softmax
    for (int r = 0; r < per && first + r < p.T; ++r) {
      const int64_t row = first + r;
      float z[NV];
      const Raw* src = static_cast<const Raw*>(p.logits) + row * p.E + base;
#pragma unroll
      for (int v = 0; v < NV / kPer; ++v) {
        alignas(16) Raw raw[kPer];
        if (v * kPer < n) {                                      // vector loads only where every lane's n is a multiple
          if constexpr (VB == 16) *reinterpret_cast<uint4*>(raw) = *reinterpret_cast<const uint4*>(src + v * kPer);
          else if constexpr (VB == 8) *reinterpret_cast<uint2*>(raw) = *reinterpret_cast<const uint2*>(src + v * kPer);
          else raw[0] = src[v];
        } else {
#pragma unroll
          for (int i = 0; i < kPer; ++i) raw[i] = Elem::kNegInf;
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const float x = __uint_as_float(Elem::bits(raw[i]));
          z[v * kPer + i] = x == x ? x : neg_inf();              // not a number: never preferred
        }
      }

      // Scores in fp32.  Their error is within tol / 2.
      float s[NV], tol = 0.f;
      if (all_scores) {
        if (p.softmax) {
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
          if (lane / kPickLanes == r) {
            my_max = row_max;
            my_sum = sum;
          }
          // x e^-x <= 0.37: the rounded argument moves a score by 2^-23 * 0.37 * 1.45 of
          // the row's largest, ex2.approx by 2^-22 of itself, the sum of at most 64
          // values a lane and 5 steps by 69 * 2^-24 of itself: 5e-6 covers them
          tol = 1e-5f * inv;
        } else {
#pragma unroll
          for (int i = 0; i < NV; ++i) s[i] = rcp_approx(1.f + ex2_approx(z[i] * -kLog2e));
          // e = exp(-z) is off by 2^-22 + 2^-24 * 1.45 |z| of itself; s moves by
          // s (1 - s) of that, below 2^-23, and rcp.approx and 1 + e by 2^-22 of s: 6e-7 covers them
          tol = 1.2e-6f;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] = z[i] > neg_inf() ? s[i] + bv[i] : neg_inf();
      }
      uint32_t key[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) key[i] = i < n ? float_key((has_bias ? s[i] : z[i]) + 0.f) : 0u;

      bool unsure = false;                                       // whether the choice of groups hangs on rounding
      if (grouped) {
        uint32_t gkey;
        float gtol = tol;
        if (p.top2) {
          float a = neg_inf(), b = neg_inf();
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const float v = i < n ? s[i] : neg_inf();
            b = fmaxf(b, fminf(a, v));
            a = fmaxf(a, v);
          }
          for (int off = 1; off < p.L; off <<= 1) {
            const float a2 = __shfl_xor_sync(kFull, a, off), b2 = __shfl_xor_sync(kFull, b, off);
            b = fmaxf(fminf(a, a2), fmaxf(b, b2));
            a = fmaxf(a, a2);
          }
          gkey = g < p.G ? float_key((b > neg_inf() ? a + b : a) + 0.f) : 0u;
          gtol = 2.f * tol;
        } else {
          gkey = key[0];
#pragma unroll
          for (int i = 1; i < NV; ++i) gkey = max(gkey, key[i]);
          for (int off = 1; off < p.L; off <<= 1) gkey = max(gkey, __shfl_xor_sync(kFull, gkey, off));
        }
        int rank = 0;
        for (int o = 0; o < p.G; ++o) {
          const uint32_t other = __shfl_sync(kFull, gkey, o * p.L);
          rank += other > gkey || (other == gkey && o < g);
        }
        const bool kept = rank < p.keep;
        if (has_bias || p.top2) {
          const float lo = key_float(__reduce_min_sync(kFull, kept && g < p.G ? gkey : 0xffffffffu));
          const float hi = key_float(__reduce_max_sync(kFull, kept || g >= p.G ? 0u : gkey));
          unsure = lo - hi <= gtol + 4.8e-7f * fabsf(lo);        // + the sums' own roundings
        }
        if (!kept)
#pragma unroll
          for (int i = 0; i < NV; ++i) key[i] = 0u;
      }

      unsigned long long v[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = (unsigned long long)(key[i]) << 32 | uint32_t(~i);
      sort_keys<NV>(v);
#pragma unroll
      for (int i = 1; i < kList; ++i) s_list[warp][i][lane] = v[i];
      uint32_t head = uint32_t(v[0] >> 32), place = ~uint32_t(v[0]);
      int next = 1;
      uint32_t ck = 0;                                           // lane j: the j-th largest key and its expert
      int ce = 0;
      bool close = false;
      float prev = __uint_as_float(0x7f800000u);
      for (int j = 0; j < rounds; ++j) {
        const uint32_t top = __reduce_max_sync(kFull, head);
        const int from = __ffs(__ballot_sync(kFull, head == top)) - 1;
        const int e = __shfl_sync(kFull, base + int(place), from);
        if (lane == j) {
          ck = top;
          ce = e;
        }
        if (lane == from) {
          const unsigned long long w = next < kList ? s_list[warp][next][lane] : 0ull;
          head = uint32_t(w >> 32);
          place = ~uint32_t(w);
          ++next;
        }
        if (has_bias && j <= p.k) {
          const float c = key_float(top);
          close |= top != 0u && prev - c <= tol + 2.4e-7f * fabsf(prev);
          prev = c;
        }
      }
      if (close || unsure) {
        // Values next to one another: sure all the same where their inputs are equal.
        const bool there = lane < rounds && ck != 0u;
        const float zc = there ? load_logit<Elem>(p.logits, row * p.E + ce) : neg_inf();
        const float bc = there && has_bias ? p.bias[ce] : 0.f, c = key_float(ck);
        const float c_up = __shfl_up_sync(kFull, c, 1), z_up = __shfl_up_sync(kFull, zc, 1), b_up = __shfl_up_sync(kFull, bc, 1);
        const bool open = close && lane >= 1 && lane <= p.k && there && c_up - c <= tol + 2.4e-7f * fabsf(c_up) &&
                          !(zc == z_up && bc == b_up);
        const float last = __shfl_sync(kFull, c, p.k - 1);
        const bool beyond = lane == p.k + 1 && there && last - c <= tol + 2.4e-7f * fabsf(last);
        const bool any_open = __any_sync(kFull, open), any_beyond = __any_sync(kFull, beyond);
        if (unsure || (any_open && (any_beyond || p.softmax))) {
          ce = route_row_double<Elem>(p, row, lane);
        } else if (any_open) {
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
          ce = to;
        }
      }
      const int pe = __shfl_sync(kFull, ce, lane % kPickLanes);
      if (lane / kPickLanes == r) my_e = pe;
      __syncwarp();                                              // the lists are read before the next row's are written
    }

    const int64_t row = first + lane / kPickLanes;
    const bool pick = lane / kPickLanes < per && row < p.T && lane % kPickLanes < p.k;
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

template <class Elem, int NV, int VB>
cudaError_t fwd_launch(const RouteParams& p, int sms, cudaStream_t stream) {
  const size_t smem = size_t(p.E) * sizeof(int);
  if (p.T <= kRouteOneCtaRows) {
    route_fwd_kernel<Elem, NV, VB><<<1, kRouteThreads, smem, stream>>>(p, 1);
    return cudaGetLastError();
  }
  cudaError_t e = cudaMemsetAsync(p.counts, 0, smem, stream);
  if (e != cudaSuccess) return e;
  const int per = rows_per_warp(p.T, sms);
  const int64_t rows = int64_t(kRouteWarps) * per, want = (p.T + rows - 1) / rows;
  const int64_t most = int64_t(sms) * 8;
  route_fwd_kernel<Elem, NV, VB><<<int(want < most ? want : most), kRouteThreads, smem, stream>>>(p, per);
  if ((e = cudaGetLastError()) != cudaSuccess || p.bias_out == nullptr) return e;
  route_bias_kernel<<<(p.E + 255) / 256, 256, 0, stream>>>(p);
  return cudaGetLastError();
}

template <class Elem, int NV>
cudaError_t fwd_width(const RouteParams& p, int sms, cudaStream_t stream) {
  constexpr int kSize = int(sizeof(typename Elem::Raw));
  // A load of VB bytes needs every lane's first expert on a multiple of VB and
  // whole vectors: full groups and chunks, rows and the array aligned.
  const bool full = p.gs == p.L * p.chunk;
  const auto fits = [&](int vb) {
    return full && p.chunk * kSize % vb == 0 && p.gs * kSize % vb == 0 && int64_t(p.E) * kSize % vb == 0 &&
           reinterpret_cast<uintptr_t>(p.logits) % vb == 0;
  };
  if constexpr (NV * kSize % 16 == 0)
    if (fits(16)) return fwd_launch<Elem, NV, 16>(p, sms, stream);
  if constexpr (NV * kSize % 8 == 0)
    if (fits(8)) return fwd_launch<Elem, NV, 8>(p, sms, stream);
  return fwd_launch<Elem, NV, kSize>(p, sms, stream);
}

template <class Elem>
cudaError_t fwd_elem(const RouteParams& p, int sms, cudaStream_t stream) {
  if (p.chunk <= 4) return fwd_width<Elem, 4>(p, sms, stream);
  if (p.chunk <= 8) return fwd_width<Elem, 8>(p, sms, stream);
  if (p.chunk <= 12) return fwd_width<Elem, 12>(p, sms, stream);
  if (p.chunk <= 16) return fwd_width<Elem, 16>(p, sms, stream);
  if (p.chunk <= 32) return fwd_width<Elem, 32>(p, sms, stream);
  return fwd_width<Elem, 64>(p, sms, stream);
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

cudaError_t launch_route_fwd(const RouteParams& p, bool bf16, int sms, cudaStream_t stream) {
  return bf16 ? fwd_elem<Bf16>(p, sms, stream) : fwd_elem<Fp32>(p, sms, stream);
}

cudaError_t launch_route_bwd(const RouteBwdParams& p, bool bf16, int sms, cudaStream_t stream) {
  return bf16 ? bwd_elem<Bf16>(p, sms, stream) : bwd_elem<Fp32>(p, sms, stream);
}

}  // namespace moe
