// Host side of the C ABI declared in include/moe_experts.h: argument checks and launches.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>

#include "abi_common.h"
#include "expert_combine.h"
#include "expert_matmul.h"
#include "moe_experts.h"
#include "quantize.h"
#include "route.h"

namespace {

moe_status fail(moe_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
moe_status fail(moe_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return moe::abi_fail(s, buf);
}

moe_status launched(cudaError_t e, const char* what) {
  if (e == cudaSuccess) return MOE_OK;
  return fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

constexpr int64_t kInt32Limit = int64_t(1) << 31;

moe_status check_dtype(moe_dtype dt) {
  if (dt != MOE_DTYPE_FP32 && dt != MOE_DTYPE_BF16) return fail(MOE_ERR_UNSUPPORTED, "dtype %d is not fp32 (0) or bf16 (1)", int(dt));
  return MOE_OK;
}

moe_status check_tokens(int64_t T, int32_t k) {
  if (T < 1 || T >= kInt32Limit) return fail(MOE_ERR_INVALID, "T = %lld outside [1, 2^31)", (long long)T);
  if (k < 1 || k > MOE_MAX_TOPK) return fail(MOE_ERR_INVALID, "k = %d outside [1, %d]", k, MOE_MAX_TOPK);
  if (T * k >= kInt32Limit) return fail(MOE_ERR_INVALID, "T*k = %lld does not fit int32", (long long)(T * k));
  return MOE_OK;
}

moe_status check_experts(int32_t E) {
  if (E < 1 || E > MOE_MAX_EXPERTS) return fail(MOE_ERR_INVALID, "E = %d outside [1, %d]", E, MOE_MAX_EXPERTS);
  return MOE_OK;
}

// A row length of a quantised operand: whole 16-byte pieces, as its tiled copies need them.
moe_status check_width(const char* name, int64_t n) {
  if (n < 16 || n > MOE_MAX_WIDTH || n % 16 != 0)
    return fail(MOE_ERR_INVALID, "%s = %lld must be a multiple of 16 in [16, %d]", name, (long long)n, MOE_MAX_WIDTH);
  return MOE_OK;
}

moe_status check_rows(const char* name, int64_t n) {
  if (n < 1 || n >= kInt32Limit) return fail(MOE_ERR_INVALID, "%s = %lld outside [1, 2^31)", name, (long long)n);
  return MOE_OK;
}

moe_status check_gather(int64_t rows, int64_t M, const int32_t* perm, int32_t k) {
  moe_status s;
  if ((s = check_rows("rows", rows)) != MOE_OK || (s = check_rows("M", M)) != MOE_OK) return s;
  if (perm == nullptr && rows != M) return fail(MOE_ERR_INVALID, "without perm, rows = %lld must be M = %lld", (long long)rows, (long long)M);
  if (k < 1 || k > MOE_MAX_TOPK) return fail(MOE_ERR_INVALID, "k = %d outside [1, %d]", k, MOE_MAX_TOPK);
  if (!aligned(perm, 4)) return fail(MOE_ERR_INVALID, "perm is not 4-byte aligned");
  return MOE_OK;
}

}  // namespace

extern "C" {

int32_t moe_experts_abi_version(void) { return MOE_EXPERTS_ABI_VERSION; }

moe_status moe_route_fwd(const void* logits, moe_dtype dt, int64_t T, int32_t E, int32_t k,
                         moe_score score, int32_t n_groups, int32_t topk_groups, moe_group_score group_score,
                         const float* bias, int32_t renorm, float scale, float bias_gamma, float* bias_out,
                         int32_t* idx, float* gate, int32_t* counts, moe_stream_t stream) {
  moe_status s;
  if ((s = check_dtype(dt)) != MOE_OK || (s = check_tokens(T, k)) != MOE_OK || (s = check_experts(E)) != MOE_OK) return s;
  if (!logits || !idx || !gate || !counts) return fail(MOE_ERR_INVALID, "logits or an output is NULL");
  if (!aligned(logits, dt == MOE_DTYPE_BF16 ? 2 : 4) || !aligned(bias, 4) || !aligned(bias_out, 4) || !aligned(idx, 4) ||
      !aligned(gate, 4) || !aligned(counts, 4))
    return fail(MOE_ERR_INVALID, "an array is not element aligned");
  if (score != MOE_SCORE_SIGMOID && score != MOE_SCORE_SOFTMAX) return fail(MOE_ERR_INVALID, "score = %d is not 0 or 1", int(score));
  if (group_score != MOE_GROUP_MAX && group_score != MOE_GROUP_TOP2)
    return fail(MOE_ERR_INVALID, "group_score = %d is not 0 or 1", int(group_score));
  if (n_groups < 1 || n_groups > MOE_MAX_GROUPS || E % n_groups != 0)
    return fail(MOE_ERR_INVALID, "n_groups = %d must be in [1, %d] and divide E = %d", n_groups, MOE_MAX_GROUPS, E);
  if (topk_groups < 1 || topk_groups > n_groups) return fail(MOE_ERR_INVALID, "topk_groups = %d outside [1, %d]", topk_groups, n_groups);
  if (k > topk_groups * (E / n_groups))
    return fail(MOE_ERR_INVALID, "k = %d is more than the %d experts of %d groups", k, topk_groups * (E / n_groups), topk_groups);
  if (renorm < -1 || renorm > 1) return fail(MOE_ERR_INVALID, "renorm = %d is not -1, 0 or 1", renorm);
  if (!std::isfinite(scale)) return fail(MOE_ERR_INVALID, "scale must be finite");
  if (bias_out != nullptr && !std::isfinite(bias_gamma)) return fail(MOE_ERR_INVALID, "bias_gamma must be finite");
  int sms = 0;
  if ((s = moe::abi_sms(&sms)) != MOE_OK) return s;
  moe::RouteParams p = {};
  p.logits = logits;
  p.T = T;
  p.E = E;
  p.k = k;
  p.softmax = score == MOE_SCORE_SOFTMAX;
  p.G = n_groups;
  p.gs = E / n_groups;
  p.keep = topk_groups;
  p.top2 = group_score == MOE_GROUP_TOP2;
  p.L = 1;
  while (p.L * 2 * n_groups <= moe::kRouteLanes) p.L *= 2;
  p.chunk = (p.gs + p.L - 1) / p.L;
  p.bias = bias;
  p.renorm = renorm < 0 ? k > 1 : renorm;
  p.scale = scale;
  p.bias_gamma = bias_gamma;
  p.bias_out = bias_out;
  p.idx = idx;
  p.gate = gate;
  p.counts = counts;
  return launched(dt == MOE_DTYPE_BF16 ? moe::launch_route_fwd_bf16(p, sms, stream) : moe::launch_route_fwd_fp32(p, sms, stream), "moe_route_fwd launch");
}

moe_status moe_route_bwd(const void* logits, moe_dtype dt, int64_t T, int32_t E, int32_t k,
                         moe_score score, int32_t renorm, float scale,
                         const int32_t* idx, const float* dgate, float* dlogits, moe_stream_t stream) {
  moe_status s;
  if ((s = check_dtype(dt)) != MOE_OK || (s = check_tokens(T, k)) != MOE_OK || (s = check_experts(E)) != MOE_OK) return s;
  if (!logits || !idx || !dgate || !dlogits) return fail(MOE_ERR_INVALID, "an argument is NULL");
  if (!aligned(logits, dt == MOE_DTYPE_BF16 ? 2 : 4) || !aligned(idx, 4) || !aligned(dgate, 4) || !aligned(dlogits, 4))
    return fail(MOE_ERR_INVALID, "an array is not element aligned");
  if (score != MOE_SCORE_SIGMOID && score != MOE_SCORE_SOFTMAX) return fail(MOE_ERR_INVALID, "score = %d is not 0 or 1", int(score));
  if (renorm < -1 || renorm > 1) return fail(MOE_ERR_INVALID, "renorm = %d is not -1, 0 or 1", renorm);
  if (!std::isfinite(scale)) return fail(MOE_ERR_INVALID, "scale must be finite");
  int sms = 0;
  if ((s = moe::abi_sms(&sms)) != MOE_OK) return s;
  moe::RouteBwdParams p = {logits, T, E, k, score == MOE_SCORE_SOFTMAX, renorm < 0 ? k > 1 : renorm, scale, idx, dgate, dlogits};
  return launched(dt == MOE_DTYPE_BF16 ? moe::launch_route_bwd_bf16(p, sms, stream) : moe::launch_route_bwd_fp32(p, sms, stream), "moe_route_bwd launch");
}

moe_status moe_quantize_rows(const void* x, moe_dtype dt, int64_t rows, int64_t M, int32_t K,
                             const int32_t* perm, int32_t k, void* q, float* scale, moe_stream_t stream) {
  moe_status s;
  if ((s = check_dtype(dt)) != MOE_OK || (s = check_gather(rows, M, perm, k)) != MOE_OK || (s = check_width("K", K)) != MOE_OK) return s;
  if (!x || !q || !scale) return fail(MOE_ERR_INVALID, "an argument is NULL");
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4)) return fail(MOE_ERR_INVALID, "x or q is not 16-byte aligned");
  moe::QuantRowsParams p = {x, rows, M, K, k, perm, static_cast<uint8_t*>(q), scale};
  return launched(moe::launch_quantize_rows(p, dt == MOE_DTYPE_BF16, stream), "moe_quantize_rows launch");
}

int64_t moe_quantize_cols_width(int64_t M, int32_t E) {
  if (M < 1 || M >= kInt32Limit || E < 1 || E > MOE_MAX_EXPERTS) return -1;
  return (M + int64_t(MOE_SCALE_BLOCK - 1) * E) / MOE_SCALE_BLOCK * MOE_SCALE_BLOCK;
}

moe_status moe_quantize_cols(const void* x, moe_dtype dt, int64_t rows, int64_t M, int32_t K, int32_t E,
                             const int32_t* offsets, const int32_t* kept, const int32_t* perm, int32_t k,
                             void* q, float* scale, moe_stream_t stream) {
  moe_status s;
  if ((s = check_dtype(dt)) != MOE_OK || (s = check_gather(rows, M, perm, k)) != MOE_OK || (s = check_width("K", K)) != MOE_OK ||
      (s = check_experts(E)) != MOE_OK)
    return s;
  if (!x || !offsets || !q || !scale) return fail(MOE_ERR_INVALID, "an argument is NULL");
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 16)) return fail(MOE_ERR_INVALID, "x, q or scale is not 16-byte aligned");
  if (!aligned(offsets, 4) || !aligned(kept, 4)) return fail(MOE_ERR_INVALID, "offsets or kept is not 4-byte aligned");
  moe::QuantColsParams p = {x, rows, M, K, k, E, offsets, kept, perm, moe_quantize_cols_width(M, E), static_cast<uint8_t*>(q), scale};
  if (p.width >= kInt32Limit) return fail(MOE_ERR_INVALID, "M = %lld over E = %d experts is too wide", (long long)M, E);
  int sms = 0;
  if ((s = moe::abi_sms(&sms)) != MOE_OK) return s;
  return launched(moe::launch_quantize_cols(p, dt == MOE_DTYPE_BF16, sms, stream), "moe_quantize_cols launch");
}

moe_status moe_quantize_weights(const void* w, moe_dtype dt, int32_t E, int32_t N, int32_t K,
                                void* q, float* scale, void* qt, float* scalet, moe_stream_t stream) {
  moe_status s;
  if ((s = check_dtype(dt)) != MOE_OK || (s = check_experts(E)) != MOE_OK || (s = check_width("N", N)) != MOE_OK ||
      (s = check_width("K", K)) != MOE_OK)
    return s;
  if (!w || (!q && !qt)) return fail(MOE_ERR_INVALID, "w or both outputs are NULL");
  if ((q != nullptr) != (scale != nullptr) || (qt != nullptr) != (scalet != nullptr))
    return fail(MOE_ERR_INVALID, "codes and scales come in pairs");
  if (!aligned(w, 16) || !aligned(q, 16) || !aligned(qt, 16) || !aligned(scale, 4) || !aligned(scalet, 4))
    return fail(MOE_ERR_INVALID, "w, q or qt is not 16-byte aligned");
  moe::QuantWeightsParams p = {w, E, N, K, static_cast<uint8_t*>(q), scale, static_cast<uint8_t*>(qt), scalet};
  return launched(moe::launch_quantize_weights(p, dt == MOE_DTYPE_BF16, stream), "moe_quantize_weights launch");
}

moe_status moe_expert_matmul(const void* q, const float* scale, int64_t M, int32_t K,
                             const void* wq, const float* wscale, int32_t E, int32_t N,
                             const int32_t* offsets, const int32_t* kept, moe_dtype out_dt, void* out,
                             moe_stream_t stream) {
  moe_status s;
  if ((s = check_dtype(out_dt)) != MOE_OK || (s = check_rows("M", M)) != MOE_OK || (s = check_experts(E)) != MOE_OK ||
      (s = check_width("N", N)) != MOE_OK || (s = check_width("K", K)) != MOE_OK)
    return s;
  if (!q || !scale || !wq || !wscale || !out) return fail(MOE_ERR_INVALID, "an argument is NULL");
  if (offsets == nullptr && (E != 1 || kept != nullptr)) return fail(MOE_ERR_INVALID, "without offsets there is one expert and no kept");
  if (int64_t(E) * N >= kInt32Limit) return fail(MOE_ERR_INVALID, "E*N = %lld does not fit int32", (long long)E * N);
  if (!aligned(q, 16) || !aligned(wq, 16) || !aligned(out, 16)) return fail(MOE_ERR_INVALID, "q, wq or out is not 16-byte aligned");
  if (!aligned(scale, 4) || !aligned(wscale, 4) || !aligned(offsets, 4) || !aligned(kept, 4))
    return fail(MOE_ERR_INVALID, "an array is not 4-byte aligned");
  // the tiles of the launch are counted in int32
  if ((M / 128 + E) * ((N + 127) / 128) >= kInt32Limit)
    return fail(MOE_ERR_INVALID, "M = %lld by N = %d is too large", (long long)M, N);
  int sms = 0;
  if ((s = moe::abi_sms(&sms)) != MOE_OK) return s;
  moe::MatmulParams p = {};
  p.M = M;
  p.C = N;
  p.K = K;
  p.E = E;
  p.a = static_cast<const uint8_t*>(q);
  p.a_scale = scale;
  p.b = static_cast<const uint8_t*>(wq);
  p.b_scale = wscale;
  p.offsets = offsets;
  p.kept = kept;
  p.out_bf16 = out_dt == MOE_DTYPE_BF16;
  p.out = out;
  p.timeout_ns = moe::abi_wait_ns();
  p.extra = moe::abi_barrier_extra();
  const char* error = nullptr;
  const cudaError_t e = moe::launch_expert_matmul(p, sms, &error, stream);
  return error ? fail(MOE_ERR_CUDA, "moe_expert_matmul: %s", error) : launched(e, "moe_expert_matmul launch");
}

moe_status moe_expert_wgrad(const void* dyq, const float* dyscale, const void* xq, const float* xscale,
                            int64_t width, int32_t N, int32_t K, int32_t E, const int32_t* kept, float* dw,
                            moe_stream_t stream) {
  moe_status s;
  if ((s = check_experts(E)) != MOE_OK || (s = check_width("N", N)) != MOE_OK || (s = check_width("K", K)) != MOE_OK)
    return s;
  if (width < MOE_SCALE_BLOCK || width >= kInt32Limit || width % MOE_SCALE_BLOCK != 0)
    return fail(MOE_ERR_INVALID, "width = %lld must be a multiple of 128 in [128, 2^31)", (long long)width);
  if (!dyq || !dyscale || !xq || !xscale || !kept || !dw) return fail(MOE_ERR_INVALID, "an argument is NULL");
  if (!aligned(dyq, 16) || !aligned(xq, 16) || !aligned(dw, 16)) return fail(MOE_ERR_INVALID, "dyq, xq or dw is not 16-byte aligned");
  if (!aligned(xscale, 16) || !aligned(dyscale, 16) || !aligned(kept, 4))
    return fail(MOE_ERR_INVALID, "xscale, dyscale (16 bytes) or kept (4 bytes) is misaligned");
  if (int64_t(E) * ((N + 127) / 128) * ((K + 127) / 128) >= kInt32Limit) return fail(MOE_ERR_INVALID, "E x N x K is too large");
  int sms = 0;
  if ((s = moe::abi_sms(&sms)) != MOE_OK) return s;
  moe::MatmulParams p = {};
  p.wgrad = 1;
  p.R = N;
  p.C = K;
  p.E = E;
  p.blocks = width / MOE_SCALE_BLOCK;
  p.a = static_cast<const uint8_t*>(dyq);
  p.a_scale = dyscale;
  p.b = static_cast<const uint8_t*>(xq);
  p.b_scale = xscale;
  p.kept = kept;
  p.out = dw;
  p.timeout_ns = moe::abi_wait_ns();
  p.extra = moe::abi_barrier_extra();
  const char* error = nullptr;
  const cudaError_t e = moe::launch_expert_matmul(p, sms, &error, stream);
  return error ? fail(MOE_ERR_CUDA, "moe_expert_wgrad: %s", error) : launched(e, "moe_expert_wgrad launch");
}

moe_status moe_expert_device_status(moe_stream_t stream, int32_t* flags) {
  if (!flags) return fail(MOE_ERR_INVALID, "flags is NULL");
  *flags = 0;
  int bits = 0;
  const cudaError_t e = moe::expert_matmul_errors(&bits, stream);
  if (e != cudaSuccess) return launched(e, "moe_expert_device_status");
  *flags = bits;
  return bits == 0 ? MOE_OK : fail(MOE_ERR_TIMEOUT, "a device wait of an expert product expired (flags %d)", bits);
}

moe_status moe_expert_combine(const void* y, moe_dtype dt, int64_t M, int32_t H, int64_t T, int32_t k, int32_t E,
                              const int32_t* idx, const int32_t* slot, const int32_t* offsets, const float* gate,
                              void* out, moe_stream_t stream) {
  moe_status s;
  if ((s = check_dtype(dt)) != MOE_OK || (s = check_tokens(T, k)) != MOE_OK || (s = check_experts(E)) != MOE_OK ||
      (s = check_rows("M", M)) != MOE_OK)
    return s;
  if (H < 1 || H > MOE_MAX_WIDTH) return fail(MOE_ERR_INVALID, "H = %d outside [1, %d]", H, MOE_MAX_WIDTH);
  if (!y || !idx || !slot || !offsets || !out) return fail(MOE_ERR_INVALID, "an argument is NULL");
  const size_t esize = dt == MOE_DTYPE_BF16 ? 2 : 4;
  if (!aligned(y, esize) || !aligned(out, esize) || !aligned(idx, 4) || !aligned(slot, 4) || !aligned(offsets, 4) || !aligned(gate, 4))
    return fail(MOE_ERR_INVALID, "an array is not element aligned");
  int sms = 0;
  if ((s = moe::abi_sms(&sms)) != MOE_OK) return s;
  moe::CombineRowsParams p = {y, T, M, H, k, E, idx, slot, offsets, gate, out};
  return launched(moe::launch_expert_combine(p, dt == MOE_DTYPE_BF16, sms, stream), "moe_expert_combine launch");
}

moe_status moe_expert_combine_bwd(const void* dout, const void* y, moe_dtype dt, int64_t M, int32_t H, int64_t T,
                                  int32_t k, int32_t E, const int32_t* idx, const int32_t* slot,
                                  const int32_t* offsets, const float* gate, void* dy, float* dgate,
                                  moe_stream_t stream) {
  moe_status s;
  if ((s = check_dtype(dt)) != MOE_OK || (s = check_tokens(T, k)) != MOE_OK || (s = check_experts(E)) != MOE_OK ||
      (s = check_rows("M", M)) != MOE_OK)
    return s;
  if (H < 1 || H > MOE_MAX_WIDTH) return fail(MOE_ERR_INVALID, "H = %d outside [1, %d]", H, MOE_MAX_WIDTH);
  if (!dout || !y || !idx || !slot || !offsets || !gate || !dy || !dgate) return fail(MOE_ERR_INVALID, "an argument is NULL");
  const size_t esize = dt == MOE_DTYPE_BF16 ? 2 : 4;
  if (!aligned(dout, esize) || !aligned(y, esize) || !aligned(dy, esize) || !aligned(idx, 4) || !aligned(slot, 4) ||
      !aligned(offsets, 4) || !aligned(gate, 4) || !aligned(dgate, 4))
    return fail(MOE_ERR_INVALID, "an array is not element aligned");
  int sms = 0;
  if ((s = moe::abi_sms(&sms)) != MOE_OK) return s;
  moe::CombineRowsBwdParams p = {dout, y, T, M, H, k, E, idx, slot, offsets, gate, dy, dgate};
  return launched(moe::launch_expert_combine_bwd(p, dt == MOE_DTYPE_BF16, sms, stream), "moe_expert_combine_bwd launch");
}

}  // extern "C"
