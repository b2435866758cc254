/*
 * moe_experts.h -- C ABI of the expert side of the GB300 (sm_103a) MoE library:
 * what a mixture-of-experts layer does around the router and the dispatch of
 * moe_router.h.
 *
 *   moe_route_fwd / moe_route_bwd   scored, group-limited routing (sigmoid or
 *                                   softmax scores, a balance bias, groups of
 *                                   experts, top-k, renormalised gates)
 *   moe_quantize_rows / _cols / _weights
 *                                   e4m3 values with one scale for a block of 128
 *   moe_expert_matmul / moe_expert_wgrad
 *                                   the experts' matrix products on such values,
 *                                   and their weight gradient
 *   moe_expert_combine / _bwd       the experts' rows summed by gate, and its gradient
 *
 * A layer's forward: moe_route_fwd, moe_dispatch (moe_router.h), then
 * moe_quantize_rows with the dispatch's perm, moe_expert_matmul, the caller's
 * activation, moe_quantize_rows, moe_expert_matmul, moe_expert_combine.  Its
 * backward: moe_expert_combine_bwd; moe_quantize_rows and moe_expert_matmul
 * with the transposed weights for the data gradient, moe_quantize_cols of both
 * sides and moe_expert_wgrad for the weights'; moe_expert_combine with gate =
 * NULL sums a token's input gradients; moe_route_bwd takes the gates'.
 *
 * The conventions are those of moe_router.h: device pointers, dense row-major
 * arrays, work queued on `stream` without synchronising, argument errors found
 * on the host before anything is queued, moe_status results, moe_last_error().
 * Device arrays that hold positions (idx, slot, perm, offsets, kept) are those
 * that moe_route_fwd and moe_dispatch write; other values give unspecified
 * results, but no access leaves the arrays.  Calls can be captured into graphs.
 */
#ifndef MOE_EXPERTS_H
#define MOE_EXPERTS_H

#include "moe_router.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_EXPERTS_ABI_VERSION 1
MOE_API int32_t moe_experts_abi_version(void);

typedef enum { MOE_SCORE_SIGMOID = 0, MOE_SCORE_SOFTMAX = 1 } moe_score;
typedef enum { MOE_GROUP_MAX = 0, MOE_GROUP_TOP2 = 1 } moe_group_score;
#define MOE_MAX_GROUPS 32
/* Values that share a scale, along the contraction (and across it for weights). */
#define MOE_SCALE_BLOCK 128
/* Largest row length of the quantised operands. */
#define MOE_MAX_WIDTH (1 << 20)

/* ------------------------------------------------------------------------ */
/* Scored, group-limited routing                                            */
/* ------------------------------------------------------------------------ */

/* Per row t of logits z [T,E] (fp32 or bf16):
 *   s[e]    = sigmoid(z[e])  or  softmax(z)[e]
 *   c[e]    = s[e] + bias[e]: the choice value (bias NULL: s[e])
 *   groups  : E / n_groups consecutive experts each; a group's score is its
 *             largest choice value (MOE_GROUP_MAX) or the sum of its two
 *             largest (MOE_GROUP_TOP2; the one there is when only one expert of
 *             the group is not masked); the topk_groups best groups are kept
 *   idx[j]  : the k largest choice values in the kept groups, largest first
 *   gate[j] = scale * s[idx[j]], divided by sum_j s[idx[j]] when renorm (1: yes,
 *             0: no, -1: when k > 1)
 *   counts[e] = number of assignments to e over the batch
 *   bias_out[e] = bias[e] + bias_gamma * sign(T*k/E - counts[e])   (bias_out may
 *             be NULL, or bias itself; the sign from an exact integer
 *             comparison, one fp32 addition)
 * Ties go to the lower expert or group index.  Choice values and group scores
 * are compared as double precision orders them (values that fp32 cannot tell
 * apart with certainty are evaluated again in double); without a bias, scores
 * are in the order of their logits.  Renormalised gates keep their digits where
 * the scores underflow.
 * A logit of -infinity or NaN masks its expert: score 0, and picked (with gate
 * 0) only after every other expert of the kept groups.  In a row whose picks
 * are all masked every gate is 0.  A logit of +infinity gives unspecified
 * results.  The bias must be finite.
 *
 * T >= 1, T*k < 2^31; E in [1,1024]; k in [1,8]; n_groups in [1,32] dividing E;
 * topk_groups in [1,n_groups] with k <= topk_groups * E / n_groups.
 * logits is element aligned.  No workspace.  Results do not depend on T or on
 * the run: repeated calls give the same bits. */
MOE_API moe_status moe_route_fwd(const void* logits, moe_dtype dt, int64_t T, int32_t E, int32_t k,
                                 moe_score score, int32_t n_groups, int32_t topk_groups, moe_group_score group_score,
                                 const float* bias, int32_t renorm, float scale, float bias_gamma, float* bias_out,
                                 int32_t* idx, float* gate, int32_t* counts, moe_stream_t stream);

/* Gradient of sum_{t,j} dgate[t,j] * gate[t,j] with respect to the logits, the
 * picks held constant (the choice, its bias and its groups carry no gradient):
 *   sigmoid, renorm:  w_i = s_i / sum_j s_j:  scale * w_i (1 - s_i) (dgate_i - sum_j w_j dgate_j) at the picks
 *   sigmoid:          scale * s_i (1 - s_i) dgate_i at the picks
 *   softmax, renorm:  scale * w_i (dgate_i - sum_j w_j dgate_j) at the picks
 *   softmax:          scale * (s_i [i picked] dgate_i - s_i sum_j s_j dgate_j) for every i
 * and 0 elsewhere.  An expert picked twice gets the sum; an idx outside [0,E)
 * contributes nothing.  Masked logits get 0.  dlogits [T,E] fp32 is written
 * whole, not accumulated. */
MOE_API moe_status moe_route_bwd(const void* logits, moe_dtype dt, int64_t T, int32_t E, int32_t k,
                                 moe_score score, int32_t renorm, float scale,
                                 const int32_t* idx, const float* dgate, float* dlogits, moe_stream_t stream);

/* ------------------------------------------------------------------------ */
/* e4m3 values with one scale for a block of 128                            */
/* ------------------------------------------------------------------------ */

/* A block's scale is the power of two s with 224 < max|x| / s <= 448 (at least
 * 2^-126; 1 for a block of zeros); its codes are x / s rounded to nearest, ties
 * to even.  A block with an infinity or a NaN gets the scale NaN (its codes are
 * unspecified), so that every product with it is NaN.
 * x is fp32 or bf16, 16-byte aligned; row lengths are multiples of 16, up to
 * MOE_MAX_WIDTH. */

/* Blocks of 1 x 128.  q [M,K]: row r holds row perm[r] / k of x [rows,K] (the
 * gather of the token rows in dispatch order), or row r when perm is NULL (then
 * M == rows).  scale [ceil(K/128), M]: the scales of one block column lie
 * together.  A perm entry outside [0, rows*k) gives a row of zeros. */
MOE_API moe_status moe_quantize_rows(const void* x, moe_dtype dt, int64_t rows, int64_t M, int32_t K,
                                     const int32_t* perm, int32_t k, void* q, float* scale, moe_stream_t stream);

/* Blocks of 128 x 1 along the rows of each expert, written transposed: the
 * operands of moe_expert_wgrad, whose contraction runs over an expert's rows.
 * Expert e's rows are those of moe_expert_matmul; they lie in columns
 * 128 * sum_{e'<e} ceil(n_e'/128) and following of q [K,width], n_e = kept[e],
 * its last block filled up with zeros; scale [width/128, K].  Columns behind the
 * last expert's are left as they are.  width = moe_quantize_cols_width(M, E) =
 * 128 * floor((M + 127 E) / 128), which holds any split of M rows.  Rows are
 * gathered by perm as in moe_quantize_rows; offsets and kept as in
 * moe_expert_matmul (kept may be NULL: every row).  x, q and scale are 16-byte
 * aligned. */
MOE_API int64_t moe_quantize_cols_width(int64_t M, int32_t E);
MOE_API moe_status moe_quantize_cols(const void* x, moe_dtype dt, int64_t rows, int64_t M, int32_t K, int32_t E,
                                     const int32_t* offsets, const int32_t* kept, const int32_t* perm, int32_t k,
                                     void* q, float* scale, moe_stream_t stream);

/* Blocks of 128 x 128 of w [E,N,K].  q [E,N,K] with scale
 * [E, ceil(N/128), ceil(K/128)], and/or the transposed qt [E,K,N] with scalet
 * [E, ceil(K/128), ceil(N/128)] (the same codes and scales: the operand of the
 * data gradient).  Either pair may be NULL. */
MOE_API moe_status moe_quantize_weights(const void* w, moe_dtype dt, int32_t E, int32_t N, int32_t K,
                                        void* q, float* scale, void* qt, float* scalet, moe_stream_t stream);

/* ------------------------------------------------------------------------ */
/* The experts' matrix products                                             */
/* ------------------------------------------------------------------------ */

/* out[r,n] = sum_k a[r,k] w[e,n,k] for the rows r = offsets[e] ..
 * offsets[e] + n_e - 1 of every expert e, n_e = kept[e] (or all rows up to
 * offsets[e+1] with kept NULL).  Other rows of out are left as they are.
 * offsets NULL: one expert (E == 1) with all M rows, a plain product.  The
 * experts' ranges are disjoint; a row that two share holds results of either.
 *   q [M,K] e4m3, scale [ceil(K/128), M] fp32: as moe_quantize_rows
 *   wq [E,N,K] e4m3, wscale [E, ceil(N/128), ceil(K/128)] fp32: as moe_quantize_weights
 *   out [M,N] bf16 or fp32 (out_dt)
 * Scales may be any fp32 numbers.  Rows that meet a product of two scales outside
 * fp32's normal numbers (2^-126 to 2^128) are computed once more from the operands,
 * which takes longer: all rows some 30 times as long.
 * A block's 128 products are summed by the tensor core in fp32 (where products below
 * about 2^-25 of the block's largest may be lost), the blocks in fp32 registers, in
 * order; the one rounding to bf16 is at the end.  A row's result does not depend on
 * the other rows.
 * The data gradient is the same call with dy's rows and the transposed weights.
 * K and N are multiples of 16 up to MOE_MAX_WIDTH, E * N < 2^31, M >= 1, M < 2^31;
 * q, wq and out are 16-byte aligned.
 * Needs no workspace.  A device wait that runs out is reported by
 * moe_expert_device_status, and until that is read later calls on the device
 * write nothing. */
MOE_API moe_status moe_expert_matmul(const void* q, const float* scale, int64_t M, int32_t K,
                                     const void* wq, const float* wscale, int32_t E, int32_t N,
                                     const int32_t* offsets, const int32_t* kept, moe_dtype out_dt, void* out,
                                     moe_stream_t stream);

/* dw[e,n,k] = sum over expert e's rows r of dy[r,n] x[r,k], fp32, written whole
 * (zeros for an expert without rows).
 *   dyq [N,width], dyscale [width/128, N] and xq [K,width], xscale [width/128, K]:
 *   moe_quantize_cols of the rows of dy and x with the same offsets and kept
 *   kept [E]: the rows of each expert
 * Sums and scales as in moe_expert_matmul (a scale of dy outside 2^-108 to 2^103
 * takes the longer way).  K and N as there; width is a multiple of 128
 * below 2^31; all arrays but kept are 16-byte aligned. */
MOE_API moe_status moe_expert_wgrad(const void* dyq, const float* dyscale, const void* xq, const float* xscale,
                                    int64_t width, int32_t N, int32_t K, int32_t E, const int32_t* kept, float* dw,
                                    moe_stream_t stream);

/* Reads and clears the error bits that moe_expert_matmul and moe_expert_wgrad
 * calls have left on the current device (synchronises `stream`, on which they
 * were queued).  *flags = 0 when every wait completed; otherwise returns
 * MOE_ERR_TIMEOUT with bit 2 set: a wait of a kernel's pipeline expired and its
 * output is incomplete.  Bits are read and cleared in one step: each is given to one
 * reader, whichever stream its call ran on. */
MOE_API moe_status moe_expert_device_status(moe_stream_t stream, int32_t* flags);

/* ------------------------------------------------------------------------ */
/* The experts' rows back to their tokens                                   */
/* ------------------------------------------------------------------------ */

/* out[t,:] = sum_j gate[t,j] * y[offsets[idx[t,j]] + slot[t*k+j], :] over the
 * assignments with slot >= 0; a token without any gets zeros.  gate NULL: ones
 * (the plain sum: the gradient of gathering a token's row for its k experts).
 * y [M,H] and out [T,H] fp32 or bf16 (dt); idx, gate [T,k]; slot [T*k], offsets
 * [E+1] of moe_dispatch.  Sums are fp32, in the order of j.  H >= 1, k in [1,8];
 * y and out are element aligned. */
MOE_API moe_status moe_expert_combine(const void* y, moe_dtype dt, int64_t M, int32_t H, int64_t T, int32_t k, int32_t E,
                                      const int32_t* idx, const int32_t* slot, const int32_t* offsets, const float* gate,
                                      void* out, moe_stream_t stream);

/* Its gradients: dy[row,:] = gate[t,j] * dout[t,:] for the rows of kept
 * assignments (others are left as they are), dgate[t,j] = sum_h dout[t,h] y[row,h]
 * (0 for a dropped assignment).  dy has y's type, dgate is fp32.  The rows of
 * kept assignments are distinct, as moe_dispatch makes them; one that two share
 * holds values of either. */
MOE_API moe_status moe_expert_combine_bwd(const void* dout, const void* y, moe_dtype dt, int64_t M, int32_t H, int64_t T,
                                          int32_t k, int32_t E, const int32_t* idx, const int32_t* slot,
                                          const int32_t* offsets, const float* gate, void* dy, float* dgate,
                                          moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS_H */
