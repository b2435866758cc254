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
 *   moe_quantize_fp4 / moe_dequantize_fp4
 *                                   4-bit values with one scale for a block of 32
 *   moe_expert_matmul_fp4           the experts' matrix products on such values
 *   moe_expert_glu / _bwd           the gated activation between the two products,
 *                                   also quantised as it leaves, and its gradient
 *   moe_layer_small                 all that follows the routing, for the few tokens of
 *                                   a decode step, in three kernels
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

/* Reads and clears the error bits that moe_expert_matmul, moe_expert_wgrad and
 * moe_expert_matmul_fp4 calls have left on the current device (synchronises `stream`, on
 * which they were queued).  *flags = 0 when every wait completed; otherwise returns
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

/* ------------------------------------------------------------------------ */
/* 4-bit values with one scale for a block of 32                            */
/* ------------------------------------------------------------------------ */

/* Values that share a scale, along the contraction. */
#define MOE_FP4_BLOCK 32

/* A code has a sign (bit 3) and one of the sizes 0, 1/2, 1, 3/2, 2, 3, 4, 6; two
 * codes lie in a byte, the even column's in the low four bits.  A block's scale is
 * the power of two s with 3 < max|x| / s <= 6 (at least 2^-126; 1 for a block of
 * zeros), held as a byte n that stands for 2^(n - 127); its codes are x / s rounded
 * to nearest, ties to even.  A block with an infinity or a NaN gets n = 255, a NaN
 * (its codes are unspecified), so that every product with it is NaN.
 * x is fp32 or bf16 [rows,K].  q [M,K/2]: row r holds row perm[r] / k of x, or row r
 * when perm is NULL (then M == rows); a perm entry outside [0, rows*k) gives a row of
 * zeros.  scale [ceil(K/128), M, 4]: the bytes of the four blocks of 128 columns
 * together, and the rows of one such column next to one another; bytes behind
 * column K are 127.  Weights [E,N,K] are E*N rows.
 * K is a multiple of 32 up to MOE_MAX_WIDTH; x and q are 16-byte aligned, scale is
 * 4-byte aligned. */
MOE_API moe_status moe_quantize_fp4(const void* x, moe_dtype dt, int64_t rows, int64_t M, int32_t K,
                                    const int32_t* perm, int32_t k, void* q, void* scale, moe_stream_t stream);

/* y[r,c] = code * 2^(n - 127), NaN where n = 255: exact in fp32 and bf16, but for sizes
 * above their largest number, which give an infinity.  q [M,K/2] and scale as above, y [M,K]
 * fp32 or bf16 (dt), 16-byte aligned as q is. */
MOE_API moe_status moe_dequantize_fp4(const void* q, const void* scale, int64_t M, int32_t K, moe_dtype dt, void* y,
                                      moe_stream_t stream);

/* The product of moe_expert_matmul (rows, offsets, kept and out as there) on 4-bit
 * operands:
 *   q [M,K/2], scale [ceil(K/128), M, 4]: as moe_quantize_fp4 of the rows
 *   wq [E,N,K/2], wscale [ceil(K/128), E, N, 4]: as moe_quantize_fp4 of E*N rows
 * The tensor core multiplies a block's products by its two scales and adds them, over
 * the whole contraction, in fp32 (where products below about 2^-25 of the largest that
 * are added with them may be lost); the one rounding to bf16 is at the end.  A row's
 * result does not depend on the other rows, and a row or column with a NaN scale is NaN.
 * K is a multiple of 32, N of 16, both up to MOE_MAX_WIDTH; E * N < 2^31, M >= 1,
 * M < 2^31; q, wq, wscale and out are 16-byte aligned, scale 4-byte aligned.  Needs no
 * workspace.  A device wait that runs out is reported by moe_expert_device_status, and
 * until that is read later products on the device write nothing. */
MOE_API moe_status moe_expert_matmul_fp4(const void* q, const void* scale, int64_t M, int32_t K,
                                         const void* wq, const void* wscale, int32_t E, int32_t N,
                                         const int32_t* offsets, const int32_t* kept, moe_dtype out_dt, void* out,
                                         moe_stream_t stream);

/* ------------------------------------------------------------------------ */
/* The gated activation between the experts' products                       */
/* ------------------------------------------------------------------------ */

typedef enum { MOE_GLU_PLAIN = 0, MOE_GLU_E4M3 = 1, MOE_GLU_FP4 = 2 } moe_glu_form;

/* y[r,i] = g * sigmoid(g) * u with g = h[r,i], u = h[r,I+i], of h [M,2I] (fp32 or bf16),
 * in fp32.  It leaves as
 *   MOE_GLU_PLAIN: out [M,I] in h's type (scale is NULL)
 *   MOE_GLU_E4M3:  out [M,I] and scale [ceil(I/128), M] fp32, as moe_quantize_rows has them
 *   MOE_GLU_FP4:   out [M,I/2] and scale [ceil(I/128), M, 4], as moe_quantize_fp4 has them
 * (the blocks' scales are those of the fp32 values).  g = -infinity gives a NaN.  A sigmoid below
 * 2^-126 has fewer digits than others, and one below 2^-149 is 0.
 * I is a multiple of 16 (MOE_GLU_FP4: of 32) up to MOE_MAX_WIDTH; h and out are 16-byte
 * aligned, scale is 4-byte aligned.  All M rows are read and written, those of dropped assignments too. */
MOE_API moe_status moe_expert_glu(const void* h, moe_dtype dt, int64_t M, int32_t I, moe_glu_form form, void* out,
                                  void* scale, moe_stream_t stream);

/* Its gradient, with s = sigmoid(g): dh[r,i] = dy u s (1 + g (1 - s)), dh[r,I+i] = dy g s.
 * A result that fp32 holds is finite, though dy u may not be; an infinite g gives a NaN.
 * dy [M,I] and dh [M,2I] have h's type and are 16-byte aligned. */
MOE_API moe_status moe_expert_glu_bwd(const void* h, const void* dy, moe_dtype dt, int64_t M, int32_t I, void* dh,
                                      moe_stream_t stream);

/* ------------------------------------------------------------------------ */
/* The experts of a layer for few tokens                                    */
/* ------------------------------------------------------------------------ */

#define MOE_SMALL_TOKENS 64
#define MOE_SMALL_WIDTH 16384
typedef enum { MOE_WEIGHTS_E4M3 = 0, MOE_WEIGHTS_FP4 = 1 } moe_weight_kind;

/* out[t,:] = sum_j gate[t,j] * W2_e glu(W1_e x[t,:]) with e = idx[t,j] and glu as in
 * moe_expert_glu: what dispatch, the two products, the activation between them and the
 * combine compute, without a capacity, for T <= MOE_SMALL_TOKENS tokens.  The weights are
 * quantised, the tokens' values are not.
 *   x [T,H], out [T,H] bf16; idx, gate [T,k] as moe_route_fwd gives them: an idx outside
 *   [0,E) adds nothing, a token without any other gets zeros, an expert picked twice counts twice
 *   w1 [E,2I,H]: the gates' I rows, then the other I; w2 [E,H,I]; each either
 *     MOE_WEIGHTS_E4M3: q and scale as moe_quantize_weights gives them, or
 *     MOE_WEIGHTS_FP4:  q and scale as moe_quantize_fp4 gives them
 * Sums are fp32, and are finite wherever fp32 holds them and their terms, however large or small
 * the values and the scales are.  Of each 128 values of x, those below 2^-28 of the largest lose digits;
 * the activations are rounded to 11 bits, relative to the larger of themselves and 2^-28 of
 * the largest of their 128, three more than a result has.  Repeated calls give the same bits.  With e4m3 weights a token's
 * result does not depend on the others; with 4-bit ones its last bits may, on how many
 * tokens have its expert and on its place among them (up to 4 are computed in one way, more in
 * another, and of many the last few by themselves; beside one with a block of 128 values that are
 * all below 2^-78, or reach 2^111, more are computed as up to 4 are).
 * H and I are multiples of 16 (of 32 where a matrix of 4 bits has them as its row length)
 * up to MOE_SMALL_WIDTH; x, out and the codes are 16-byte aligned, the scales, idx and
 * gate 4-byte aligned.  work: moe_layer_small_work_size bytes, 16-byte aligned, of any
 * content; calls that may run at the same time each take their own.
 * With 4-bit weights and from some 16 tokens on the chain of moe_quantize_fp4, moe_expert_matmul_fp4 and
 * moe_expert_glu takes less time, on tokens and activations that are rounded to 4 bits. */
MOE_API size_t moe_layer_small_work_size(int64_t T, int32_t H, int32_t I, int32_t k);
MOE_API moe_status moe_layer_small(const void* x, int64_t T, int32_t H, int32_t I, int32_t E, int32_t k,
                                   const int32_t* idx, const float* gate,
                                   moe_weight_kind kind1, const void* w1q, const void* w1scale,
                                   moe_weight_kind kind2, const void* w2q, const void* w2scale,
                                   void* out, void* work, size_t work_bytes, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS_H */
