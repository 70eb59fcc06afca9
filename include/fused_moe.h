/*
 * fused_moe.h -- C ABI of the routed-experts operators (gfx950)
 *
 * What a layer of E experts needs around and inside its fused linear layers:
 * a router that picks k experts for each of T tokens, a plan that sorts the
 * T*k (token, choice) slots by expert, the movement of token rows into that
 * order and back, and the fused linear layer act(A @ B[e] + bias[e]) over
 * every expert's run of rows, with its backward pass.
 *
 * Conventions are those of fused_linear.h (row-major contiguous operands,
 * caller-owned device pointers, work enqueued on `stream`, no
 * synchronisation, no allocation, arguments validated before any HIP call),
 * with these additions:
 *   Slots      slot t*k + j is choice j of token t; S = T*k of them.
 *   Rows       row r of a sorted (S, ...) operand belongs to expert e where
 *              offsets[e] <= r < offsets[e+1].  Rows at or past offsets[E]
 *              belong to nobody: they are not read, and outputs leave them as
 *              they are unless an entry point says otherwise.
 *   Device     offsets, index, experts and row_of_slot are device arrays whose
 *   integers   values the host never sees.  Kernels limit them to the stated
 *              ranges before they address memory with them: offsets to
 *              [0, S], an index outside [0, rows of its operand) reads a row
 *              of zeros, an expert outside [0, E) is no expert.
 *   Errors     fl_status as in fused_linear.h; the message of the last failed
 *              call of this header is read with fl_moe_last_error().
 *   Order      every result is the same to the bit from run to run: no
 *              floating-point atomics anywhere.
 */
#ifndef FUSED_MOE_H
#define FUSED_MOE_H

#include "fused_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    FL_SCORE_SOFTMAX = 0, /* s = softmax of the token's E logits   */
    FL_SCORE_SIGMOID = 1  /* s = 1 / (1 + exp(-logit)), each alone */
} fl_score;

/* How experts are chosen and weighted.  Zero-initialise and set what you
 * need; zero means the default given here. */
typedef struct {
    int32_t score;      /* fl_score */
    int32_t groups;     /* 0 or 1 = none; else the experts form this many runs
                           of E/groups neighbours (groups <= 64 divides E) and
                           only the best top_groups runs may be chosen from */
    int32_t top_groups; /* 0 = 1; at most groups */
    int32_t group_top;  /* 0 or 1: a run scores its largest key; 2: the sum of
                           its two largest (of the one, where one is left) */
    int32_t raw;        /* 0: a token's weights are divided by their sum; 1: not */
    float scale;        /* factor on the weights, finite; 0 stands for 1 */
} fl_route_options;

/*
 * Chooses k experts for every token and weights them.
 *   logits   (T,E) in dtype.  -inf masks an expert for a token; NaN counts as
 *            -inf; a +inf logit takes the whole softmax (several share it).
 *   bias     (E,) fp32 or NULL: added to the score for the choice only (a
 *            balance term); it does not enter the weights.
 *   experts  (T,k) int32: the k largest keys in falling order, ties to the
 *            lower expert.  The key is the logit where bias is NULL (the
 *            scores have its order), else score + bias.  Slots for which no
 *            unmasked expert (in a kept run) is left hold -1.
 *   weights  (T,k) fp32: scale * s of the chosen, divided by their sum unless
 *            opt->raw; 0 where the expert is -1.
 * Choices are those of keys computed in 64 bits; the weights are fp32.
 * 1 <= k <= 64, k <= E <= 1024.  opt may be NULL (defaults).
 */
fl_status fl_moe_route(const void *logits, const float *bias, int32_t *experts, float *weights, int64_t T, int64_t E,
                       int64_t k, fl_dtype dtype, const fl_route_options *opt, void *stream);

/*
 * The gradient of the logits: dlogits[t,:] = sum_j dweights[t,j] *
 * d weights[t,j] / d logits[t,:] for the chosen experts (the choice itself
 * has no gradient, nor has the bias).  experts as fl_moe_route gave them;
 * slots with -1 count for nothing; masked logits get 0.  dlogits (T,E) in
 * dtype, overwritten; it may equal logits.  Only score, raw and scale of opt
 * are used.
 */
fl_status fl_moe_route_bwd(const void *logits, const int32_t *experts, const float *dweights, void *dlogits, int64_t T,
                           int64_t E, int64_t k, fl_dtype dtype, const fl_route_options *opt, void *stream);

/*
 * The plan of a choice: a stable sort of the slots by expert.
 *   experts       (T,k) int32; values outside [0,E) are slots without an expert.
 *   offsets       (E+1,) int32: first row of every expert; offsets[E] rows in all.
 *   token_of_row  (T*k,) int32: the token of every row, -1 at and past offsets[E].
 *   row_of_slot   (T,k) int32: the row of every slot, -1 without an expert.
 *   workspace     fl_moe_plan_workspace_bytes(T, k, E) bytes, 4-byte aligned
 *                 (may be NULL when that is 0); written and read by this
 *                 call's launches only.
 * E <= 1024, T*k <= 2^31-1.  T == 0 or k == 0 gives offsets of zeros.
 */
fl_status fl_moe_plan(const int32_t *experts, int32_t *offsets, int32_t *token_of_row, int32_t *row_of_slot, int64_t T,
                      int64_t k, int64_t E, void *workspace, size_t workspace_bytes, void *stream);
fl_status fl_moe_plan_workspace_bytes(int64_t T, int64_t k, int64_t E, size_t *bytes);

/* rows[r,:] = X[index[r],:] for the S rows (index: token_of_row), zeros where
 * index[r] is outside [0,T).  X (T,H), rows (S,H), no overlap. */
fl_status fl_moe_gather(const void *X, const int32_t *index, void *rows, int64_t T, int64_t S, int64_t H,
                        fl_dtype dtype, void *stream);

/* out[t,:] = R[t,:] + sum_j weights[t,j] * rows[row_of_slot[t,j],:], summed in
 * fp32 in the order of j, R last, one rounding.  A slot whose row is outside
 * [0,S) adds nothing (its weight is not used).  weights NULL: all 1 (the
 * gradient of fl_moe_gather).  R (T,H) or NULL; out may equal R. */
fl_status fl_moe_combine(const void *rows, const int32_t *row_of_slot, const float *weights, const void *R, void *out,
                         int64_t T, int64_t k, int64_t S, int64_t H, fl_dtype dtype, void *stream);

/* Gradients of fl_moe_combine: drows[row_of_slot[t,j],:] = weights[t,j] *
 * dout[t,:] (each rounded once; rows no slot points at are left alone) and
 * dweights[t,j] = sum_h dout[t,h] * rows[row_of_slot[t,j],h] in fp32 (0 for a
 * slot without a row).  Every row may belong to one slot at most.  drows or
 * dweights may be NULL (not both, unless T*k, S or H is 0); rows is only read
 * for dweights; weights NULL: all 1.  drows may equal rows. */
fl_status fl_moe_combine_bwd(const void *dout, const void *rows, const int32_t *row_of_slot, const float *weights,
                             void *drows, float *dweights, int64_t T, int64_t k, int64_t S, int64_t H, fl_dtype dtype,
                             void *stream);

/*
 * out[r,:] = act(A[index[r],:] @ B[e] + bias[e]) for every row r of every
 * expert e: the fused linear layer of fused_linear.h over the experts' runs
 * of rows in one launch, products summed in fp32, the epilogue in fp32, one
 * rounding.
 *   A        (A_rows, K); row r of the product is A[r] (then A_rows >= S) or,
 *            with index (S,) int32, A[index[r]].
 *   offsets  (E+1,) int32, as fl_moe_plan gives them.
 *   B        (E,K,N).  bias (E,N) or NULL.
 *   Y        (S,N), for FL_ACT_GLU only.
 *   out      (S,N); may equal Y.
 *   pre      (S,N) or NULL: also receives X = A @ B[e] + bias[e], rounded once
 *            (what the backward pass needs).
 * Every dtype.  K == 0 gives act(bias).  Each B[e], 256 rows of any operand
 * and, with index, the whole of A must span less than 2 GiB.
 *   workspace  fl_grouped_workspace_bytes(S, N, K, E, dtype) bytes, 16-byte
 *            aligned (may be NULL when that is 0): few rows of a long K are
 *            summed in parts, which meet there in a fixed order.
 */
fl_status fl_grouped_linear(const void *A, const int32_t *index, const int32_t *offsets, const void *B,
                            const void *bias, const void *Y, void *out, void *pre, int64_t A_rows, int64_t S,
                            int64_t N, int64_t K, int64_t E, fl_act act, fl_dtype dtype, void *workspace,
                            size_t workspace_bytes, void *stream);
fl_status fl_grouped_workspace_bytes(int64_t S, int64_t N, int64_t K, int64_t E, fl_dtype dtype, size_t *bytes);

/*
 * The backward epilogue over the experts' rows (fl_fused_linear_bwd's, per
 * expert): D = G @ W[e]^T, dX = D * act'(X), the gate's dY = D * X.
 *   G (S,K); W (E,N,K), the weight whose product takes this layer's output;
 *   X (S,N) the saved pre-activation (NULL only with FL_ACT_NONE, where it is
 *   not read); Y (S,N) and dY (S,N) for the gate only.  dX may equal X, dY may
 *   equal Y.  Every dtype; limits as fl_grouped_linear's.
 */
fl_status fl_grouped_linear_bwd(const void *G, const int32_t *offsets, const void *W, const void *X, const void *Y,
                                void *dX, void *dY, int64_t S, int64_t N, int64_t K, int64_t E, fl_act act,
                                fl_dtype dtype, void *stream);

/*
 * The weight gradients: dW[e] = sum over expert e's rows of A[r,:]^T G[r,:]
 * and dbias[e] = the sum of its rows of G, both summed in fp32.
 *   A (S,K), G (S,N) in dtype; dW (E,K,N) in dw_dtype, which is dtype or
 *   FL_F32; dbias (E,N) fp32 or NULL.  An expert without rows gets zeros.
 * Every row of A spans less than 2 GiB / 256, as every row of G.
 */
fl_status fl_grouped_weight_grad(const void *A, const void *G, const int32_t *offsets, void *dW, float *dbias,
                                 int64_t S, int64_t N, int64_t K, int64_t E, fl_dtype dtype, fl_dtype dw_dtype,
                                 void *stream);
/* The same with a workspace of fl_grouped_grad_workspace_bytes(S, N, K, E,
 * dtype) bytes, 16-byte aligned: long runs of a small dW are summed in parts
 * that meet there in a fixed order (the rounding of fp32 sums may then differ
 * from the call without).  NULL: no parts. */
fl_status fl_grouped_weight_grad_ws(const void *A, const void *G, const int32_t *offsets, void *dW, float *dbias,
                                    int64_t S, int64_t N, int64_t K, int64_t E, fl_dtype dtype, fl_dtype dw_dtype,
                                    void *workspace, size_t workspace_bytes, void *stream);
fl_status fl_grouped_grad_workspace_bytes(int64_t S, int64_t N, int64_t K, int64_t E, fl_dtype dtype, size_t *bytes);

const char *fl_moe_last_error(void); /* thread-local; "" when none */

#ifdef __cplusplus
}
#endif

#endif /* FUSED_MOE_H */
