/*
 * ppstage.h -- C ABI of the operators of one pipeline stage in libppsched: the
 * work whose time and held bytes the schedule evaluator (ppsched.h) takes as
 * costs.  A stage's op is F (forward), B (input gradient) or W (weight
 * gradient; split from B by the Zero Bubble schedules).
 *
 *   head   the last stage's loss: softmax cross entropy over a large
 *          vocabulary, taken in pieces of the vocabulary so that the logits
 *          are never kept, with the gradients of the activations (B) and of
 *          the output matrix (W).
 *   kept   activation checkpoints in 8 bits: what a microbatch holds between
 *          its F and its W, and the weight gradient taken from them.
 *   join   the end of one block and the start of the next: the norm after the
 *          block, its gate, the residual scale and sum, the norm before the
 *          next block; forward and backward.
 *
 * Conventions for every entry point (as in ppsched.h):
 *   - Arrays are caller-owned DEVICE memory; matrices are row-major with
 *     contiguous rows and an element stride between rows (>= the row's length).
 *     bf16 matrices are passed as uint16_t.
 *   - Calls are asynchronous on `stream`, allocate nothing and never
 *     synchronize.  Scratch memory is the caller's: each *_workspace function
 *     gives the bytes that the call with the same arguments needs (256-byte
 *     aligned).  A workspace may be used again by later calls on the same
 *     stream.
 *   - Inputs are only read; outputs must not overlap inputs or one another,
 *     except where an entry point says so.
 *   - Any row stride and any element-aligned base is accepted.  Rows whose base
 *     or stride is not a multiple of 16 bytes cost an aligned copy (head,
 *     weight gradient) or narrower accesses (kept, join).
 *   - Return value: PP_OK or a PP_ERR_* code of ppsched.h; arguments are checked
 *     on the host before anything is launched.
 *   - Sums, softmax statistics and norms are held in 32 bits.  Every result is
 *     the same on every call with the same inputs: nothing depends on the order
 *     in which blocks run.
 */
#ifndef PPSTAGE_H
#define PPSTAGE_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Limits (PP_ERR_SIZE beyond them, and where a product would have more than
 * 2^31 tiles). */
#define PP_STAGE_MAX_ROWS (1 << 24)   /* T: tokens of one call */
#define PP_STAGE_MAX_VOCAB (1 << 24)  /* V, and N of the weight gradient */
#define PP_STAGE_MAX_WIDTH (1 << 16)  /* H of head and kept */
#define PP_STAGE_MAX_JOIN_WIDTH 16384 /* H of the join */

/* Columns of a checkpoint that share one exponent. */
#define PP_STAGE_BLOCK 64
/* Exponent of a block that holds an infinity or a NaN: it stands for NaN. */
#define PP_STAGE_NONFINITE (-128)

/* ---- head ---------------------------------------------------------------
 * logits l = x w^T (never stored), x [T][H] bf16, w [V][H] bf16.
 *   lse[t]  = log sum_v exp l[t][v]
 *   loss[t] = lse[t] - l[t][target[t]], and 0 for a token that is left out: one
 *             whose target is outside 0..V-1 (any negative number, for example)
 * loss or lse may be NULL, not both. */
size_t pp_stage_head_forward_workspace(const uint16_t *x, int64_t stride_x, const uint16_t *w, int64_t stride_w,
                                       int64_t T, int64_t V, int64_t H);
int pp_stage_head_forward(const uint16_t *x, int64_t stride_x, const uint16_t *w, int64_t stride_w,
                          const int64_t *target, int64_t T, int64_t V, int64_t H, float *loss, float *lse,
                          void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* Gradients of sum_t scale * weight[t] * loss[t] (weight NULL: 1), from lse as
 * pp_stage_head_forward returned it:
 *   d[t][v] = weight[t] (exp(l[t][v] - lse[t]) - [v == target[t]]), 0 where left out
 *   dx [T][H] = scale * d w           bf16
 *   dw [V][H] = scale * d^T x         bf16, or float (dw_float = 1); with
 *               dw_add = 1 (float only) it is added to what dw holds
 * dx or dw may be NULL, not both (B and W as two calls).  d is taken piece by
 * piece of the vocabulary, rounded to bf16 before `scale` is applied; what the
 * rounding leaves over at a token's target is added to dx, and to dw where up to
 * eight tokens share the target, in 32 bits.  A row of x that is left out is not
 * read into dw, whatever it holds. */
size_t pp_stage_head_backward_workspace(const uint16_t *x, int64_t stride_x, const uint16_t *w, int64_t stride_w,
                                        int64_t T, int64_t V, int64_t H);
int pp_stage_head_backward(const uint16_t *x, int64_t stride_x, const uint16_t *w, int64_t stride_w,
                           const int64_t *target, const float *lse, const float *weight, float scale,
                           int64_t T, int64_t V, int64_t H, uint16_t *dx, int64_t stride_dx,
                           void *dw, int64_t stride_dw, int dw_float, int dw_add,
                           void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* ---- kept ---------------------------------------------------------------
 * The checkpoint of x [T][H] bf16: q [T][H] int8 and e [T][ceil(H/64)] int8.
 * Per row and block of 64 columns, with a = max |x|:
 *   e = max(floor(log2 a) - 6, -126), q = rint(x / 2^e) (ties to even) within
 *   +-127; a = 0: e = -126, q = 0; a not finite: e = PP_STAGE_NONFINITE, q = 0
 * and q 2^e is what an element stands for.  The step is a power of two so that
 * every value is a bf16 number: what reads a checkpoint adds no rounding. */
int pp_stage_pack(const uint16_t *x, int64_t stride_x, int64_t T, int64_t H, int8_t *q, int64_t stride_q,
                  int8_t *e, int64_t stride_e, cudaStream_t stream);
int pp_stage_unpack(const int8_t *q, int64_t stride_q, const int8_t *e, int64_t stride_e, int64_t T, int64_t H,
                    uint16_t *x, int64_t stride_x, cudaStream_t stream);

/* W of a linear layer whose input was kept: dw [N][H] = add + dy^T v, with
 * dy [T][N] bf16, v what (q, e) stands for, add [N][H] float (NULL: 0; it may be
 * dw itself, the running sum of the microbatches).  T = 0 gives add. */
size_t pp_stage_weight_grad_workspace(const uint16_t *dy, int64_t stride_dy, int64_t T, int64_t N, int64_t H);
int pp_stage_weight_grad(const uint16_t *dy, int64_t stride_dy, const int8_t *q, int64_t stride_q,
                         const int8_t *e, int64_t stride_e, int64_t T, int64_t N, int64_t H,
                         const float *add, int64_t stride_add, float *dw, int64_t stride_dw,
                         void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* ---- join ---------------------------------------------------------------
 * A block's output f joins the residual stream x; all [T][H] bf16:
 *   rstd_post[t] = 1 / sqrt(mean_h f^2 + eps)
 *   y = alpha * x + gate[g] * w_post * f * rstd_post
 *   rstd_pre[t]  = 1 / sqrt(mean_h y^2 + eps)      (y before it is rounded)
 *   h = y * rstd_pre * w_pre
 * w_post, w_pre [H] bf16; gate [G][H] bf16, row t uses gate[t / rows_per_gate]
 * (rows_per_gate <= 0: one gate for all rows; gate NULL: 1).  y, h bf16; rstd_*
 * float [T].  With the four kept pointers given (or all NULL), y as rounded and
 * f are also packed as by pp_stage_pack: what pp_stage_join_backward reads. */
int pp_stage_join_forward(const uint16_t *x, int64_t stride_x, const uint16_t *f, int64_t stride_f,
                          const uint16_t *w_post, const uint16_t *w_pre, const uint16_t *gate, int64_t stride_gate,
                          int64_t rows_per_gate, float alpha, float eps, int64_t T, int64_t H,
                          uint16_t *y, int64_t stride_y, uint16_t *h, int64_t stride_h,
                          float *rstd_post, float *rstd_pre,
                          int8_t *y_q, int64_t stride_yq, int8_t *y_e, int64_t stride_ye,
                          int8_t *f_q, int64_t stride_fq, int8_t *f_e, int64_t stride_fe, cudaStream_t stream);

/* Gradients of the join, given dh (of h) and dy (what reaches y by other paths;
 * NULL: 0), with n1 = f rstd_post, n2 = y rstd_pre, c = dh w_pre:
 *   d  = dy + rstd_pre (c - n2 mean_h(c n2))       dx = alpha d           bf16
 *   s  = d gate w_post                             df = rstd_post (s - n1 mean_h(s n1))   bf16
 *   dw_pre = sum_t dh n2     dw_post = sum_t d gate n1     dgate[g] = sum_{t of g} d n1 w_post   float
 * y and f come as bf16 (y, f given) or as checkpoints (y_q, y_e, f_q, f_e given):
 * one form for both.  dgate is NULL exactly where gate is; of it only the rows
 * of gates that some token uses are written. */
size_t pp_stage_join_backward_workspace(int64_t T, int64_t H, int64_t rows_per_gate);
int pp_stage_join_backward(const uint16_t *dh, int64_t stride_dh, const uint16_t *dy, int64_t stride_dy,
                           const uint16_t *y, int64_t stride_y, const uint16_t *f, int64_t stride_f,
                           const int8_t *y_q, int64_t stride_yq, const int8_t *y_e, int64_t stride_ye,
                           const int8_t *f_q, int64_t stride_fq, const int8_t *f_e, int64_t stride_fe,
                           const float *rstd_post, const float *rstd_pre,
                           const uint16_t *w_post, const uint16_t *w_pre, const uint16_t *gate, int64_t stride_gate,
                           int64_t rows_per_gate, float alpha, int64_t T, int64_t H,
                           uint16_t *dx, int64_t stride_dx, uint16_t *df, int64_t stride_df,
                           float *dw_post, float *dw_pre, float *dgate, int64_t stride_dgate,
                           void *workspace, size_t workspace_bytes, cudaStream_t stream);

/* ---- waits --------------------------------------------------------------
 * The blocks of the products and of the join's rings wait for their own copies
 * and matrix instructions with a limit of two seconds.  A wait that runs out is
 * recorded, its block gives up (the call's outputs are then wrong), lets what it
 * has in flight land, with a limit again, and the kernel ends.  Calls are
 * asynchronous and return PP_OK all the same: a program asks here once its work
 * has run, before it relies on the results.  *first_failure (HOST) receives a
 * record of the current device made since the previous call, 0 if there is none,
 * and the records are cleared: bit 63 set, the waiting role in bits 32..39 (of a
 * product: 1 loads, 2 and 3 matrix instructions, 4 results; of a ring: 5 forward,
 * 6 backward), the block below.  Synchronizes the device.  Errors: PP_ERR_ARG;
 * PP_ERR_CUDA, also where a record could not be read. */
int pp_stage_wait_failure(uint64_t *first_failure);

#ifdef __cplusplus
}
#endif

#endif /* PPSTAGE_H */
