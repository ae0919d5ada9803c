/*
 * muon_stack.h -- C ABI of the Muon step (muon.h) on stacks of matrices with a
 * short side: the heads of attention projections, low-rank adapters, any
 * batch of matrices of which one side is at most MUON_STACK_MAX_SHORT.
 *
 * Every matrix of a stack gets the update of muon.h by itself (its own norm,
 * its own iteration):
 *
 *   buf' = mu * buf + G           (stored back at the set's dtype, RNE)
 *   u    = G + mu * buf'  (Nesterov)   or   u = buf'
 *   X    = u / (||u||_F + eps)    (transposed if rows > cols)
 *   k times:  A = X X^T;  B = b A + c A A;  X = a X + B X
 *   out  = X (transposed back), or  W <- W (1 - lr' wd') - lr' X
 *
 * (blog.hotdry.top, "How to train a GPT model in 3 minutes", section 2,
 * customised Muon optimizer; the weight application as in muon.h.) A stack is
 * a 3-D view: element (t, i, j) at base + t * stride + i * ld + j, so the
 * heads of a fused projection are row blocks (stride = rows * ld) or column
 * blocks (stride = cols) of one matrix, without a copy.
 *
 * muon_plan_create takes the same matrices one by one, each padded to 256 x
 * 256 tiles of its products. Here the iteration runs on the short side's
 * Gram matrix: with m <= 128 the powers of A fit one workgroup, and s steps
 * become X <- (Q_s .. Q_1) X, Q_i = a I + b A_i + c A_i^2, A_{i+1} = Q_i A_i Q_i,
 * so that X is read and written once per s steps instead of once per product.
 * After s steps A is formed anew from X: s is chosen from the polynomial so
 * that rounding errors of A grow by less than 2^15 (bf16 sets) or 2^3 (fp32
 * sets) within a run of s (five and one steps for the usual quintic, thirteen
 * and three for the cubic). What that leaves of X stands below.
 *
 * Arithmetic: buf' is the exact mu * buf + G rounded once to the set's dtype,
 * as in muon.h; everything else is fp32. The products run on the matrix
 * cores with fp32 accumulation; every operand x is taken as two fp16 numbers,
 * x 2^e = hi + lo with |x 2^e - hi - lo| <= 2^-22 |x 2^e| (2^-24 for the
 * smallest, entries being scaled to at most 2^15), and a product as hi hi +
 * hi lo + lo hi, for both dtypes. Sums of squares are kept relative to a power
 * of two, so no finite u overflows them.
 *
 * Accuracy of X before its rounding, relative to its norm, five quintic steps,
 * measured on shapes from 2 x 50 to 128 x 2048. fp32 sets: 4e-6 on random
 * gradients, 7e-5 on gradients of rank one. bf16 sets, whose five steps come
 * from one A: 5e-6 on random gradients (4e-5 on square ones), up to 6e-4 where
 * singular values span two decades, a median of up to 1e-3 where they span
 * three to five, and of 1.8e-3 on gradients of rank one, whose other singular
 * values are the rounding of their entries; the worst of thousands of
 * matrices 6.3e-3, with a short side of four (2.4e-3 with one of 64). The
 * rounding of a bf16 output is 1.7e-3, and muon_plan_step on the same gradients
 * is off by a median of 1.0e-3 to 3.1e-3 and by 5.8e-3 at worst before it.
 *
 * Conventions are those of muon.h: pointers are device memory owned by the
 * caller, arguments are validated before any work is enqueued (nothing is
 * launched or written on an error), work is asynchronous on `stream`, results
 * are deterministic, NaN and infinities propagate (within their matrix), a
 * step allocates nothing and can be captured into a graph.
 */
#ifndef MUON_STACK_H
#define MUON_STACK_H

#include <stddef.h>
#include <stdint.h>

#include "muon.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Limits (MUON_E_SHAPE beyond them): the shorter side of a matrix, its longer
 * side, and the matrices of all stacks of a plan. */
#define MUON_STACK_MAX_SHORT 128
#define MUON_STACK_MAX_LONG MUON_MAX_DIM
#define MUON_STACK_MAX_MATRICES MUON_MAX_MATRICES

/* count matrices of rows x cols; grad, momentum and out share ld and stride
 * (elements). A stack with count, rows or cols 0 is skipped. `grad` is read;
 * `momentum` is read and overwritten with buf' (NULL iff the config's momentum
 * is 0, and must then not be used); `out` is written. `out` may equal `grad`.
 * The matrices of a stack must be apart: blocks one behind another (stride >=
 * a matrix's span, (rows - 1) * ld + cols) or side by side in the columns of
 * one matrix (stride >= cols, (count - 1) * stride + cols <= ld).
 * Otherwise nothing written may overlap anything else of the plan
 * (MUON_E_INVALID). Stacks may lie in one buffer in turn, matrix by matrix, and
 * column slices at one row stride are told apart by their columns; matrices
 * of different row strides whose rows lie between each other's count as
 * overlapping. */
typedef struct {
  int64_t count;
  int64_t rows;
  int64_t cols;
  int64_t ld;
  int64_t stride;
  const void* grad;
  void* momentum;
  void* out;
} muon_stack;

/* The weights of a stack: same count, rows, cols and dtype, its own ld and
 * stride (the same rule). lr_mul, wd_mul: multipliers of the whole stack. */
typedef struct {
  void* weight;
  int64_t ld;
  int64_t stride;
  float lr_mul;
  float wd_mul;
} muon_stack_weight;

typedef struct muon_stack_plan_s muon_stack_plan;

/* Bytes of device workspace a step on these stacks needs, whatever its
 * configuration (host only, no device calls; 0 when all are empty). Most of it
 * is room for every X in float32, which a configuration whose steps are one run
 * does not touch. */
muon_status muon_stack_workspace_bytes(const muon_stack* stacks, int32_t n, muon_dtype dtype,
                                       size_t* bytes);

/* Validates the stacks and uploads their tables to the current device (a few
 * KB to MB owned by the plan; *plan receives NULL on error). No state is kept
 * between steps. */
muon_status muon_stack_plan_create(const muon_stack* stacks, int32_t n, muon_dtype dtype,
                                   muon_stack_plan** plan);

/* One Muon update of every matrix: `out` and the momentum are written. cfg as
 * in muon.h; the range check of its coefficients holds for both dtypes here
 * (the fp16 operands need it). `workspace` must hold at least
 * muon_stack_workspace_bytes bytes, 256-byte aligned, overlap nothing of the
 * plan and be used by nothing else until the work ends; its contents need not
 * be initialised. A matrix of zeros gives zeros. */
muon_status muon_stack_plan_step(muon_stack_plan* plan, const muon_config* cfg, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* Attaches weights, one record per stack (records of empty stacks are
 * ignored). Waits for the device, then updates the plan's table; a captured
 * graph follows. On error the plan keeps its previous weights. */
muon_status muon_stack_plan_set_weights(muon_stack_plan* plan, const muon_stack_weight* w,
                                        int32_t n);

/* muon_stack_plan_step, except that the weights receive W <- W (1 - lr' wd') -
 * lr' X (fp32, one rounding) and `out` is left untouched. MUON_E_INVALID if
 * the plan has no weights. */
muon_status muon_stack_plan_step_apply(muon_stack_plan* plan, const muon_config* cfg,
                                       const muon_apply* ap, void* workspace,
                                       size_t workspace_bytes, void* stream);

/* Attaches a gradient factor in device memory (NULL detaches it): G * *scale
 * in place of G, as muon_plan_set_grad_scale does. */
muon_status muon_stack_plan_set_grad_scale(muon_stack_plan* plan, const float* scale);

/* Frees a plan after waiting for the device (NULL is a no-op). A captured
 * graph reads the plan's tables: it must not be replayed afterwards. */
void muon_stack_plan_destroy(muon_stack_plan* plan);

#ifdef __cplusplus
}
#endif

#endif /* MUON_STACK_H */
