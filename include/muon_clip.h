/*
 * muon_clip.h -- C ABI of the global gradient norm over a whole list of
 * gradient tensors and of clipping by it, the step that stands between the
 * backward pass and the optimizer step (muon.h, muon_adam.h).
 *
 * For gradients g_0 .. g_{n-1} (any mix of the two element types), a limit
 * max_norm, eps and a multiplier c (grad_mul: 1, or the reciprocal of a loss
 * scale or of a number of accumulated micro-batches):
 *
 *   N_i    = c * sqrt(sum of the squares of tensor i)
 *   N      = c * sqrt(sum of the squares of all tensors)
 *   factor = c                        if N + eps <= max_norm
 *            c * max_norm / (N + eps) otherwise
 *   out_i  = g_i * factor             (muon_clip_plan_step)
 *
 * The factor is left in device memory. Instead of writing clipped gradients,
 * the optimizer steps can read it and multiply each gradient as they load it:
 * muon_plan_set_grad_scale (muon.h) and muon_adam_plan_set_grad_scale
 * (muon_adam.h). One or the other: muon_clip_plan_step leaves the same factor
 * as muon_clip_plan_norm, and a step that still reads it would multiply
 * gradients clipped in place a second time. A call writes the factor when it
 * runs, so the call for the next step has to be ordered behind the steps that
 * read the last one (the same stream does), or write another result.
 *
 * Arithmetic: squares and sums are float64 (no finite gradient over- or
 * underflows them), in a fixed order, and so are N and the factor before
 * their one rounding to float32. N beyond float32's range is reported as
 * infinity while the factor stays right; a factor below 2^-126 loses bits as
 * any subnormal number does. out is the float32 product g * factor, rounded
 * to nearest even for bf16. NaN and infinities propagate: a NaN makes N and
 * the factor NaN; otherwise an infinite gradient makes N infinite and, with
 * a finite max_norm, the factor 0 (which clears the finite gradients and
 * turns infinite ones into NaN), so a caller that wants to skip such a step
 * tests N.
 *
 * Conventions are those of muon.h: pointers are device memory owned by the
 * caller, arguments are validated before any work is enqueued, work is
 * asynchronous on `stream`, results are deterministic (equal inputs give
 * bitwise-equal outputs), no call allocates except plan creation, and every
 * call can be captured into a graph.
 */
#ifndef MUON_CLIP_H
#define MUON_CLIP_H

#include <stddef.h>
#include <stdint.h>

#include "muon.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest number of elements (of a tensor, and of all together; strides
 * count as elements skipped) and list length accepted, else MUON_E_SHAPE. */
#define MUON_CLIP_MAX_NUMEL 1099511627776LL /* 2^40 */
#define MUON_CLIP_MAX_TENSORS 1048576

/* One gradient tensor: row-major, element (i, j) at grad + i * ld + j and
 * out + i * out_ld + j, both of type dtype and aligned to its size; a
 * contiguous tensor of any shape is one row of all its elements. rows == 0
 * or cols == 0 is an empty tensor (N_i = 0; its pointers are ignored). out
 * may be NULL (the plan then computes norms only), equal to grad with the
 * same ld (in place), or a buffer of its own. What is written may not
 * overlap anything else of the list, else MUON_E_INVALID; what is only read
 * may. Tensors count from their first to their last element, except column
 * slices of one matrix: where such ranges run into each other, all of them
 * with one row stride, tensors in disjoint columns do not overlap. */
typedef struct {
  int64_t rows;
  int64_t cols;
  int64_t ld;
  int64_t out_ld;
  const void* grad;
  void* out;
  int32_t dtype; /* muon_dtype */
  int32_t reserved; /* 0 */
} muon_clip_tensor;

/* Per-call scalars. max_norm >= 0 (infinity: no limit); eps >= 0 and
 * finite (1e-6 is the usual value); grad_mul > 0 and finite. Otherwise
 * MUON_E_INVALID. */
typedef struct {
  float max_norm;
  float eps;
  float grad_mul;
} muon_clip_config;

/* What a call leaves in device memory. */
typedef struct {
  float norm;   /* N */
  float scale;  /* the factor, grad_mul included */
} muon_clip_result;

typedef struct muon_clip_plan_s muon_clip_plan;

/* Bytes of device workspace a call on this list needs (host only, no device
 * calls; 0 is never returned for a valid list). */
muon_status muon_clip_workspace_bytes(const muon_clip_tensor* ts, int32_t n, size_t* bytes);

/* Validates the list, splits it into work items and uploads them to the
 * current device (a few KB to MB owned by the plan; *plan receives NULL on
 * error). The plan keeps no state between calls. */
muon_status muon_clip_plan_create(const muon_clip_tensor* ts, int32_t n, muon_clip_plan** plan);

/* Enqueues the norm: writes *result (device memory, 4-byte aligned) and,
 * unless norms is NULL, N_i into norms[i] (n floats of device memory).
 * Gradients are only read. `workspace` must hold at least
 * muon_clip_workspace_bytes bytes, 256-byte aligned; its contents need not
 * be initialised. Calls that overlap in time (other streams, graphs replayed
 * at once) need a workspace, a result and a norms array each. None of the
 * three may overlap another one or any tensor of the list. */
muon_status muon_clip_plan_norm(muon_clip_plan* plan, const muon_clip_config* cfg,
                                muon_clip_result* result, float* norms, void* workspace,
                                size_t workspace_bytes, void* stream);

/* muon_clip_plan_norm, then out_i = g_i * factor for every tensor.
 * MUON_E_INVALID if a non-empty tensor of the plan has no out. */
muon_status muon_clip_plan_step(muon_clip_plan* plan, const muon_clip_config* cfg,
                                muon_clip_result* result, float* norms, void* workspace,
                                size_t workspace_bytes, void* stream);

/* Frees a plan after waiting for the device (NULL is a no-op). A captured
 * graph reads the plan's tables: it must not be replayed afterwards. */
void muon_clip_plan_destroy(muon_clip_plan* plan);

#ifdef __cplusplus
}
#endif

#endif /* MUON_CLIP_H */
