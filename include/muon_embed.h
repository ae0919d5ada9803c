/*
 * muon_embed.h -- C ABI of a model's embedding table on the Adam path: the
 * lookup of its rows, the gradient of that lookup by sorted tokens, and the
 * Adam step of the rows a batch has touched.
 *
 * For a table E (vocab x cols), tokens t_0 .. t_{n-1} and a scale s:
 *
 *   lookup          out_i = s E[t_i]
 *   gradient        G[v]  = s sum of dout_i over all i with t_i = v
 *   gradient_rows   the v with at least one token, ascending, their G[v], and
 *                   how many there are
 *   adam_rows       the update of muon_adam.h on those rows of E and of its
 *                   moments; all other rows stay as they are
 *
 * A token outside [0, vocab) (-1 for padding, say) looks up a row of zeros
 * and carries no gradient; nothing is read or written through it.
 *
 * The embeddings take the Adam path (mhpq.cn, modded-nanogpt track_1_short
 * technical guide, section 6.2: every parameter that is not a projection
 * matrix). Of a GPT-2 124M's 39.5 M parameters on that path the token
 * embedding holds 38.6 M, of which one batch touches a fraction: adam_rows
 * reads and writes those rows alone. It is not the dense step: rows without
 * a token are not decayed and their moments do not fade.
 *
 * Arithmetic: out is the float32 product, rounded once to its type. Sums are
 * taken in an order fixed by the batch's tokens: a token's positions ascending,
 * in float32 runs of at most 64, whose sums are added in float64, so that no
 * sum is further off than 63 float32 roundings of what it adds up, however
 * long. It is then rounded to float32, multiplied by s and
 * rounded once to the table's type (with `accumulate` after the float32
 * addition to what grad holds).
 *
 * Conventions are those of muon.h: pointers are device memory owned by the
 * caller, arguments are validated before any work is enqueued, work is
 * asynchronous on `stream`, results are deterministic (equal inputs give
 * bitwise-equal outputs), NaN and infinities propagate, no call allocates
 * except plan creation, and every call can be captured into a graph. Buffers
 * that must not overlap (MUON_E_INVALID) are taken from their first element to
 * their last, the gaps between rows included.
 */
#ifndef MUON_EMBED_H
#define MUON_EMBED_H

#include <stddef.h>
#include <stdint.h>

#include "muon.h"
#include "muon_adam.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Limits (MUON_E_SHAPE beyond them; also above 2^23 runs of 64 tokens x 256
 * columns begun in a batch, 2^24 tokens of 8192 columns). */
#define MUON_EMBED_MAX_VOCAB 16777216  /* 2^24 */
#define MUON_EMBED_MAX_TOKENS 16777216 /* 2^24 */
#define MUON_EMBED_MAX_COLS 65536
#define MUON_EMBED_MAX_LD 1099511627776LL /* 2^40 elements from row to row */

/* The table: row-major, element (v, j) at table + v * ld + j, aligned to its
 * element size. The moments (vocab x cols, contiguous float32, 4-byte
 * aligned) are needed by adam_rows only; both may be NULL. None of the three
 * may overlap another. lr_mul and wd_mul as in muon_adam.h. */
typedef struct {
  int64_t vocab;
  int64_t cols;
  int64_t ld;
  void* table;
  float* exp_avg;
  float* exp_avg_sq;
  float lr_mul;
  float wd_mul;
} muon_embed_table;

/* n tokens: int32 (wide = 0) or int64 (wide = 1), aligned to their size. */
typedef struct {
  const void* data;
  int64_t n;
  int32_t wide;
  int32_t reserved; /* 0 */
} muon_embed_tokens;

/* n rows of cols elements, one per token, of either element type (not
 * necessarily the table's), ld elements apart. */
typedef struct {
  void* data;
  int64_t ld;
  int32_t dtype;    /* muon_dtype */
  int32_t reserved; /* 0 */
} muon_embed_acts;

typedef struct muon_embed_plan_s muon_embed_plan;

/* Bytes of device workspace gradient and gradient_rows need for up to
 * max_tokens tokens (host only, no device calls; never 0 for valid sizes). */
muon_status muon_embed_workspace_bytes(int64_t vocab, int64_t cols, int64_t max_tokens,
                                       size_t* bytes);

/* Validates the table (of element type dtype) and binds a plan to it and to
 * the current device. The plan holds no device memory and no state between
 * calls. *plan receives NULL on error. */
muon_status muon_embed_plan_create(const muon_embed_table* table, muon_dtype dtype,
                                   int64_t max_tokens, muon_embed_plan** plan);

/* out_i = scale E[t_i], rounded to out's type. `out` must not overlap the
 * table or the tokens. At most max_tokens tokens (all calls), else
 * MUON_E_SHAPE; n == 0 does nothing. scale must be finite (all calls). */
muon_status muon_embed_plan_lookup(muon_embed_plan* plan, const muon_embed_tokens* tokens,
                                   float scale, const muon_embed_acts* out, void* stream);

/* G into grad (vocab x cols of the table's type, row-major, grad_ld >= cols):
 * accumulate = 0 writes every row (zeros where there is no token, everywhere
 * for n == 0), accumulate = 1 adds to the rows that have tokens and leaves
 * the others. dout is read only. `workspace` must hold at least
 * muon_embed_workspace_bytes bytes, 256-byte aligned; its contents need not
 * be initialised, and calls that overlap in time need one each. grad must
 * not overlap the workspace, dout, the tokens, the table or its moments. */
muon_status muon_embed_plan_gradient(muon_embed_plan* plan, const muon_embed_tokens* tokens,
                                     const muon_embed_acts* dout, float scale, void* grad,
                                     int64_t grad_ld, int32_t accumulate, void* workspace,
                                     size_t workspace_bytes, void* stream);

/* G as rows: rows[r] (int32, ascending) and values (row r contiguous behind
 * row r - 1, cols elements of the table's type) for r < *count. Both have room
 * for min(n, vocab) rows; those behind *count are left as they are. What is
 * written must not overlap anything else of the call, the table or its
 * moments. */
muon_status muon_embed_plan_gradient_rows(muon_embed_plan* plan, const muon_embed_tokens* tokens,
                                          const muon_embed_acts* dout, float scale, int32_t* rows,
                                          void* values, int32_t* count, void* workspace,
                                          size_t workspace_bytes, void* stream);

/* One Adam update (muon_adam.h: the same expressions, multipliers and
 * scalars) of rows rows[r] of the table and its moments with gradients
 * values[r], r < *count, as gradient_rows leaves them. At most `capacity`
 * rows are taken, whatever *count says. rows must be distinct; a row outside
 * the table is skipped. MUON_E_INVALID without moments. */
muon_status muon_embed_plan_adam_rows(muon_embed_plan* plan, const muon_adam_config* cfg,
                                      const int32_t* rows, const void* values,
                                      const int32_t* count, int64_t capacity, void* stream);

/* Attaches a gradient factor in device memory to adam_rows (NULL detaches
 * it), as muon_adam_plan_set_grad_scale does: values * *scale in place of
 * values. With muon_clip_plan_set_live_rows (muon_clip.h) the factor comes
 * from a norm over the live rows of `values` and the other gradients. */
muon_status muon_embed_plan_set_grad_scale(muon_embed_plan* plan, const float* scale);

/* Frees a plan (NULL is a no-op). */
void muon_embed_plan_destroy(muon_embed_plan* plan);

#ifdef __cplusplus
}
#endif

#endif /* MUON_EMBED_H */
