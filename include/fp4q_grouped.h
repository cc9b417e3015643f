/* fp4q_grouped.h -- products whose rows choose their weights, on gfx950.
 *
 * Beside the products of fp4q_gemm.h, where every row meets the same
 * weights: routing of tokens to experts, the experts' MXFP4 products, the
 * weighted sum of what they give, and low-rank adapters of many requests
 * beside a shared projection.  The pages know FP4 weights of models with
 * experts ("TORQ": a 30B model with 3B active parameters) and W4A4 products
 * ("Bridging the Gap Between Promise and Performance for Microscaling FP4
 * Quantization", 2. Metodologia).
 *
 * Conventions of every call, beyond those of fp4q.h
 *   - An entry is a row that belongs to at most one group (an expert, an
 *     adapter).  Entries are numbered from 0; those that a token's top_k
 *     choices make are numbered token * top_k + choice.
 *   - fp4q_row_groups_t lists the entries by group.
 *   - Data errors set bits of the status word at byte 0 of the workspace, as
 *     described in fp4q.h.  No data error makes a call read or write outside
 *     the given tensors: a number out of range is not followed.
 *   - Calls on one stream run in order.  The library allocates nothing and
 *     keeps no state, so every call can be captured into a HIP graph.  Calls
 *     that may overlap need a workspace each.
 */
#ifndef FP4Q_GROUPED_H
#define FP4Q_GROUPED_H

#include <stddef.h>
#include <stdint.h>

#include "fp4q.h"

#ifdef __cplusplus
extern "C" {
#endif

/* further bit of the device status word: a group number past the last, or
 * offsets or entry numbers of a fp4q_row_groups_t out of range */
#define FP4Q_DATA_BAD_GROUP 0x200u

/* Entries by group (device memory, 4-byte aligned):
 *   offsets [groups + 1]  group g's entries are rows[offsets[g]] ..
 *           rows[offsets[g + 1] - 1]; offsets[0] is 0, and they do not decrease.
 *   rows    [entries]  the entries' numbers, each once: by group, ascending
 *           within a group, those of no group last (also ascending).
 *   groups  1 .. 2048;  entries  0 .. 2^30.
 * Rows of results of an entry that is listed twice are unspecified. */
typedef struct fp4q_row_groups {
  const int32_t *offsets, *rows;
  int64_t groups, entries;
} fp4q_row_groups_t;

/* The entries of ids sorted by group (stable).
 *   ids      [entries] int32: the entry's group; negative: none.  One past
 *            the last group sets FP4Q_DATA_BAD_GROUP and counts as none.
 *   offsets, rows  written as fp4q_row_groups_t describes them.
 *   workspace  fp4q_group_rows_workspace_bytes() bytes, 16-byte aligned. */
fp4q_status_t fp4q_group_rows(const int32_t *ids, int64_t entries, int64_t groups, int32_t *offsets, int32_t *rows,
                              void *workspace, size_t workspace_bytes, void *stream);
size_t fp4q_group_rows_workspace_bytes(int64_t entries, int64_t groups);

typedef enum fp4q_score { FP4Q_SOFTMAX = 0, FP4Q_SIGMOID = 1 } fp4q_score_t;

/* How experts are chosen.
 *   score    FP4Q_SOFTMAX: over all experts; FP4Q_SIGMOID: of each logit.
 *   bias     [experts] float32 added to the scores for the choice alone, or
 *            NULL.  Minus infinity turns an expert off.
 *   top_k    experts for each token, 1 .. 64 and at most `experts`.
 *   n_groups, top_groups  the experts in n_groups runs of equal length (at
 *            most 64), of which a token chooses within the top_groups best;
 *            n_groups 1: all of them.
 *   group_best  1 or 2: a group counts as the sum of its that many best
 *            choices (of one, where it has no second).
 *   renormalize  1: the weights of a token's choices are divided by their sum.
 *   scale    factor of the weights. */
typedef struct fp4q_router {
  fp4q_score_t score;
  const float *bias;
  int32_t top_k, n_groups, top_groups, group_best, renormalize;
  float scale;
} fp4q_router_t;

/* Routing: the top_k experts of each token and their weights.
 *   logits, dtype  [tokens][experts], rows ld elements apart (FP4Q_F32 or
 *            FP4Q_BF16, aligned to its type); experts 1 .. 1024.
 *   weights  [tokens][top_k] float32; chosen [tokens][top_k] int32, best
 *            first.
 *   offsets, rows  the entries by expert as fp4q_group_rows gives them for
 *            chosen (both NULL: not wanted).
 *   workspace  fp4q_route_experts_workspace_bytes() bytes, 16-byte aligned.
 *
 * Choices compare scores + bias (groups: their sums) in float64, and without
 * a bias the logits themselves; ties go to the lowest index.  Weights are the
 * scores without the bias, renormalised and scaled, rounded once.
 * A logit of minus infinity, or a bias of minus infinity, turns its expert
 * off: it is never chosen.  Choices that a token lacks are -1 with weight 0,
 * and belong to no group; where the weights' sum is 0 they stay 0.
 * A token with a NaN or plus infinity among its logits, or among its scores
 * with the bias added, sets FP4Q_DATA_NONFINITE_INPUT and makes no choices. */
fp4q_status_t fp4q_route_experts(const void *logits, fp4q_dtype_t dtype, int64_t tokens, int64_t experts, int64_t ld,
                                 const fp4q_router_t *router, float *weights, int32_t *chosen, int32_t *offsets,
                                 int32_t *rows, void *workspace, size_t workspace_bytes, void *stream);
size_t fp4q_route_experts_workspace_bytes(int64_t tokens, int64_t experts, int64_t top_k);

/* Grouped MXFP4 product: for every entry e of group g
 *   C[e] = alpha * A_hat[row(e)] * B_hat[g]^T.
 *   a_codes, a_scales  a_rows rows of k elements, as for fp4q_gemm_mxfp4.
 *   b_codes, b_scales  [groups->groups][n][k] MXFP4: a matrix for each group.
 *   gather   0: A has a row for each entry, in the order of groups->rows.
 *            f > 0: entry e takes row e / f (f = top_k: the token's).
 *   scatter  0: C's rows are in the order of groups->rows.  1: row e of C is
 *            entry e's.
 *   gated    1: n is even, and of the n products the first half are gates:
 *            C has n / 2 columns, silu(gate) * up, with silu(z) =
 *            z / (1 + exp(-z)) in float32, off by at most 7 * 2^-24 of it.
 *   c, ldc, out_dtype  [groups->entries] rows of n (n / 2) columns,
 *            FP4Q_F32 or FP4Q_BF16; it must not overlap the inputs.
 *   workspace  fp4q_workspace_bytes() bytes (status word).
 * Rows of C that belong to entries of no group are left as they are.
 *
 * n >= 0; k > 0 and a multiple of 32; with f > 0 a_rows * f, else a_rows, is
 * at least the number of entries.  a_codes and b_codes 16-byte, the scales
 * 4-byte aligned where k is a multiple of 128.  A call of more than 2^22
 * output tiles (about 2^36 values of C) is refused with FP4Q_ERR_SHAPE.
 *
 * Arithmetic: as fp4q_gemm_mxfp4's (products of decoded elements are exact,
 * sums are float32); the order of a sum depends on n, k and the numbers of
 * groups, entries and rows of A, and not on what the rows hold. */
fp4q_status_t fp4q_gemm_mxfp4_grouped(const uint8_t *a_codes, const uint8_t *a_scales, int64_t a_rows,
                                      const uint8_t *b_codes, const uint8_t *b_scales,
                                      const fp4q_row_groups_t *groups, int64_t n, int64_t k, int64_t gather,
                                      int scatter, int gated, float alpha, fp4q_dtype_t out_dtype, void *c,
                                      int64_t ldc, void *workspace, size_t workspace_bytes, void *stream);

/* The same, and rows of C that belong to entries of no group become zeros:
 * for a fresh C that is read as a whole, as fp4q_quantize_mxfp4 does. */
fp4q_status_t fp4q_gemm_mxfp4_grouped_zeroed(const uint8_t *a_codes, const uint8_t *a_scales, int64_t a_rows,
                                             const uint8_t *b_codes, const uint8_t *b_scales,
                                             const fp4q_row_groups_t *groups, int64_t n, int64_t k, int64_t gather,
                                             int scatter, int gated, float alpha, fp4q_dtype_t out_dtype, void *c,
                                             int64_t ldc, void *workspace, size_t workspace_bytes, void *stream);

/* out[t] = sum over j of weights[t][j] * y[t * top_k + j], plus add[t].
 *   y, dtype  [tokens * top_k] rows of n, ld_y elements apart.
 *   weights  [tokens][top_k] float32; chosen [tokens][top_k] int32 or NULL:
 *            rows of negative choices are not read.
 *   add      [tokens] rows of n, ld_add apart, of out's type, or NULL; it may
 *            be out itself.
 *   out, out_dtype  [tokens] rows of n, ld_out apart; it must not overlap y.
 * float32 sums in the order of j, add last, rounded once.  top_k 1 .. 64.
 * Pointers aligned to their type.  Where the rows of y, add and out are all
 * 16-byte aligned and n is a multiple of 8, a call of 2^24 or more pieces of
 * 2048 columns, else of 256, is refused with FP4Q_ERR_SHAPE. */
fp4q_status_t fp4q_combine_experts(const void *y, fp4q_dtype_t dtype, int64_t tokens, int64_t top_k, int64_t n,
                                   int64_t ld_y, const float *weights, const int32_t *chosen, const void *add,
                                   int64_t ld_add, fp4q_dtype_t out_dtype, void *out, int64_t ld_out, void *stream);

/* Low-rank adapters beside a shared projection: for every entry e of group g
 *   out[e] = y[e] + scales[g] * (x[e] A[g]^T) B[g]^T,
 * and out[e] = y[e] for entries of no group.
 *   y, out, dtype  [groups->entries] rows of n, ld_y and ld_out apart
 *            (FP4Q_F32 or FP4Q_BF16); out is y itself or does not overlap it.
 *   x        bfloat16 [groups->entries] rows of k, ld_x apart.
 *   a        bfloat16 [groups][rank][k];  b  bfloat16 [groups][n][rank].
 *   scales   [groups] float32, or NULL for 1.
 *   k and rank multiples of 8, rank 8 .. 256; n >= 0.  x, a and b 16-byte
 *   aligned, ld_x a multiple of 8; y and out aligned to their type.
 *   workspace  fp4q_lora_add_workspace_bytes() bytes, 16-byte aligned.
 *
 * Arithmetic: products are exact; x A^T is summed in float32, multiplied by
 * the scale, and enters the second product as three bfloat16 parts that hold
 * its 24 bits; one rounding at the end.  Elements of b that are not finite
 * give infinities or NaN in their column.  The order of a sum depends on the
 * sizes alone.  A call of more than 2^22 tiles (of 16 rows or more and 256
 * columns) is refused with FP4Q_ERR_SHAPE. */
fp4q_status_t fp4q_lora_add(const void *y, fp4q_dtype_t dtype, int64_t ld_y, const void *x, int64_t ld_x,
                            const void *a, const void *b, const float *scales, const fp4q_row_groups_t *groups,
                            int64_t n, int64_t k, int64_t rank, void *out, int64_t ld_out, void *workspace,
                            size_t workspace_bytes, void *stream);
size_t fp4q_lora_add_workspace_bytes(int64_t entries, int64_t groups, int64_t n, int64_t k, int64_t rank);

#ifdef __cplusplus
}
#endif

#endif /* FP4Q_GROUPED_H */
