/* fp4q_kv.h -- serving attention over an MXFP4 key/value cache on gfx950.
 *
 * Between the q/k/v product and the output product of a layer: norm and
 * rotation of each head, quantization of keys and values into the pages of
 * a cache held in 4 bits, and attention that reads those pages.  "Resumo
 * Tecnico: ScaleSweep" (4. Resultados) quantizes the key/value cache beside
 * weights and activations; "Bridging the Gap Between Promise and Performance
 * for Microscaling FP4 Quantization" (2. Metodologia, component 3) rotates
 * operands by a block Hadamard matrix that cancels in their product, which
 * holds for queries and keys too (H H^T = I).
 *
 * Conventions of every call, beyond those of fp4q.h
 *   - Tensors of heads are [tokens][heads][head_dim] with a dense last axis
 *     and given strides (elements) of the other two; head_dim is 64, 128 or
 *     256, and a tensor has fewer than 2^33 elements, the last of them less
 *     than 2^60 elements from the first.  Pointers are 16-byte aligned and
 *     the strides, in bytes, multiples of 16.
 *   - The cache is described by fp4q_kv_cache_t (host memory, read during the
 *     call).  A slot number s names row s % page_size of page s / page_size.
 *   - Data errors set bits of the status word at byte 0 of the workspace, as
 *     described in fp4q.h.  No data error makes a call read or write outside
 *     the given tensors: an index out of range is not followed.
 *   - Calls on one stream run in order.  The library allocates nothing and
 *     keeps no state, so every call can be captured into a HIP graph.
 */
#ifndef FP4Q_KV_H
#define FP4Q_KV_H

#include <stddef.h>
#include <stdint.h>

#include "fp4q.h"

#ifdef __cplusplus
extern "C" {
#endif

/* further bits of the device status word */
#define FP4Q_DATA_BAD_POSITION 0x40u /* a position outside the rotation table */
#define FP4Q_DATA_BAD_SLOT 0x80u     /* a slot number past the end of the cache */
#define FP4Q_DATA_BAD_TABLE 0x100u   /* a page number, sequence length or row offset out of range */

/* An MXFP4 key/value cache: rows of head_dim elements, one per (page, head,
 * row of the page), for keys and for values.  A row's codes are
 * head_dim / 2 bytes (element 2i in the low nibble of byte i) and its scales
 * head_dim / 32 E8M0 bytes, exactly a row that fp4q_quantize_mxfp4 writes.
 *   codes of (p, h, r) start at p * page_stride + h * head_stride +
 *   r * token_stride (bytes), the same for keys and values; scales start at
 *   a sixteenth of that offset, so they lie in the same order as the codes.
 *   Strides are multiples of 16 and do not make rows overlap, token_stride is
 *   at most 2^26, the code pointers are 16-byte aligned, page_size is a power of two from 16 to
 *   1024, heads * head_dim at most 65536, and pages * page_size * heads below
 *   2^40.  Any byte may be in the rows that no token was written to. */
typedef struct fp4q_kv_cache {
  uint8_t *k_codes, *k_scales, *v_codes, *v_scales; /* device */
  int64_t pages;
  int32_t page_size, heads, head_dim;
  int64_t page_stride, head_stride, token_stride;
} fp4q_kv_cache_t;

/* How the heads of queries or keys are normed and rotated.
 *   norm_weight [head_dim] float32, or NULL for no norm;  eps >= 0.
 *   positions   [tokens] int64 and
 *   table       [table_positions][rotary_dim] float32, 16-byte aligned: the
 *               cosines, then the sines, of a position's rotary_dim / 2
 *               angles (any scaling for long contexts is in them).  Both
 *               NULL for no rotation.
 *   rotary_dim  a multiple of 16, at most head_dim: the first rotary_dim
 *               elements of a head are rotated, the rest are left.
 *   interleaved 0: element i is paired with i + rotary_dim / 2;
 *               1: element 2i with 2i + 1.
 *   hadamard_n  0, or 16, 32, 64, 128 (at most head_dim): the groups of n
 *               elements times H_n / sqrt(n) at the end.
 *
 * Computation, for a head x (every float32 step rounds to nearest even, none
 * fused):
 *   r = fp32(1 / sqrt(sum x_i^2 / head_dim + eps)), in float64 up to the last
 *   rounding; y_i = fp32(fp32(x_i * r) * norm_weight_i);
 *   a pair (a, b) with (c, s) becomes (fp32(fp32(a c) - fp32(b s)),
 *   fp32(fp32(b c) + fp32(a s)));
 *   then fp4q_block_hadamard's stages.
 * A position outside 0 .. table_positions - 1 sets FP4Q_DATA_BAD_POSITION
 * and its token's results are unspecified. */
typedef struct fp4q_head_map {
  const float *norm_weight;
  double eps;
  const int64_t *positions;
  const float *table;
  int64_t table_positions;
  int32_t rotary_dim, interleaved, hadamard_n;
} fp4q_head_map_t;

/* Norm and rotation of each head of x, rounded once to the output type.
 *   x, dtype, tokens, heads, head_dim, token_stride, head_stride  the input
 *            (FP4Q_F32 or FP4Q_BF16).
 *   map      what is done (host memory).
 *   out_dtype, out  [tokens][heads][head_dim], dense, 16-byte aligned; out
 *            may be x itself where x is dense and of the same type, and must
 *            not overlap it otherwise.
 *   workspace  fp4q_workspace_bytes() bytes (status word).
 * Inf and NaN propagate. */
fp4q_status_t fp4q_rotate_heads(const void *x, fp4q_dtype_t dtype, int64_t tokens, int64_t heads, int64_t head_dim,
                                int64_t token_stride, int64_t head_stride, const fp4q_head_map_t *map,
                                fp4q_dtype_t out_dtype, void *out, void *workspace, size_t workspace_bytes,
                                void *stream);

/* Quantizes the keys and values of tokens into cache slots: keys through
 * fp4q_rotate_heads's computation (in float32, not rounded to a shorter type
 * in between), then both through fp4q_quantize_mxfp4's with the same window
 * and the MSE loss.  The rows written are bit for bit those of that call.
 *   k, v, dtype  [tokens][cache->heads][cache->head_dim] with their strides.
 *   slots    [tokens] int64.  A negative slot skips its token; one past the
 *            cache sets FP4Q_DATA_BAD_SLOT and is skipped.  The slots of a
 *            call that are not negative are distinct: a slot given twice is
 *            left with an unspecified mix of its tokens' rows.
 *   off_lo, off_hi  the exponent window, -16 <= off_lo <= 0 <= off_hi <= 16.
 * Rows of other slots are left as they are.  A non-finite key (after the
 * map) or value of a token that is written sets FP4Q_DATA_NONFINITE_INPUT and
 * leaves its row unspecified. */
fp4q_status_t fp4q_kv_append_mxfp4(const fp4q_kv_cache_t *cache, const void *k, int64_t k_token_stride,
                                   int64_t k_head_stride, const void *v, int64_t v_token_stride,
                                   int64_t v_head_stride, fp4q_dtype_t dtype, int64_t tokens, const int64_t *slots,
                                   const fp4q_head_map_t *map, int off_lo, int off_hi, void *workspace,
                                   size_t workspace_bytes, void *stream);

/* The decoded rows of cache slots: k_out and v_out [tokens][heads][head_dim]
 * dense, 16-byte aligned, float32 (exact) or bfloat16 (exact unless the
 * value is below bfloat16's normal range).  Either may be NULL.  A negative
 * slot gives zeros; one past the cache too, and sets FP4Q_DATA_BAD_SLOT. */
fp4q_status_t fp4q_kv_read_mxfp4(const fp4q_kv_cache_t *cache, const int64_t *slots, int64_t tokens,
                                 fp4q_dtype_t out_dtype, void *k_out, void *v_out, void *workspace,
                                 size_t workspace_bytes, void *stream);

/* Attention of q over the cached keys and values of each sequence:
 *   out = softmax(scale * q K^T + mask) V
 * for every row of q and every query head, head h of q_heads on cache head
 * h / (q_heads / cache->heads).
 *   q        [tokens][q_heads][cache->head_dim] bfloat16 with its strides
 *            (rotated, by the caller); q_heads a multiple of cache->heads.
 *   batch    sequences; sequence b has seq_lens[b] cached tokens, whose token
 *            j is row j % page_size of page block_table[b * table_stride +
 *            j / page_size], and the rows cu_q[b] .. cu_q[b + 1] - 1 of q,
 *            its last tokens (already in the cache).  cu_q NULL: one row
 *            each, tokens == batch.
 *   block_table, seq_lens, cu_q  int32, 4-byte aligned; table_width is the
 *            number of entries of a row of the table.  Entries past a
 *            sequence's last page are not read.  block_table may be NULL
 *            where max_len is 0.
 *   max_new, max_len  no sequence has more rows of q, or more cached tokens
 *            (max_new at most tokens, max_len at most table_width * page_size
 *            and 2^30).
 *   causal   1: row i of n sees the keys up to its own position, seq_len - n
 *            + i; 0: every key.
 *   window   0: no limit; w > 0 (below 2^31): no row sees keys at its
 *            position minus w or before.
 *   scale    factor of the scores (float32), at most 2^127 in magnitude.
 *   out      [tokens][q_heads][head_dim] bfloat16, dense, 16-byte aligned;
 *            it must not overlap the inputs.
 *   lse      [tokens][q_heads] float32 natural logarithm of the row's sum of
 *            exp(scores), or NULL.
 * A row that sees no key gets zeros and minus infinity.  Rows of q that
 * belong to no sequence are left as they are in out and lse.
 *   workspace  fp4q_attention_mxfp4_workspace_bytes() bytes, 16-byte aligned
 *            (status word at byte 0; partial results).  Calls that may
 *            overlap need one each.
 *
 * Arithmetic: keys and values are decoded to bfloat16, which holds them
 * exactly (above its normal range's lower end), so products with q are
 * exact.  Scores, the softmax's maximum and sum, and the outputs are
 * accumulated in float32; probabilities enter the second product rounded to
 * bfloat16, as the matrix core takes them.  The result does not depend on
 * anything but the arguments (no atomics on results).
 *
 * Data errors: a page number outside 0 .. pages - 1 (its tokens count as
 * masked), a sequence length or row offset outside its bounds (cut to them)
 * set FP4Q_DATA_BAD_TABLE and leave that sequence's rows unspecified, and row
 * offsets that decrease those of every sequence.  Bytes
 * of tokens that no row of a sequence sees do not matter, whatever they are;
 * a key or value scale of 255 (NaN) that some row sees can reach the other
 * rows of its sequence.
 *
 * Returns FP4Q_ERR_NULL, FP4Q_ERR_WORKSPACE, FP4Q_ERR_ARG, FP4Q_ERR_SHAPE,
 * FP4Q_ERR_ALIGN or FP4Q_ERR_HIP. */
fp4q_status_t fp4q_attention_mxfp4(const fp4q_kv_cache_t *cache, const void *q, int64_t q_token_stride,
                                   int64_t q_head_stride, int64_t tokens, int64_t q_heads,
                                   const int32_t *block_table, int64_t table_stride, int64_t table_width,
                                   int64_t batch, const int32_t *seq_lens, const int32_t *cu_q, int64_t max_new,
                                   int64_t max_len, float scale, int causal, int64_t window, void *out, float *lse,
                                   void *workspace, size_t workspace_bytes, void *stream);

/* Workspace of such a call: a header, and the partial results of sequences
 * that several workgroups share.  0 for invalid sizes. */
size_t fp4q_attention_mxfp4_workspace_bytes(int64_t tokens, int64_t batch, int64_t q_heads, int64_t heads,
                                            int64_t head_dim, int64_t max_new, int64_t max_len, int64_t window);

#ifdef __cplusplus
}
#endif

#endif /* FP4Q_KV_H */
