/*
 * ds_token_rows.h -- the row operators at a model's two ends and at its heads,
 * on AMD Instinct MI355X (gfx950).  Same library, conventions, status codes
 * and stream handle as ds_rows.h.
 *
 *  ds_embed_rows             rows of an embedding table by token id, scaled
 *  ds_embed_rows_backward    the table's gradient, summed token by token
 *  ds_qk_rows_rms            q and k heads: RMS norm with a learned weight,
 *                            then rotate-half RoPE, in one pass (ds_qk_rows_l2
 *                            is the unit-length form that rotates first)
 *  ds_qk_rows_rms_backward   its gradient, for q, k and both weights
 *  ds_logprob_rows           per row of logits: the log probability of a given
 *                            token, the entropy, the top alternatives
 *  ds_logprob_rows_backward  the gradient of log probability and entropy, for
 *                            the logits and their column scale
 *
 * Numerics.  bf16 values are passed as their 16-bit patterns.  Everything is
 * computed in fp32 (a rotation's angle in fp64) and rounded once, to nearest
 * even, into each bf16 output.  Sums are held in fp32 or more.
 *
 * Determinism.  The bits of an output row depend on that row's inputs and the
 * row width alone, not on the row count, the grid or the stream.  A gradient
 * that sums over rows (an embedding row, the q/k weights, the logits' column
 * scale) is summed in an order fixed by the sizes (and, for an embedding, by
 * the ids); repeated calls give identical bits.  No atomic adds a float.
 *
 * Errors, ownership, streams: as in ds_rows.h.  Every argument is checked
 * before anything is enqueued.  All calls may be captured into a HIP graph.
 * The library allocates nothing: calls that need scratch memory take a
 * `workspace` of the caller's, of at least the size that their _workspace
 * function returns for the same sizes (16-byte aligned device memory; NULL
 * where that size is 0).  Its contents before the call do not matter, and two
 * calls that may run at the same time need a workspace each.
 */
#ifndef DS_TOKEN_ROWS_H
#define DS_TOKEN_ROWS_H

#include "ds_rows.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DS_MAX_TOP 32                  /* most alternatives ds_logprob_rows lists */
#define DS_MAX_VOCAB 1048576           /* widest row of logits */

/* Element types of tables and logits. */
enum { DS_TYPE_BF16 = 0, DS_TYPE_F32 = 1 };

/*
 * ds_embed_rows -- out_i = bf16(scale * table[ids_i]), one fp32 product per
 * element.
 *
 * table    : [vocab, cols] of table_type, row-major, contiguous, 16-byte
 *            aligned: fp32 master weights, or a bf16 W_eff as
 *            ds_weight_rownorm_gain makes it.
 * ids      : [rows] token ids, int32 (id_bytes 4) or int64 (id_bytes 8),
 *            aligned to their size.  An id below 0 or at or beyond vocab
 *            (padding, another shard's token) gives a row of zeros.
 * scale    : finite (sqrt(cols) in models that scale their embeddings).
 * out      : [rows, cols] bf16 bit patterns, contiguous, 16-byte aligned, not
 *            overlapping table or ids.
 * rows     : >= 0 (0: no-op).  vocab: 0 <= vocab < 2^31.
 * cols     : multiple of 8, 8 <= cols <= DS_MAX_COLS.
 */
int ds_embed_rows(const void* table, int32_t table_type, int64_t vocab, const void* ids,
                  int32_t id_bytes, float scale, uint16_t* out, int64_t rows, int64_t cols,
                  ds_stream_t stream);

/*
 * ds_embed_rows_backward -- the gradient of ds_embed_rows for its table.
 *
 *   dtable[t] = scale * sum_{i : ids_i = t} dy_i              (accumulate 0)
 *   dtable[t] = dtable[t] + scale * sum_{i : ids_i = t} dy_i  (accumulate 1)
 *
 * The rows of one token are summed in fp32 in ascending i, long stretches of
 * them by runs of 32 rows first.  With accumulate 0 every row of dtable is written
 * (zeros for a token that does not occur); with 1 only the rows of tokens
 * that occur are touched, so a tied head's gradient may already be there.
 *
 * dy       : [rows, cols] bf16 bit patterns, contiguous, 16-byte aligned.
 * ids, id_bytes, scale, vocab, cols : the forward call's.  Ids outside
 *            [0, vocab) add to nothing.
 * dtable   : [vocab, cols] of grad_type (fp32, or bf16 as
 *            ds_weight_rownorm_gain_backward takes its dw_eff), contiguous,
 *            16-byte aligned, overlapping no input.
 * rows     : 0 <= rows <= 2^30; dy and dtable hold at most 400 GiB each.
 */
int ds_embed_rows_backward(const uint16_t* dy, const void* ids, int32_t id_bytes, float scale,
                           void* dtable, int32_t grad_type, int32_t accumulate, int64_t vocab,
                           int64_t rows, int64_t cols, void* workspace, int64_t workspace_bytes,
                           ds_stream_t stream);

/* Bytes of workspace of that call (a negative status for sizes it refuses). */
int64_t ds_embed_rows_backward_workspace(int64_t vocab, int64_t rows, int64_t cols);

/*
 * ds_qk_rows_rms -- q and k heads of a token row: RMS norm with a learned
 * weight per head dimension, then rotate-half RoPE.
 *
 * For each row with position p and each head x of q and of k (HD values):
 *   n   = x / sqrt(sum x^2 / HD + eps) * weight        q_weight or k_weight
 *   t_i = p * inv_freq_i                               in fp64, i < HD/2
 *   out = bf16([n1 cos t - n2 sin t, n2 cos t + n1 sin t])
 * with n1, n2 the halves of n; nothing is rounded to bf16 in between.
 *
 * q, q_out : [rows, ldq] / [rows, ldq_out] bf16 bit patterns, the first
 *            n_q_heads * head_dim elements of each row used; 16-byte aligned,
 *            strides multiples of 8.  q_out may be q itself (with ldq_out ==
 *            ldq); otherwise it must not overlap any input.
 * k, k_out : likewise for the n_kv_heads heads of k (may be NULL when
 *            n_kv_heads == 0).
 * positions: [rows] int32; 4-byte aligned.
 * inv_freq : [head_dim / 2] fp32; 16-byte aligned.  A frequency of 0 leaves
 *            its pair unrotated.
 * q_weight, k_weight : [head_dim] fp32, 16-byte aligned; NULL for weights of 1.
 * head_dim : multiple of 16, 16 <= head_dim <= 256.
 * eps      : finite, >= 0.  rows >= 0 (0: no-op).
 *
 * A head whose fp32 sum of squares overflows, or whose mean square plus eps
 * is below 2^-96, is summed again scaled by a power of two, as in ds_rows.h.
 */
int ds_qk_rows_rms(const uint16_t* q, int64_t ldq, const uint16_t* k, int64_t ldk,
                   const int32_t* positions, const float* inv_freq, const float* q_weight,
                   const float* k_weight, uint16_t* q_out, int64_t ldq_out, uint16_t* k_out,
                   int64_t ldk_out, int64_t rows, int32_t n_q_heads, int32_t n_kv_heads,
                   int32_t head_dim, float eps, ds_stream_t stream);

/*
 * ds_qk_rows_rms_backward -- the gradient of ds_qk_rows_rms.
 *
 * With u = x / sqrt(sum x^2 / HD + eps), D that root, and d the incoming
 * gradient of the head's output turned back by its angles:
 *   dweight += d * u               summed over rows and heads, in fp32
 *   dx       = bf16((w d - u <w d, u> / HD) / D)
 *
 * q .. k_weight, sizes, eps : the forward call's.
 * dq_out, dk_out : the gradients reaching q_out and k_out, rows of lddq_out /
 *            lddk_out elements; aligned as q and k.
 * dq, dk   : receive the gradients for q and k, rows of lddq / lddk elements;
 *            dq may be exactly dq_out or q (with its stride; likewise dk);
 *            otherwise no output overlaps an input or another output.
 * dq_weight, dk_weight : [head_dim] fp32, 4-byte aligned, or NULL when not
 *            wanted.  Written also where the weight was NULL (1).  rows == 0
 *            (or no heads) writes zeros.
 */
int ds_qk_rows_rms_backward(const uint16_t* q, int64_t ldq, const uint16_t* k, int64_t ldk,
                            const int32_t* positions, const float* inv_freq,
                            const float* q_weight, const float* k_weight, const uint16_t* dq_out,
                            int64_t lddq_out, const uint16_t* dk_out, int64_t lddk_out,
                            uint16_t* dq, int64_t lddq, uint16_t* dk, int64_t lddk,
                            float* dq_weight, float* dk_weight, int64_t rows, int32_t n_q_heads,
                            int32_t n_kv_heads, int32_t head_dim, float eps, void* workspace,
                            int64_t workspace_bytes, ds_stream_t stream);

/* Bytes of workspace of that call (needed only when a weight gradient is wanted). */
int64_t ds_qk_rows_rms_backward_workspace(int64_t rows, int32_t n_q_heads, int32_t n_kv_heads,
                                          int32_t head_dim);

/*
 * ds_logprob_rows -- what a row of logits says of a given token.
 *
 *   z_j     = x_j * scale_j * inv_temp         fp32 products in this order
 *   lse     = log sum_j exp z_j
 *   logp    = z_label - lse
 *   entropy = lse - sum_j p_j z_j,  p_j = exp(z_j - lse)
 *   top     : the top_k tokens of largest z, largest first, equal values in
 *             ascending token order, and their log probabilities z - lse
 * (log probabilities are formed as (z - max) - log sum exp(z - max), so a row
 * far from zero loses none of them)
 *
 * logits   : [rows, ld] of logits_type, the first vocab elements of each row
 *            used; ld >= vocab; aligned to the element (any row alignment).
 * scale    : [vocab] fp32, shared by all rows, 4-byte aligned; NULL for 1.
 * inv_temp : finite, > 0.
 * labels   : [rows] int32 or int64 (label_bytes); NULL when logp is NULL.  A
 *            label outside [0, vocab) marks a row to ignore: its logp is 0.
 * logp, entropy, lse : [rows] fp32; each may be NULL.
 * top_ids, top_logp : [rows, top_k] int32 and fp32; needed when top_k > 0.
 * top_k    : 0 <= top_k <= min(DS_MAX_TOP, vocab).
 * vocab    : 1 <= vocab <= DS_MAX_VOCAB.  rows >= 0 (0: no-op).
 *
 * A token with z = -infinity is masked: probability 0, logp -infinity,
 * never listed.  A list with fewer than top_k unmasked tokens ends in id -1
 * and log probability -infinity.  A row with every token masked has lse
 * -infinity, entropy 0 and logp -infinity (0 if ignored).  A row holding a
 * NaN or +infinity has NaN for its three numbers and its list's log
 * probabilities; the list orders the values that are numbers.
 */
int ds_logprob_rows(const void* logits, int32_t logits_type, int64_t ld, const float* scale,
                    float inv_temp, const void* labels, int32_t label_bytes, float* logp,
                    float* entropy, float* lse, int32_t* top_ids, float* top_logp, int32_t top_k,
                    int64_t rows, int64_t vocab, void* workspace, int64_t workspace_bytes,
                    ds_stream_t stream);

/* Bytes of workspace of that call (a negative status for sizes it refuses). */
int64_t ds_logprob_rows_workspace(int64_t rows, int64_t vocab, int32_t top_k);

/*
 * ds_logprob_rows_backward -- the gradient of ds_logprob_rows' logp and
 * entropy (top alternatives pass none).
 *
 *   dz_j      = dlogp ([j = label] - p_j) - dentropy p_j (z_j - lse + entropy)
 *   dlogits_j = dz_j inv_temp scale_j            in logits_type
 *   dscale_j  = sum over rows of dz_j inv_temp x_j          fp32: up to 32 rows
 *               in fp32, these sums in fp64
 *
 * lse, entropy : the forward call's outputs; entropy may be NULL when
 *            dentropy is (rows with |lse| >= 2^24 then get no gradient, see
 *            below).
 * dlogp, dentropy : [rows] fp32, the gradients reaching logp and entropy;
 *            either may be NULL (zero).  An ignored row's dlogp counts as 0.
 * dlogits  : [rows, ld_out], may be logits itself (with ld_out == ld);
 *            otherwise overlapping no input.
 * dscale   : [vocab] fp32, needs scale; or NULL when not wanted.  rows == 0
 *            writes zeros.
 * A masked token (by its scale too: an infinite one, a product past fp32) gets
 * no gradient, and a row with every token masked none.
 * p_j is exp(z_j - lse) of the lse given, so it is known to |lse| 2^-24 of
 * itself: fp32 logits thousands from zero lose digits of their gradient.  From
 * |lse| = 2^24 on lse holds the row's maximum alone, and the row has a gradient
 * only where one token holds that maximum alone (a runaway logit, a temperature
 * near 0), which the entropy tells: where it is given and below 0.6875 (n equal
 * tokens have log n, 0.693 at least).  Any other such row (a finite mask, as
 * -1e30, over every token; a maximum that tokens share) counts as masked whole
 * and gets none.
 */
int ds_logprob_rows_backward(const void* logits, int32_t logits_type, int64_t ld,
                             const float* scale, float inv_temp, const void* labels,
                             int32_t label_bytes, const float* lse, const float* entropy,
                             const float* dlogp, const float* dentropy, void* dlogits,
                             int64_t ld_out, float* dscale, int64_t rows, int64_t vocab,
                             void* workspace, int64_t workspace_bytes, ds_stream_t stream);

/* Bytes of workspace of that call (needed only when dscale is wanted). */
int64_t ds_logprob_rows_backward_workspace(int64_t rows, int64_t vocab);

#ifdef __cplusplus
}
#endif

#endif /* DS_TOKEN_ROWS_H */
