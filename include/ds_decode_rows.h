/*
 * ds_decode_rows.h -- the rows of a decoding step, between its heads and its
 * next token, on AMD Instinct MI355X (gfx950).  Same library, conventions,
 * status codes and stream handle as ds_rows.h.
 *
 *  ds_rope_rows              rotary positions on q and k heads: half or
 *                            neighbouring pairs, all or part of each head
 *  ds_rope_rows_backward     its gradient
 *  ds_rope_frequencies       a frequency table, scaled for long contexts (host)
 *  ds_cache_append_rows      keys and values put into a paged cache, normed and
 *                            rotated on the way, with the step's q heads
 *  ds_cache_attention_rows   attention of each sequence's newest tokens over
 *                            the cache
 *  ds_draft_verify_rows      drafted tokens accepted by given random numbers,
 *                            and the token that follows them
 *
 * Numerics.  bf16 values are passed as their 16-bit patterns; e4m3 values are
 * the 8-bit format without infinities (largest 448).  Everything is computed
 * in fp32 (a rotation's angle and a verification's probabilities in fp64) and
 * rounded once, to nearest even, into each output.  Sums are held in fp32 or
 * more.
 *
 * Determinism.  The bits of an output row depend on that row's inputs alone
 * (its sequence's cached tokens and length among them, for attention), not on
 * the other rows, the batch, the page numbers, the grid or the stream.  No
 * atomic adds a float.
 *
 * Errors, ownership, streams, workspaces: as in ds_token_rows.h.  Every
 * argument that the host can see is checked before anything is enqueued; what
 * lies on the device (positions, lengths, page numbers, token ids) is checked
 * by the kernels, which read and write nothing outside the buffers given.
 * All calls may be captured into a HIP graph.  The library allocates nothing.
 */
#ifndef DS_DECODE_ROWS_H
#define DS_DECODE_ROWS_H

#include "ds_token_rows.h"

#ifdef __cplusplus
extern "C" {
#endif

#define DS_MAX_NEW 16                  /* most new tokens of a sequence in one attention call */
#define DS_MAX_DRAFTS 32               /* most drafted tokens of a sequence */
#define DS_MAX_PAGE 4096               /* largest page */

/* A cache's element type, beside DS_TYPE_BF16. */
enum { DS_TYPE_E4M3 = 2 };

/*
 * ds_rope_rows -- rotary positions.
 *
 * For each row with position p and each head x of q and of k:
 *   t_i = p * inv_freq_i                               in fp64, i < rotary_dim / 2
 *   (a, b) -> amplitude * (a cos t_i - b sin t_i, b cos t_i + a sin t_i)
 * for the pairs  (a, b) = (x_i, x_{i + rotary_dim / 2})      interleaved 0
 *                (a, b) = (x_{2i}, x_{2i + 1})               interleaved 1
 * of the head's first rotary_dim values; the others are copied bit for bit.
 *
 * q, q_out : [rows, ldq] / [rows, ldq_out] bf16 bit patterns, the first
 *            n_q_heads * head_dim elements of each row used; 16-byte aligned,
 *            strides multiples of 8.  q_out may be q itself (with ldq_out ==
 *            ldq); otherwise it must not overlap any input.
 * k, k_out : likewise for the n_kv_heads heads of k (may be NULL when
 *            n_kv_heads == 0).
 * positions: [rows] int32; 4-byte aligned.
 * inv_freq : [rotary_dim / 2] fp32; 4-byte aligned.
 * rotary_dim : even, 2 <= rotary_dim <= head_dim.
 * amplitude: finite (1, or what a context-scaling method raises cos and sin by).
 * head_dim : multiple of 16, 16 <= head_dim <= 256.  rows >= 0 (0: no-op).
 */
int ds_rope_rows(const uint16_t* q, int64_t ldq, const uint16_t* k, int64_t ldk,
                 const int32_t* positions, const float* inv_freq, int32_t rotary_dim,
                 int32_t interleaved, float amplitude, uint16_t* q_out, int64_t ldq_out,
                 uint16_t* k_out, int64_t ldk_out, int64_t rows, int32_t n_q_heads,
                 int32_t n_kv_heads, int32_t head_dim, ds_stream_t stream);

/*
 * ds_rope_rows_backward -- the gradient of ds_rope_rows: each pair turned back,
 * amplitude * (da cos t + db sin t, db cos t - da sin t).
 *
 * dq_out, dk_out : the gradients reaching q_out and k_out, laid out as q and k.
 * dq, dk   : receive the gradients for q and k; dq may be dq_out itself (with
 *            its stride; likewise dk).
 */
int ds_rope_rows_backward(const uint16_t* dq_out, int64_t lddq_out, const uint16_t* dk_out,
                          int64_t lddk_out, const int32_t* positions, const float* inv_freq,
                          int32_t rotary_dim, int32_t interleaved, float amplitude, uint16_t* dq,
                          int64_t lddq, uint16_t* dk, int64_t lddk, int64_t rows,
                          int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                          ds_stream_t stream);

/*
 * ds_rope_frequencies -- inv_freq for ds_rope_rows, in HOST memory.
 *
 *   f_i = base^(-2i / rotary_dim)                      in fp64, rounded to fp32
 * and, for a context `factor` times as long as the `original` positions that a
 * model was trained on, with n_i = original f_i / (2 pi) the turns of pair i
 * over them and w_i = clamp((n_i - low) / (high - low), 0, 1):
 *   inv_freq_i = f_i (w_i + (1 - w_i) / factor)
 * so pairs of more than `high` turns keep their frequency and pairs of fewer
 * than `low` are slowed by the factor.  low == high == 0 slows every pair
 * (positions interpolated); factor 1 leaves all as they are.
 *
 * rotary_dim : even, 2 <= rotary_dim <= 256.  base finite, > 0.  factor
 * finite, >= 1.  original finite, > 0.  0 <= low <= high, finite; low == high
 * only when both are 0.
 */
int ds_rope_frequencies(float* inv_freq, int32_t rotary_dim, double base, double factor,
                        double original, double low, double high);

/*
 * A paged cache of keys and values, and the table that says which pages hold
 * which sequence.  Token t of sequence s lies in page
 * page_table[s * ld_table + t / page_size] at t % page_size.
 *
 * k, v       : n_pages pages of page_size tokens of n_heads heads of head_dim
 *              elements; element e of head h of token t of page p is at
 *              p * page_stride + t * token_stride + h * head_stride + e
 *              (elements).  16-byte aligned; strides multiples of 16 bytes;
 *              k and v share the strides and no element (they may lie in
 *              one buffer).
 * type       : DS_TYPE_BF16 or DS_TYPE_E4M3.
 * k_scale, v_scale : [n_heads] fp32, 4-byte aligned, or NULL for 1: a stored
 *              value stands for itself times its head's scale.
 * page_table : [n_seqs, ld_table] int32, the first pages_per_seq of each row
 *              used.  A page below 0 or at or beyond n_pages is none: nothing
 *              is stored there and its tokens are not seen.
 * page_size  : a power of two, 1 <= page_size <= DS_MAX_PAGE.
 * head_dim   : multiple of 16, 16 <= head_dim <= 256.
 * pages_per_seq * page_size <= 2^30 tokens a sequence.
 */
typedef struct ds_kv_cache {
  void* k;
  void* v;
  const float* k_scale;
  const float* v_scale;
  const int32_t* page_table;
  int64_t page_stride, token_stride, head_stride;
  int64_t ld_table;
  int32_t type;
  int32_t n_pages;
  int32_t page_size;
  int32_t n_heads;
  int32_t head_dim;
  int32_t n_seqs;
  int32_t pages_per_seq;
} ds_kv_cache;

/*
 * ds_cache_append_rows -- a step's (or a prompt's) keys and values into the
 * cache, and its q heads beside them, in one pass.
 *
 * For row i of sequence s = seqs_i at position p = positions_i:
 *   n(x)  = x, or x / sqrt(sum x^2 / HD + eps) * weight      rms 0, 1
 *   q_out = bf16(turn_p(n(q)))
 *   K[s, p] = turn_p(n(k)),  V[s, p] = v     bf16, or e4m3(value / scale of the head)
 * with turn_p the rotation of ds_rope_rows; nothing is rounded in between.
 * Values past e4m3's range are stored as its largest; a NaN stays one.  A row
 * whose sequence, position or page is outside the cache stores nothing (its
 * q_out is written).  No two rows of a call may hold the same token of the
 * cache (which of them is stored is not defined).
 *
 * cache    : its buffers are written at those tokens alone.
 * q, q_out : as in ds_rope_rows (q_out may be q); NULL when n_q_heads == 0.
 * k, v     : [rows, ldk] / [rows, ldv] bf16 bit patterns, the first n_heads *
 *            head_dim elements used; 16-byte aligned, strides multiples of 8.
 * positions: [rows] int32.  seqs: [rows] int32; NULL gives rows / n_seqs rows
 *            in turn to each sequence (rows must be a multiple of n_seqs).
 * inv_freq, rotary_dim, interleaved, amplitude : as in ds_rope_rows;
 *            rotary_dim 0 (inv_freq may be NULL) turns nothing.
 * rms      : 0 or 1.  q_weight, k_weight : [head_dim] fp32, 16-byte aligned,
 *            or NULL for 1; NULL when rms is 0.  eps finite, >= 0.
 * A head whose sum of squares overflows or is tiny is summed scaled, as in
 * ds_qk_rows_rms.  (A unit-length head, x / sqrt(sum x^2 + eps'), is rms 1
 * with eps = eps' / HD and weights 1 / sqrt(HD).)
 */
int ds_cache_append_rows(const ds_kv_cache* cache, const uint16_t* q, int64_t ldq,
                         const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                         const int32_t* positions, const int32_t* seqs, const float* inv_freq,
                         int32_t rotary_dim, int32_t interleaved, float amplitude, int32_t rms,
                         const float* q_weight, const float* k_weight, float eps, uint16_t* q_out,
                         int64_t ldq_out, int64_t rows, int32_t n_q_heads, ds_stream_t stream);

/*
 * ds_cache_attention_rows -- attention of the `new_tokens` newest tokens of
 * each sequence (q rows s * new_tokens + j) over its cached tokens, their own
 * keys and values among them.
 *
 * With L = min(lens_s, pages_per_seq * page_size), row j stands at token
 * t = L - new_tokens + j and sees the tokens u with
 *   0 <= u <= t,   u > t - window (window 0: all),   u's page in the cache.
 * For each of its q heads g, of kv head h = g / (n_q_heads / n_heads):
 *   z_u = scale * k_scale_h * <q_g, K[s, u, h]>
 *   lse = log sum exp z_u
 *   out = bf16(v_scale_h * sum exp(z_u - lse) V[s, u, h])
 * A row that sees nothing (t < 0, no page, every z_u -infinity) has out 0 and
 * lse -infinity.  What lies in the cache at tokens that a row does not see
 * (NaN and infinity too) does not reach it.
 * The weights are formed relative to a maximum within log 2^8 of the largest z
 * so far and go into the matrix instructions as three bf16 parts, which hold
 * all their 24 bits; sums are in fp32.  Rows whose sums are not finite (V holds an infinity or a
 * NaN, or values whose sum overflows) are summed again one key at a time, which
 * is right and slow.
 *
 * Where a sequence is cut for that goes by L, n_heads and, with a window, where
 * its first row's window begins; by nothing else.
 *
 * q, out   : [rows, ldq] / [rows, ldout] bf16 bit patterns, the first
 *            n_q_heads * head_dim elements used, rows = n_seqs * new_tokens;
 *            16-byte aligned, strides multiples of 8; out overlaps no input.
 * n_q_heads: a multiple of the cache's n_heads.
 * lens     : [n_seqs] int32, tokens each sequence holds, the new ones
 *            included; below 0 counts as 0.
 * new_tokens : 1 <= new_tokens <= DS_MAX_NEW.  window >= 0.  scale: finite.
 * lse      : [rows, n_q_heads] fp32, or NULL.
 * workspace: of the size ds_cache_attention_rows_workspace returns: head_dim + 2
 *            floats for each chunk that a row's head may make by the table's
 *            capacity (pages_per_seq * page_size, or the window), at most 128,
 *            whatever the lengths are; 0 where that is one.  1,024 sequences of 32
 *            q over 8 kv heads of 128 and up to 131,072 tokens: 2.2 GB.  A cache
 *            described with the first columns of the same table, as many as the
 *            longest sequence needs, takes less and gives the same bits.
 */
int ds_cache_attention_rows(const ds_kv_cache* cache, const uint16_t* q, int64_t ldq,
                            int32_t n_q_heads, const int32_t* lens, int32_t new_tokens,
                            int32_t window, float scale, uint16_t* out, int64_t ldout, float* lse,
                            void* workspace, int64_t workspace_bytes, ds_stream_t stream);

/* Bytes of workspace of that call, from the cache's sizes (no pointer of it is
 * looked at); a negative status for sizes that it refuses. */
int64_t ds_cache_attention_rows_workspace(const ds_kv_cache* cache, int32_t n_q_heads,
                                          int32_t new_tokens, int32_t window);

/*
 * ds_draft_verify_rows -- drafted tokens against a model's probabilities, from
 * given random numbers.
 *
 * Sequence s has n_drafts + 1 rows of target logits and n_drafts rows of draft
 * logits.  In fp64, from z = x * scale * inv_temp (fp32 products in this order),
 * with exp(-d) off by at most (2 + d / 3) 2^-53 of itself:
 *   p_i = softmax of target row s * (n_drafts + 1) + i
 *   q_i = softmax of draft row s * n_drafts + i; without draft logits, 1 at
 *         the drafted token d_i and 0 elsewhere
 * Tokens are accepted in order while  u_accept_i * q_i(d_i) < p_i(d_i); a drafted
 * id outside [0, vocab) ends the drafts.  With a tokens accepted, the next is
 * the first j with
 *   sum_{k <= j} w_k > u_sample * sum_k w_k,     in ascending token order,
 *   w = max(p_a - q_a, 0) where d_a was refused, p_a where the drafts had ended
 * so the tokens are distributed as the target model's own.
 *
 * tokens   : [n_seqs, n_drafts + 1] int32: the accepted, the next one, then -1.
 * accepted : [n_seqs] int32.
 * logp     : [n_seqs, n_drafts + 1] fp32, log p_i of each token (0 past the last).
 * target, draft : rows of ldt / ldd elements of their type; the strides are at
 *            least vocab; aligned to the element.  draft NULL: certain drafts.
 * scale, draft_scale : [vocab] fp32, shared by all rows, or NULL for 1.
 * inv_temp, draft_inv_temp : finite, > 0.
 * drafted  : [n_seqs, n_drafts] int32 or int64 (id_bytes).
 * u_accept : [n_seqs, n_drafts] fp32, u_sample : [n_seqs] fp32, in [0, 1).
 * n_drafts : 0 <= n_drafts <= DS_MAX_DRAFTS (0: one token sampled from each row;
 *            draft, drafted and u_accept may be NULL).
 * vocab    : 1 <= vocab <= DS_MAX_VOCAB.  n_seqs >= 0 (0: no-op).
 *
 * A token with z = -infinity has probability 0.  A target row that is masked
 * whole or holds a NaN or +infinity has p = 0: its draft is refused, and the
 * next token is -1 with logp 0.  Such a draft row has q = 0 everywhere and
 * refuses its token: the next comes from p.  Where w is 0 everywhere (p = q to
 * rounding) it is taken as p.  Outside [0, 1), u_accept is compared as it is (a
 * NaN accepts nothing), and u_sample counts as 0 below it; at or above 1, or
 * NaN, it gives the last token of w > 0.
 */
int ds_draft_verify_rows(const void* target, int32_t target_type, int64_t ldt, const float* scale,
                         float inv_temp, const void* draft, int32_t draft_type, int64_t ldd,
                         const float* draft_scale, float draft_inv_temp, const void* drafted,
                         int32_t id_bytes, const float* u_accept, const float* u_sample,
                         int32_t* accepted, int32_t* tokens, float* logp, int64_t n_seqs,
                         int32_t n_drafts, int64_t vocab, void* workspace,
                         int64_t workspace_bytes, ds_stream_t stream);

/* Bytes of workspace of that call (a negative status for sizes it refuses). */
int64_t ds_draft_verify_rows_workspace(int64_t n_seqs, int32_t n_drafts, int64_t vocab,
                                       int32_t with_draft);

#ifdef __cplusplus
}
#endif

#endif /* DS_DECODE_ROWS_H */
