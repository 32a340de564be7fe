/*
 * kvring_latent — a paged FP8 cache for latent attention on one GPU (sm_103a)
 * and the attention of both its forms.
 *
 * In latent attention a token leaves one row: a latent vector c of C numbers,
 * which every head uses as key and as value, and a part r of R = 64 numbers,
 * rotated by RoPE, that is added to every head's key.  This cache keeps such
 * rows in pages that the caller hands out to sequences, as kvring_paged.h does
 * with keys and values; batches (seq_start, kv_len, page_table, pos), the
 * ownership of memory, streams, graphs, threads and errors are described there
 * and are the same here.
 *
 *   prompt   kvring_latent_append, then kvring_latent_read (the rows back, for
 *            the caller's product that makes keys and values of every head),
 *            then kvring_latent_attend_expanded; or kvring_latent_attend
 *   decode   kvring_latent_append, then kvring_latent_attend with the queries
 *            brought into the latent space by the caller (absorbed form)
 *
 * Numbers and layouts (L = layers, P = page_tokens, W = C + 64):
 *   codes are e4m3 [L][n_pages][P][W], a token's latent first; scales are fp32
 *   [L][n_pages][P], one for each token, powers of two.  A cached value is
 *   code * scale; a scale of NaN marks a token whose row held a NaN, an infinity
 *   or a magnitude above 448 * 2^40: its codes are zeros.  Codes are never NaN (a
 *   caller who fills the arrays keeps to that).
 *   Queries, keys, values and outputs are bf16 or fp16 as configured.  Where a
 *   call takes a token and a head stride, row (i, h) begins at i * token + h *
 *   head: both in elements, multiples of 8, rows apart from one another;
 *   pointers are 16-byte aligned.
 */
#ifndef KVRING_LATENT_H
#define KVRING_LATENT_H

#include "kvring_paged.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct kvring_latent kvring_latent; /* opaque host handle */

/* numbers of the rotated part; of a head's own key part and of its value in the
 * expanded form */
enum { KVRING_LATENT_ROPE = 64, KVRING_LATENT_HEAD = 128 };

/*
 *   layers        >= 1: pools of the same shape, chosen by each call
 *   q_heads       1 .. 256
 *   latent_dim    C: 128, 256, 384 or 512
 *   page_tokens   16, 32, 64 or 128
 *   n_pages       >= 1; layers * n_pages * page_tokens < 2^31
 *   in_dtype      KVRING_IN_BF16 or KVRING_IN_F16
 *   n_axes, axis_dims, pos_min, pos_count, rope_base   as kvring_config's, for
 *                 the rotated part: axis_dims add up to 64
 */
typedef struct {
  int32_t layers;
  int32_t q_heads;
  int32_t latent_dim;
  int32_t page_tokens;
  int32_t n_pages;
  int32_t in_dtype;
  int32_t n_axes;
  int32_t axis_dims[3];
  int32_t pos_min[3];
  int32_t pos_count[3];
  double rope_base;
} kvring_latent_config;

/* Bytes of device workspace (0 if the configuration is invalid). */
size_t kvring_latent_workspace_bytes(const kvring_latent_config* cfg);

/* Create a cache in the caller's device workspace.  Enqueued on ``stream``:
 * zeroes the state, codes and scales, and fills the RoPE tables. */
int kvring_latent_create(const kvring_latent_config* cfg, void* workspace, size_t workspace_bytes,
                         kvring_stream stream, kvring_latent** out);

/*
 * Append the new tokens of every sequence (latent_append).
 *   latent   device [N][C], tokens latent_stride elements apart (a multiple of 8, >= C)
 *   k_rope   device [N][64], tokens rope_stride elements apart (a multiple of 8, >= 64)
 * x = (latent, k_rope rotated at pos in fp32); its scale is the smallest power of
 * two s with max |x| <= 448 s, at least 2^-40; codes are e4m3(x / s), round to
 * nearest even.  Every token is by itself: nothing that was there changes.
 * kv_len must count the new tokens.  N is at most 2^24; N or B of 0: nothing to do.
 */
int kvring_latent_append(kvring_latent* p, int32_t layer, const void* latent, int64_t latent_stride,
                         const void* k_rope, int64_t rope_stride, const int32_t* pos, const int32_t* seq_start,
                         const int32_t* kv_len, int32_t n_seqs, int32_t n_tokens, const int32_t* page_table,
                         int64_t table_stride, int32_t table_width, kvring_stream stream);

/*
 * Read cached rows back (latent_read): row i of n of sequence b (out rows
 * seq_start[b] .. seq_start[b+1] - 1) is the value of its cache index
 * kv_len[b] - n + i, rounded to the cache's type (a row whose scale is NaN: all
 * NaN).  n = kv_len[b] reads all of it.
 *   out      device [N][W], rows out_stride elements apart (a multiple of 8, >= W);
 *            rows that belong to no sequence, or whose page id is outside the pool, are
 *            left as they were
 */
int kvring_latent_read(kvring_latent* p, int32_t layer, const int32_t* seq_start, const int32_t* kv_len,
                       int32_t n_seqs, int32_t n_rows, const int32_t* page_table, int64_t table_stride,
                       int32_t table_width, void* out, int64_t out_stride, kvring_stream stream);

/*
 * Attention over the cache in the absorbed form (latent_attend):
 *   out[i, h] = sum_t softmax_t(scale (q_latent[i, h] . c_t + rope(q_rope[i, h]) . r_t)) c_t
 *   q_latent device [N][q_heads][C], q_rope device [N][q_heads][64] (rotated here,
 *            at q_pos), out the same as q_latent; each with strides of its own
 *   scale    the softmax scale, 2^-100 .. 2^100
 *   causal, window, max_new   as kvring_paged_attend's
 * The products run on e4m3 codes.  A query is a sum of two (bf16) or three
 * (fp16) e4m3 numbers at a power-of-two scale of its row: off by at most 2^-8
 * (2^-12) of itself or 2^-17.8 of the row's largest number or 2^-136, whichever is
 * most (a number of q_latent is exact but for the last two).  A weight is a sum of
 * three (bf16) or four (fp16) 8-bit numbers: off by at most 2^-9 + 2^-11 (2^-13) of
 * itself, or, where that is more, 2^-28.8 (2^-27.8) of the largest product of a weight
 * and its token's scale in the row, divided by its own token's scale.  Sums and
 * statistics are fp32.
 * A query that sees nothing gives zeros.  N * q_heads is at most 2^30.
 */
int kvring_latent_attend(kvring_latent* p, int32_t layer, const void* q_latent, int64_t q_latent_token,
                         int64_t q_latent_head, const void* q_rope, int64_t q_rope_token, int64_t q_rope_head,
                         const int32_t* q_pos, const int32_t* seq_start, const int32_t* kv_len, int32_t n_seqs,
                         int32_t n_tokens, int32_t max_new, const int32_t* page_table, int64_t table_stride,
                         int32_t table_width, int32_t causal, int32_t window, float scale, void* out,
                         int64_t out_token, int64_t out_head, kvring_stream stream);

/*
 * Attention in the expanded form (latent_expanded): every head has a key part and
 * a value of its own, made by the caller from the rows.
 *   q        device [N][q_heads][128 + 64], the last 64 rotated here at q_pos
 *   k, v     device [n_keys][q_heads][128]
 *   k_rope   device [n_keys][64], rows k_rope_stride elements apart; rotated
 *            already (as kvring_latent_read gives it)
 *   kv_start device int32 [B]: sequence b's keys are rows kv_start[b] ..
 *            kv_start[b] + kv_len[b] - 1; new token i of n has index kv_len - n + i.
 *            A sequence whose rows are not all in 0 .. n_keys - 1 (kv_start beyond
 *            n_keys too) is left out and flagged KVRING_DEVERR_SEQ
 *   out      device [N][q_heads][128]
 *   scale    0: 1 / sqrt(192)
 *   causal, window, max_new   as kvring_paged_attend's
 * Rotated queries are rounded to the inputs' type once (fp16: what is beyond 65504
 * after the rotation is an infinity); weights are sums of two numbers of it; sums and
 * statistics are fp32.  A value that is no number spreads to the rows that see it, in
 * its channel or in all of the head's, and to no other.
 */
int kvring_latent_attend_expanded(kvring_latent* p, const void* q, int64_t q_token, int64_t q_head, const void* k,
                                  int64_t k_token, int64_t k_head, const void* k_rope, int64_t k_rope_token,
                                  const void* v, int64_t v_token, int64_t v_head, int32_t n_keys, const int32_t* q_pos,
                                  const int32_t* seq_start, const int32_t* kv_start, const int32_t* kv_len,
                                  int32_t n_seqs, int32_t n_tokens, int32_t max_new, int32_t causal, int32_t window,
                                  float scale, void* out, int64_t out_token, int64_t out_head, kvring_stream stream);

/* Free the host handle (the workspace stays the caller's). NULL is allowed. */
int kvring_latent_destroy(kvring_latent* p);

/* Device pointers into the workspace: codes, scales and the int32 state words
 * {error, internal}.  Any out pointer may be NULL. */
int kvring_latent_layout(const kvring_latent* p, void** codes, void** scales, void** state);

/* DEBUG, SYNCHRONISING: wait for ``stream`` and copy the error bits to *err. */
int kvring_latent_debug_state(const kvring_latent* p, kvring_stream stream, int32_t* err);

#ifdef __cplusplus
}
#endif
#endif /* KVRING_LATENT_H */
