/*
 * kvring_paged — a paged FP8 KV cache for many sequences on one GPU (sm_103a)
 * and the attention that reads it.
 *
 * Where kvring.h keeps one ring per cache, this cache is a pool of pages of
 * page_tokens tokens that the caller hands out to sequences: a page table per
 * call says which pages a sequence holds, in order.  Sequences of any lengths
 * are worked on in one call (packed rows, no padding), a single new token or
 * a whole prompt each.
 *
 * Every call is asynchronous on the caller's CUDA stream, moves no data
 * between host and device (except kvring_paged_debug_state) and can be
 * captured in a CUDA graph: lengths and page tables are read on the device
 * when the kernels run, so a replayed graph follows their contents.
 *
 * Memory: the caller owns all device memory.  kvring_paged_create carves one
 * caller-allocated device workspace (kvring_paged_workspace_bytes bytes,
 * 256-byte aligned) into the state, the RoPE tables, the code and scale
 * arrays and the attention's scratch.  The handle owns host memory only.
 *
 * Numbers and layouts (L = layers, H = kv_heads, P = page_tokens, D =
 * head_dim, N = n_tokens, B = n_seqs):
 *   inputs are bf16 or fp16 as configured; a token's heads lie side by side
 *   (head h at h * D), tokens are a stride apart that the call gives, so q, k
 *   and v may be slices of one projection's output;
 *   K and V codes are e4m3 [L][n_pages][H][P][D]; K and V scales are fp32
 *   [L][n_pages][H], one for each page and head, powers of two (or 0); a
 *   cached value is code * scale.
 *
 * A batch (the same in both calls):
 *   seq_start  device int32 [B + 1]: sequence b's new tokens are rows
 *              seq_start[b] .. seq_start[b+1] - 1; rows past seq_start[B]
 *              belong to nobody and are neither read nor written
 *   kv_len     device int32 [B]: the sequence's tokens in the cache once the
 *              new ones are in; new token i of n has cache index kv_len - n + i
 *   page_table device int32 [B][table_stride], table_width used: entry j is
 *              the page of cache indices j P .. j P + P - 1; entries past the
 *              sequence's last page (and pages a window has left behind) are
 *              not read
 *   pos        device int32 [N][n_axes]: RoPE positions of the new tokens
 * A sequence whose numbers contradict each other or the call's sizes is left
 * out and flagged (KVRING_DEVERR_SEQ); a page id outside 0 .. n_pages - 1 is
 * flagged (KVRING_DEVERR_PAGE): such a page is not written, and attention reads
 * page 0 in its place.  The kernels never trap.
 * (Where seq_start decreases, sequences whose rows overlap may be left out of
 * an append as well.)
 * Non-finite inputs spread to what is computed from them and no further: a
 * query or key with a NaN to the outputs of the query heads that it belongs to
 * or that see it, a value's NaN to the same channel or the whole of them.  An
 * infinity in k or v gives its page and head the scale 2^120: the page's other
 * values there become zeros, other pages and heads are as they were.
 * A handle must not be used by two host threads at once.  The caller orders
 * calls that touch the same pages, and the attention's scratch belongs to the
 * handle: two kvring_paged_attend calls on one handle must not run at the same
 * time (one stream, or events; graphs that captured them included).
 *
 * Status codes and the device error bits are kvring.h's, with two more bits.
 */
#ifndef KVRING_PAGED_H
#define KVRING_PAGED_H

#include "kvring.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct kvring_paged kvring_paged; /* opaque host handle */

enum { KVRING_IN_BF16 = 0, KVRING_IN_F16 = 1 };

/* bits of the device-side error word, beside KVRING_DEVERR_POS_RANGE and
 * KVRING_DEVERR_TIMEOUT */
enum {
  KVRING_DEVERR_SEQ = 8,  /* a sequence's numbers contradict each other or the call's sizes */
  KVRING_DEVERR_PAGE = 16 /* a page id outside the pool */
};

/* sequences of one call; tokens of one sequence (table_width * page_tokens) */
enum { KVRING_PAGED_MAX_SEQS = 2048, KVRING_PAGED_MAX_LEN = 1 << 22 };

/*
 *   layers        >= 1: pools of the same shape, chosen by each call; a page
 *                 id means the same page in all of them (one table for all)
 *   kv_heads      1 .. 128
 *   q_heads       a multiple of kv_heads, at most 1024; query head h reads key
 *                 head h / (q_heads / kv_heads)
 *   head_dim      64 or 128
 *   page_tokens   16, 32, 64 or 128
 *   n_pages       >= 1; layers * n_pages * kv_heads * page_tokens < 2^31
 *   in_dtype      KVRING_IN_BF16 or KVRING_IN_F16: q, k, v and the output
 *   n_axes, axis_dims, pos_min, pos_count, rope_base   as kvring_config's
 */
typedef struct {
  int32_t layers;
  int32_t kv_heads;
  int32_t q_heads;
  int32_t head_dim;
  int32_t page_tokens;
  int32_t n_pages;
  int32_t in_dtype;
  int32_t n_axes;
  int32_t axis_dims[3];
  int32_t pos_min[3];
  int32_t pos_count[3];
  double rope_base;
} kvring_paged_config;

/* Bytes of device workspace (0 if the configuration is invalid). */
size_t kvring_paged_workspace_bytes(const kvring_paged_config* cfg);

/*
 * Create a cache in the caller's device workspace.  Enqueued on ``stream``:
 * zeroes the state, codes and scales, and fills the RoPE tables (cos and sin
 * of pos * omega in fp64, rounded once to fp32).
 */
int kvring_paged_create(const kvring_paged_config* cfg, void* workspace, size_t workspace_bytes,
                        kvring_stream stream, kvring_paged** out);

/*
 * Append the new tokens of every sequence (paged_append).
 *   k, v      device [N][H][D], tokens k_stride / v_stride elements apart
 *             (multiples of 8, >= H * D), 16-byte aligned; not modified
 * K is rotated by RoPE at pos (fp32, the operations of kvring_write), V is
 * not.  For each page touched and each head, K and V apart: a = the largest
 * |value| of the new rows, NaN left out; need = the smallest power of two s with
 * a <= 448 s (0 if a < 2^-100).  A page that held no row of the sequence before gets
 * scale = need; another keeps its scale unless need is larger, and then its
 * older rows' codes become e4m3(code * (old scale / need)).  New codes are
 * e4m3(x / scale), round to nearest even; 0 where the scale is 0, and 0x7F for a
 * NaN at any scale.  Rows of the page past the last new
 * one are left as they are.
 * kv_len must count the new tokens (n <= kv_len).  Pages written by a call
 * belong to one place of one sequence each: a page that two sequences of the
 * batch append to, or that a table names twice among its new tokens, ends up
 * with rows of either.
 * N (at most 2^24) or B of 0: nothing to do.
 */
int kvring_paged_append(kvring_paged* p, int32_t layer, const void* k, int64_t k_stride, const void* v,
                        int64_t v_stride, const int32_t* pos, const int32_t* seq_start, const int32_t* kv_len,
                        int32_t n_seqs, int32_t n_tokens, const int32_t* page_table, int64_t table_stride,
                        int32_t table_width, kvring_stream stream);

/*
 * Attention of the new tokens' queries over the cache (paged_attend).
 *   q        device [N][q_heads][D], tokens q_stride elements apart (a multiple
 *            of 8, >= q_heads * D), 16-byte aligned
 *   out      the same for the output, out_stride apart, apart from q; rows
 *            past seq_start[B] are left as they were
 *   max_new  the largest number of new tokens a sequence of this call has, as
 *            far as the host knows (1 .. N): it chooses what is launched.  A
 *            sequence with more is left out and flagged (KVRING_DEVERR_SEQ).
 *   causal   1: a query sees the cache indices up to its own, kv_len - n + i;
 *            0: all kv_len of them (n may then exceed kv_len)
 *   window   0, or with causal the number of indices a query sees at most,
 *            its own included
 *   scale    the softmax scale; 0: 1 / sqrt(D).  scale * log2(e) is an fp32 number
 * Queries are rotated by RoPE at q_pos (fp32) and then held in fp16 at a
 * power-of-two scale of their row; out = softmax(scale q.k) v with fp32 sums
 * and statistics and weights of V in fp16.  (A weight is rounded by half a step
 * of itself or 2^-17 of the row's largest one, whichever is more; where the V
 * scales that a part of a row meets are more than 2^14 apart, that part is
 * computed in fp32, slowly.)  A query that sees nothing gives zeros.  N * q_heads / kv_heads is at most 2^30.
 */
int kvring_paged_attend(kvring_paged* p, int32_t layer, const void* q, int64_t q_stride, const int32_t* q_pos,
                        const int32_t* seq_start, const int32_t* kv_len, int32_t n_seqs, int32_t n_tokens,
                        int32_t max_new, const int32_t* page_table, int64_t table_stride, int32_t table_width,
                        int32_t causal, int32_t window, float scale, void* out, int64_t out_stride,
                        kvring_stream stream);

/* Free the host handle (the workspace stays the caller's). NULL is allowed. */
int kvring_paged_destroy(kvring_paged* p);

/* Device pointers into the workspace: codes, scales and the int32 state words
 * {error, internal}.  Any out pointer may be NULL. */
int kvring_paged_layout(const kvring_paged* p, void** k_codes, void** v_codes, void** k_scales, void** v_scales,
                        void** state);

/* DEBUG, SYNCHRONISING: wait for ``stream`` and copy the error bits to *err. */
int kvring_paged_debug_state(const kvring_paged* p, kvring_stream stream, int32_t* err);

#ifdef __cplusplus
}
#endif
#endif /* KVRING_PAGED_H */
