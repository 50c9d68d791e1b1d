/*
 * pfkv_latent.h -- C ABI of libpfkv.so, continued: a paged cache that holds one
 * latent vector and one rotated key a token, shared by all heads, and the
 * attention over it in its two forms.  Conventions (memory, streams, alignment,
 * errors, hardware) are those of pfkv.h; rotations and row layouts are those of
 * pfkv_rope.h.
 *
 * With latent c_j (latent_dim values) and rotated key r_j (rope_dim values) of
 * token j, head h of a model with up-projections U_h (keys) and W_h (values)
 * attends by
 *     expanded form:  s_j = scale * (q_h . U_h c_j + qr_h . r_j),
 *                     o_h = sum_j softmax(s)_j W_h c_j
 *     absorbed form:  s_j = scale * ((U_h^T q_h) . c_j + qr_h . r_j),
 *                     o_h = W_h sum_j softmax(s)_j c_j
 * The absorbed form reads the cache itself (decode: many heads share every
 * token's latent_dim + rope_dim values); the expanded form works on keys and
 * values of 128 elements a head (prompts: fewer operations a pair).  The
 * projections are matrix products of the caller's.
 */
#ifndef PFKV_LATENT_H
#define PFKV_LATENT_H

#include "pfkv_rope.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PFKV_LATENT_DIM 512 /* the latent_dim that is built            */
#define PFKV_LATENT_ROPE 64 /* the rope_dim that is built              */
#define PFKV_LATENT_NOPE 128 /* expanded heads: elements of q and k that are not rotated */
#define PFKV_LATENT_VDIM 128 /* expanded heads: elements of v          */

/*
 * The page pool of a latent cache; pages hold PFKV_PAGE_SIZE tokens.
 *   c_pages  : [num_pages][16][latent_dim], bf16 (dtype BF16) or e4m3 bytes
 *              (dtype FP8_E4M3)
 *   r_pages  : bf16 [num_pages][16][rope_dim] for either dtype (the rotated key
 *              carries the position and is an eighth of the latent: it is not
 *              quantised)
 *   c_scale  : fp32 [num_pages] for FP8 (value = e4m3 value x page scale);
 *              ignored for BF16.  Scales are finite and positive; the attention
 *              takes one below 2^-100 for 2^-100.
 *   page_tags: uint32 [num_pages], or NULL (not tracked)
 */
typedef struct pfkv_latent_cache {
    int32_t num_pages;
    int32_t page_size;   /* must be PFKV_PAGE_SIZE   */
    int32_t latent_dim;  /* must be PFKV_LATENT_DIM  */
    int32_t rope_dim;    /* must be PFKV_LATENT_ROPE */
    int32_t dtype;       /* pfkv_kv_dtype            */
    void *c_pages;
    void *r_pages;
    float *c_scale;
    const uint32_t *page_tags;
} pfkv_latent_cache;

/* `pages` is a pfkv_pages with one table and one length per request:
 * bt_stride_h and len_stride_h must be 0. */

/*
 * pfkv_latent_append -- write new tokens' latents and rotated keys into their
 * page slots, and turn their queries' rotated parts, in one launch.
 *
 *   c_new     : rows of latent_dim elements (stride_h is not read)
 *   r_new     : rows of rope_dim elements, not yet turned (stride_h not read)
 *   q, q_out  : rows of rope_dim elements, h < num_q_heads: the queries' parts
 *               that are turned, and where they go; NULL, in place and rows past
 *               a request's tokens as in pfkv_rope_append
 *   rope      : rot_dim <= rope_dim
 *
 * FP8: the call that writes slot 0 of a page sets its scale to absmax / 448
 * (fp32 division; 1 if absmax is 0) over the latents that it writes into the
 * page; other calls keep the stored scale; each byte is the e4m3 encoding of
 * the fp32 quotient, as in pfkv_kv_append.  Turned keys are rounded once, to
 * bf16.  Checks and flags are those of pfkv_kv_append.
 */
pfkv_status pfkv_latent_append(const pfkv_latent_cache *cache, const pfkv_pages *pages,
                               const pfkv_rope *rope, const pfkv_new_tokens *tokens,
                               const pfkv_rows *c_new, const pfkv_rows *r_new,
                               const pfkv_rows *q, const pfkv_rows *q_out, int32_t num_q_heads,
                               uint8_t *flags, void *stream);

/*
 * pfkv_latent_gather -- read requests' cached tokens out of their pages as
 * contiguous bf16 rows: the operand of the up-projections that the expanded
 * form needs over a cached prefix.
 *
 *   row_starts : int32 [batch + 1]: token j < seq_lens[b] of request b goes to
 *                row row_starts[b] + j, which must lie below row_starts[b + 1]
 *                and total_rows
 *   max_seq_len: host-known upper bound of every length (0: nothing is done)
 *   c_out      : bf16, row i at c_out + i * c_stride (latent_dim elements);
 *                FP8 pools: e4m3 value x page scale, rounded to bf16
 *   r_out      : bf16, row i at r_out + i * r_stride (rope_dim elements)
 *                strides >= the row and multiples of 8; with total_rows 0 the arrays
 *                may be NULL
 *   flags      : uint8 [batch] or NULL; bits are OR-ed in, never cleared
 *
 * A request whose length or rows are out of range is flagged
 * PFKV_FLAG_BAD_LENGTH and none of its rows is written.  The rows of a page
 * whose id or tag fails its check are zero, and the request is flagged.
 * Other rows of the arrays are left as they were.
 */
pfkv_status pfkv_latent_gather(const pfkv_latent_cache *cache, const pfkv_pages *pages,
                               const int32_t *row_starts, int64_t total_rows, int32_t max_seq_len,
                               void *c_out, int64_t c_stride, void *r_out, int64_t r_stride,
                               uint8_t *flags, void *stream);

/*
 * pfkv_latent_decode_attn -- attention in the absorbed form, for the last
 * num_query_tokens tokens of every request (1 for a decode step; more to verify
 * candidates, causal among them).
 *
 *   q_c  : rows of latent_dim elements (b, t, h), t < num_query_tokens, h <
 *          num_q_heads: queries times the key up-projection
 *   q_r  : rows of rope_dim elements: the queries' rotated parts, turned
 *   out  : rows of latent_dim elements: sum_j softmax_j c_j, rounded to bf16
 *   cache: the pages are device memory (tensor copies fetch them)
 *   num_q_heads x num_query_tokens: any count >= 1 (up to 2^20 rows a request)
 *   max_seq_len: host-known upper bound of every seq_lens entry
 *   workspace  : >= pfkv_latent_decode_workspace_size(...) bytes, 256-byte
 *          aligned; contents on entry are ignored; not used by two calls at once
 *   flags: uint8 [batch], written (not OR-ed), with PFKV_FLAG_DEVICE_TIMEOUT where a
 *          wait inside the kernel gave up; may be NULL
 *
 * Query token t attends to the first n - num_query_tokens + 1 + t tokens, n =
 * seq_lens[b]; a row that attends to none is zero.  Every live page id, and its
 * tag when tags are tracked, is checked; a request with a mismatch or a bad
 * length is flagged and all of its rows are zero.  Slots past a request's last
 * token, and tokens that a row does not see, do not reach it, whatever they hold.
 *
 * Arithmetic: both products run on the tensor cores with fp32 accumulation.
 * BF16 pools: q, c, r are exact; a softmax weight is rounded once to bf16.  FP8
 * pools: e4m3 values are exact in f16; q_c enters as f16 after a power-of-two
 * scaling a row (exact for elements within 2^14 of the row's largest); a weight
 * times its page's scale is rounded once to f16 (within 2^-11, or 2^-32 of the
 * row's largest where that is more), where it enters the second product.  Scores, the
 * running maximum, the weights' sums and the merge of partial results are fp32.
 */
pfkv_status pfkv_latent_decode_workspace_size(const pfkv_latent_cache *cache, const pfkv_pages *pages,
                                              int32_t num_q_heads, int32_t num_query_tokens,
                                              int32_t max_seq_len, size_t *bytes);
pfkv_status pfkv_latent_decode_attn(const pfkv_latent_cache *cache, const pfkv_pages *pages,
                                    const pfkv_rows *q_c, const pfkv_rows *q_r, int32_t num_q_heads,
                                    int32_t num_query_tokens, float sm_scale, int32_t max_seq_len,
                                    void *workspace, size_t workspace_bytes, const pfkv_rows *out,
                                    uint8_t *flags, void *stream);

/*
 * pfkv_latent_prefill_attn -- attention in the expanded form over packed rows:
 * prompts, or parts of prompts with a prefix before them.
 *
 *   q_starts, k_starts : int32 [batch + 1]: request b holds query rows
 *             q_starts[b] .. q_starts[b+1] - 1 and key rows k_starts[b] ..
 *             k_starts[b+1] - 1; rows total_q and total_k in all.  Query ranges of
 *             two requests must not overlap (their results would race); key
 *             ranges may
 *   q_nope  : rows of 128 elements (t, h); q_rope: rows of 64, turned
 *   k_nope  : rows of 128 elements (t, h); k_rope: rows of 64, turned, one for
 *             all heads (stride_h is not read)
 *   v, out  : rows of 128 elements (t, h)
 *             stride_b of every array is not read; strides of h may interleave
 *             arrays (k_nope and v are often two halves of one row).  The arrays that
 *             are read are device memory (tensor copies fetch them).  An array with
 *             more than one row has stride_t > 0 (else PFKV_ERR_UNSUPPORTED); one
 *             without rows is not read and may be NULL
 *   max_q_len: host-known upper bound of a request's query rows (a longer one is
 *             flagged PFKV_FLAG_BAD_LENGTH); a bound far above the lengths costs time
 *   causal  : nonzero: query i of nq sees keys j <= i + nk - nq (the queries are
 *             the last of the keys' tokens); zero: every key
 *   flags   : uint8 [batch], written; PFKV_FLAG_DEVICE_TIMEOUT in all of them where a
 *             wait inside the kernel gave up (any row may then be unwritten); may be NULL
 *
 * A query that sees no key gives a zero row; keys and values that a query does not see
 * do not reach its row, whatever they hold (tiles of queries in which one that is not
 * finite might have are computed again, which costs their time twice).  A request whose rows are not
 * within the arrays is flagged and nothing of it is written.  Rows outside every
 * request's range are left as they were.  Arithmetic: tensor cores with fp32
 * accumulation, softmax statistics in fp32, a weight rounded once to bf16 where it
 * enters the second product.
 */
pfkv_status pfkv_latent_prefill_attn(int32_t batch, int32_t num_heads, const int32_t *q_starts,
                                     const int32_t *k_starts, int64_t total_q, int64_t total_k,
                                     int32_t max_q_len, const pfkv_rows *q_nope,
                                     const pfkv_rows *q_rope, const pfkv_rows *k_nope,
                                     const pfkv_rows *k_rope, const pfkv_rows *v, float sm_scale,
                                     int32_t causal, const pfkv_rows *out, uint8_t *flags,
                                     void *stream);

/*
 * pfkv_selftest_latent_decode, pfkv_selftest_latent_prefill -- the two attention calls
 * with waits that give up after `tries` tries (0 .. 100000, which is what the calls
 * themselves take; 0.2 to 4 us each; 1000 times as many for waits that last as long as
 * a tile's work), so that a test can let them run out: the call ends, requests are
 * flagged PFKV_FLAG_DEVICE_TIMEOUT (and their rows zero: decode), and the context stays
 * usable.
 */
pfkv_status pfkv_selftest_latent_decode(int32_t tries, const pfkv_latent_cache *cache,
                                        const pfkv_pages *pages, const pfkv_rows *q_c,
                                        const pfkv_rows *q_r, int32_t num_q_heads,
                                        int32_t num_query_tokens, float sm_scale,
                                        int32_t max_seq_len, void *workspace, size_t workspace_bytes,
                                        const pfkv_rows *out, uint8_t *flags, void *stream);
pfkv_status pfkv_selftest_latent_prefill(int32_t tries, int32_t batch, int32_t num_heads,
                                         const int32_t *q_starts, const int32_t *k_starts,
                                         int64_t total_q, int64_t total_k, int32_t max_q_len,
                                         const pfkv_rows *q_nope, const pfkv_rows *q_rope,
                                         const pfkv_rows *k_nope, const pfkv_rows *k_rope,
                                         const pfkv_rows *v, float sm_scale, int32_t causal,
                                         const pfkv_rows *out, uint8_t *flags, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PFKV_LATENT_H */
