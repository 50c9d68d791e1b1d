/*
 * pfkv_rope.h -- C ABI of libpfkv.so, continued: appending keys and values to
 * the paged cache of pfkv.h with the rotary position embedding applied on the
 * way.  Conventions (memory, streams, alignment, errors, hardware) are those of
 * pfkv.h.
 *
 * A rotation turns each pair (x_i, x_j) of a row's first rot_dim elements by
 * the angle a = position * inv_freq[i]:
 *     x_i' = scale * (x_i cos a - x_j sin a)
 *     x_j' = scale * (x_j cos a + x_i sin a)
 * The angle is reduced to a fraction of a turn exactly, in 64-bit fixed point
 * (inv_freq / 2 pi is rounded once to 2^-64 of a turn, or to fp64's 53 bits
 * where that is coarser), so that a far position costs no accuracy; sine,
 * cosine and the products are fp32.
 */
#ifndef PFKV_ROPE_H
#define PFKV_ROPE_H

#include "pfkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The rotation. */
typedef struct pfkv_rope {
    const float *inv_freq;  /* fp32 [rot_dim / 2], radians per position          */
    int32_t rot_dim;        /* elements turned: a multiple of 16, at most the row */
    int32_t interleaved;    /* 0: element i pairs with i + rot_dim / 2;
                               1: element 2i pairs with 2i + 1                    */
    float scale;            /* multiplies the turned elements (1: plain rotation) */
} pfkv_rope;

/*
 * bf16 rows in the caller's layout: row (b, t, h) starts at element
 * b*stride_b + t*stride_t + h*stride_h of data and its elements are
 * contiguous.  data 16-byte aligned; strides >= 0 and multiples of 8.
 * With packed rows (row_starts below) row (b, t, h) starts at
 * (row_starts[b] + t)*stride_t + h*stride_h, and stride_b is not read.
 */
typedef struct pfkv_rows {
    void *data;
    int64_t stride_b, stride_t, stride_h;
} pfkv_rows;

/*
 * The new tokens of an append.
 *   num_new_tokens : T >= 1, host-known upper bound of every request's count
 *   positions      : int32, cache position of the first new token of (b, h), as
 *                    in pfkv_kv_append (length strides of `pages`)
 *   new_lens       : int32 (same indexing) number of new tokens; NULL: T (padded
 *                    rows) or row_starts[b+1] - row_starts[b] (packed rows).
 *                    With packed rows the smaller of the two counts holds.
 *   rope_positions : int32 [batch], the position that turns the first new token
 *                    of request b (it may differ from the cache position, for
 *                    instance after evictions, and may be negative); NULL: the
 *                    cache position, which needs one length per request
 *                    (len_stride_h 0, else PFKV_ERR_INVALID_ARG)
 *   row_starts     : int32 [batch + 1], or NULL for padded rows: packed rows,
 *                    request b holding rows row_starts[b] .. row_starts[b+1] - 1
 *   total_rows     : packed: rows that the arrays hold (0: the arrays are not read and
 *                    their data may be NULL).  A request whose range is
 *                    not within [0, total_rows] or longer than T is flagged
 *                    PFKV_FLAG_BAD_LENGTH and nothing of it is read or written.
 */
typedef struct pfkv_new_tokens {
    int32_t num_new_tokens;
    const int32_t *positions;
    const int32_t *new_lens;
    const int32_t *rope_positions;
    const int32_t *row_starts;
    int64_t total_rows;
} pfkv_new_tokens;

/*
 * pfkv_rope_append -- turn new tokens' queries and keys by their positions and
 * write keys and values into their page slots: pfkv_kv_append with the
 * rotation on the way, in one launch.
 *
 *   k_new, v_new : rows of head_dim elements, h < num_kv_heads
 *   q, q_out     : rows of head_dim elements, h < num_q_heads (any count >= 1);
 *                  q_out receives the turned queries, rounded to bf16.  Both
 *                  NULL: no queries.  q_out may be q itself (same data and
 *                  strides); otherwise the two must not overlap.  Query rows of
 *                  a request are turned for its first n tokens, n the count of
 *                  kv head 0; rows past them are not written.
 *   flags        : uint8 [batch] or NULL; bits are OR-ed in, never cleared
 *
 * Keys are turned in fp32 and rounded once: to e4m3 of the fp32 quotient by the
 * unit's scale (FP8 pool), or to bf16.  Scales, slots, checks of page ids and
 * tags, and flags are those of pfkv_kv_append; values get exactly its bytes.
 * A destination that fails a check is not written; queries are turned all the
 * same.  Two calls, or two (b, h), that write the same unit concurrently race.
 */
pfkv_status pfkv_rope_append(const pfkv_cache *cache, const pfkv_pages *pages,
                             const pfkv_rope *rope, const pfkv_new_tokens *tokens,
                             const pfkv_rows *k_new, const pfkv_rows *v_new,
                             const pfkv_rows *q, const pfkv_rows *q_out, int32_t num_q_heads,
                             uint8_t *flags, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PFKV_ROPE_H */
