/*
 * pfkv_prefix.h -- C ABI of libpfkv.so, continued: decode attention of a batch
 * whose requests share prefixes (a system prompt, a document), over the paged
 * cache of pfkv.h.  Conventions (memory, streams, alignment, errors, hardware)
 * are those of pfkv.h; row layouts are those of pfkv_rope.h.
 *
 * A block table lets requests name the same physical pages ("Workers AI targets the
 * inference bottleneck", section "KV cache compression goes open source"), but
 * attention request by request reads them once per request.  Here the pages of a
 * prefix have a table of their own, and its keys and values are read once for all of
 * its requests: their query rows are one matrix for the tensor cores.
 */
#ifndef PFKV_PREFIX_H
#define PFKV_PREFIX_H

#include "pfkv_rope.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Prefixes of one call. */
#define PFKV_PREFIX_MAX 4096

/*
 * pfkv_prefix_decode_attn -- attention for num_query_tokens = kq tokens of every
 * request (1 for a decode step; more to verify candidates, or for decoder tokens that
 * attend to an encoder's states).
 *
 * Request b attends to the tokens of its prefix and then to its own.  With P the
 * prefix's length for kv head h (0 without a prefix) and n = seq_lens(b, h) of `pages`,
 * query token t sees all P tokens of the prefix and the first max(0, n - kq + 1 + t)
 * of its own, the candidates being the last kq of them:
 *   out = sum_j softmax_j(sm_scale * q . k_j) v_j
 * over the tokens seen, and zero where there are none.
 *
 *   pages     : the requests' own tokens (pages->batch must be `batch`); NULL: no request
 *               has any, and out is attention to the prefix alone
 *   prefixes  : tables, lengths and expected tags of the prefixes, prefixes->batch of
 *               them (0: none, the rest is not read), at most PFKV_PREFIX_MAX; strides
 *               and heads as for requests
 *   prefix_of : int32 [batch], the request's prefix, or -1 for none.  Any number of
 *               requests may share a prefix, in any order
 *   q, out    : bf16 rows (b, t, hq) of head_dim elements; out may be q
 *   num_q_heads: a multiple G of num_kv_heads with G in {1, 2, 4, 8}
 *   max_seq_len, max_prefix_len: host-known upper bounds of the lengths (a longer one is
 *               flagged PFKV_FLAG_BAD_LENGTH), 2^30 at most; max_seq_len is not read without
 *               pages
 *   attn_mass : NULL, or as in pfkv_paged_decode_attn_mass for the requests' own tokens:
 *               to each is added its softmax weight, normalised over all that the row
 *               sees, summed over the G query heads.  Needs pages and kq = 1
 *   workspace : >= pfkv_prefix_decode_workspace_size(...) bytes (with_mass nonzero when
 *               attn_mass is given), 256-byte aligned; contents on entry are ignored; not
 *               used by two calls at once
 *   flags     : uint8 [batch] or NULL, written (not OR-ed)
 *
 * The pools are device memory.  Page ids, lengths and tags of requests and prefixes are
 * checked before any page is read; a request that fails, or whose prefix does, is flagged
 * and all of its rows are zero (and add no mass), as is one whose prefix_of is neither -1
 * nor below prefixes->batch (PFKV_FLAG_BAD_PAGE).  Every wait of the kernels is bounded: when one over
 * the prefixes gives up, all requests that have a prefix are flagged PFKV_FLAG_DEVICE_TIMEOUT and
 * zero; when one over own tokens does, that request is flagged and its rows of that kv head are zero
 * (and no mass is added).  Slots past a last token do not reach
 * any row, whatever they hold; a score that is NaN or +inf, over the prefix or among own tokens,
 * makes its row NaN, and the totals that the row adds to; a value that is NaN or infinite makes
 * its element of the rows that see it NaN or infinite.
 *
 * Arithmetic: scores, softmax statistics, sums and the merge of partial results are fp32;
 * own tokens are those of pfkv_paged_decode_attn.  Over a prefix, BF16 pools: q, k, v are
 * exact and a softmax weight enters the second product as a pair of bf16 values whose sum is
 * within 2^-16 of it; sums are finite for values up to 2^90, whatever the scores.
 * FP8 pools: e4m3 values are exact; q enters as a pair of an e4m3 and an e5m2 value after a
 * power-of-two scaling of its row (exact for elements within 2^13 of the row's largest, others
 * within 2^-21 of it); a weight
 * times its unit's V scale enters as a pair of f16 values (within 2^-22 of it, or, where that is
 * more, within 2^-30 of the row's largest weight times the largest V scale that the prefix's pages
 * have for the kv head, whether its page gets weight or holds zeros, whose scale is 1).
 */
pfkv_status pfkv_prefix_decode_workspace_size(const pfkv_cache *cache, const pfkv_pages *pages,
                                              const pfkv_pages *prefixes, int32_t batch,
                                              int32_t num_q_heads, int32_t num_query_tokens,
                                              int32_t max_seq_len, int32_t max_prefix_len,
                                              int32_t with_mass, size_t *bytes);
pfkv_status pfkv_prefix_decode_attn(const pfkv_cache *cache, const pfkv_pages *pages,
                                    const pfkv_pages *prefixes, int32_t batch,
                                    const int32_t *prefix_of, const pfkv_rows *q,
                                    int32_t num_q_heads, int32_t num_query_tokens, float sm_scale,
                                    int32_t max_seq_len, int32_t max_prefix_len, void *workspace,
                                    size_t workspace_bytes, const pfkv_rows *out, float *attn_mass,
                                    int64_t mass_stride_b, int64_t mass_stride_h, uint8_t *flags,
                                    void *stream);

/*
 * pfkv_selftest_prefix_decode -- the call with waits that give up after `tries` tries
 * (0 .. 100000, which is what the call itself takes; 0.2 to 4 us each; 1000 times as many for
 * waits that last as long as a segment's work), so that a test can let them run out: the call
 * ends, every request with a prefix is flagged PFKV_FLAG_DEVICE_TIMEOUT and its rows are zero,
 * and the context stays usable.
 */
pfkv_status pfkv_selftest_prefix_decode(int32_t tries, const pfkv_cache *cache,
                                        const pfkv_pages *pages, const pfkv_pages *prefixes,
                                        int32_t batch, const int32_t *prefix_of, const pfkv_rows *q,
                                        int32_t num_q_heads, int32_t num_query_tokens,
                                        float sm_scale, int32_t max_seq_len, int32_t max_prefix_len,
                                        void *workspace, size_t workspace_bytes,
                                        const pfkv_rows *out, float *attn_mass,
                                        int64_t mass_stride_b, int64_t mass_stride_h,
                                        uint8_t *flags, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PFKV_PREFIX_H */
