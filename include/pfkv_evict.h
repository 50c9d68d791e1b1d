/*
 * pfkv_evict.h -- C ABI of libpfkv.so, continued: eviction from the paged cache
 * of pfkv.h by accumulated attention weight.  Conventions (memory, streams,
 * alignment, errors, hardware) are those of pfkv.h.
 *
 * pfkv_paged_decode_attn_mass and pfkv_prefix_decode_attn keep, for every token
 * of a (request, kv head), the sum of the softmax weights that it has received.
 * "Workers AI targets the inference bottleneck" (section "KV cache compression
 * goes open source", 3rd paragraph) evicts the entries with the lowest total, and
 * lets every head keep a number of tokens of its own.
 */
#ifndef PFKV_EVICT_H
#define PFKV_EVICT_H

#include "pfkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * pfkv_kv_evict -- move the tokens that are kept to new pages.
 *
 * For every (b, h), with n = seq_lens of `src` and k = min(keep_lens, n):
 *   the first  f = min(keep_first, k) tokens and
 *   the last   l = min(keep_last, k - f) are kept, and
 *   of those between, the k - f - l with the largest attn_mass; of equal totals
 *   the lower index.  A total that is NaN counts as larger than any other, and
 *   -0 as 0.
 * The kept tokens go, in their order, to slots 0 .. k - 1 of the pages of `dst`.
 *
 *   src       : the tokens as they are; its pages are read and stay as they were, so
 *               they may be shared with other requests
 *   dst       : batch, max_pages, tables (with strides of their own) and expected tags
 *               of the pages that receive the kept tokens, ceil(k / 16) a (b, h); its
 *               lengths are not read (seq_lens may be NULL).  No page of dst may be a
 *               live page of src or belong to two (b, h): such a call races
 *   keep_lens : int32, indexed with the length strides of `src`
 *   attn_mass : float, total of token j of (b, h) at b*mass_stride_b + h*mass_stride_h + j
 *   max_seq_len, max_keep_len: host-known upper bounds of seq_lens and of k (2^30 at most, as
 *               is new_mass_len).  They size the launches: bounds far above the lengths cost time
 *               where there are many heads (32 x 8 of up to 8,192 tokens: 58 us, with four times
 *               the bounds 79)
 *   new_lens  : int32, written with k (0 for a flagged request); length strides of `src`
 *               (stride_b > 0 for more than one request).  May be seq_lens or keep_lens
 *   new_mass  : float, NULL or rows of new_mass_len >= max_keep_len elements: the kept
 *               tokens' totals at 0 .. k - 1, zero at k .. new_mass_len - 1 (tokens that
 *               will be appended).  Must not overlap attn_mass
 *   kept      : int32, NULL or rows of >= max_keep_len elements: the old index of the
 *               token in slot j < k; the rest of a row is left as it was
 *               (strides in elements, >= 0; rows must not overlap)
 *   workspace : >= pfkv_kv_evict_workspace_size(...) bytes, 256-byte aligned; contents on
 *               entry are ignored; not used by two calls at once
 *   flags     : uint8 [batch] or NULL, written (not OR-ed)
 *
 * FP8: a unit of dst whose tokens all come from one unit of src gets its bytes and its
 * scales unchanged.  Any other gets, for K and for V, the scale absmax / 448 (fp32
 * division; 1 if absmax is 0) over its tokens' values (fp32 product of e4m3 value and
 * scale), and bytes that are the e4m3 encoding of the fp32 quotient, as in
 * pfkv_kv_append.  BF16: values are copied.  Slots of a last page past token k - 1 are
 * left as they were.
 *
 * A length outside its bounds, or a k above max_keep_len or dst's table, flags the
 * request PFKV_FLAG_BAD_LENGTH; live table entries of src, and those of dst that are
 * written, are checked like pfkv_paged_decode_attn's (PFKV_FLAG_BAD_PAGE,
 * PFKV_FLAG_TAG_MISMATCH).  Of a flagged request nothing but new_lens is written.
 */
pfkv_status pfkv_kv_evict_workspace_size(const pfkv_cache *cache, const pfkv_pages *src,
                                         int32_t max_seq_len, int32_t max_keep_len,
                                         size_t *bytes);
pfkv_status pfkv_kv_evict(const pfkv_cache *cache, const pfkv_pages *src, const pfkv_pages *dst,
                          const int32_t *keep_lens, int32_t keep_first, int32_t keep_last,
                          const float *attn_mass, int64_t mass_stride_b, int64_t mass_stride_h,
                          int32_t max_seq_len, int32_t max_keep_len, void *workspace,
                          size_t workspace_bytes, int32_t *new_lens, float *new_mass,
                          int64_t new_mass_stride_b, int64_t new_mass_stride_h,
                          int32_t new_mass_len, int32_t *kept, int64_t kept_stride_b,
                          int64_t kept_stride_h, uint8_t *flags, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PFKV_EVICT_H */
